"""GPU parity of the weight-only linear layer (BF16 / FP16 rows, NVFP4 weights).

The expected product is the oracle's FP64 product of the dequantized weights.  Error bound,
from the arithmetic: x * e2m1 * e4m3 is exact in the MMA's operands (FP16, or BF16 where a row's
values span too many binades); the FP32 accumulation over K terms in any order, with the
multiplication by s2 and the exact power-of-two descaling, errs by at most
(K + 4) * 2^-23 * sum|x||w| -- each addition rounds its partial sum by at most 2^-23 (the tensor
core truncates) -- for which (K/16 + 40) * 2^-23 * sum|x||w| is used here: an MMA adds 16 products
at once, and at most 40 more additions follow; rounding to the output adds eps / 2.
"""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def weights(rng, N, K, lo=0x20, hi=0x48):
    return (rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(lo, hi + 1, (N, K // 16), dtype=np.uint8))


def rows(rng, T, K, dt, spread=False):
    x = rng.laplace(size=(T, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 200))] *= 50.0
    if spread:                                              # exponents over the whole BF16 range
        x *= np.exp2(rng.integers(-60, 60, (T, K))).astype(np.float32)
    return torch.from_numpy(x).to(DT[dt])


def check(orc, x, q, sc, s2, out_dt, out=None):
    K = x.shape[1]
    f = G.flags_dev()
    d_s2 = torch.tensor([s2], dtype=torch.float32, device=G.DEV)
    if out is None:
        out = nv4.linear_w4a16(x, G.u8_dev(q), G.u8_dev(sc), d_s2, dtype=DT[out_dt], d_flags=f)
    else:
        nv4.nv4_linear_w4a16(x, G.u8_dev(q), G.u8_dev(sc), d_s2, out, f)
    torch.cuda.synchronize()
    assert f.item() == 0
    y, yabs = orc.linear_w4a16(x.double().cpu().numpy(), q, sc, float(np.float32(s2)))
    got = out.double().cpu().numpy()
    tol = (K / 16 + 40) * 2.0 ** -23 * yabs + torch.finfo(DT[out_dt]).eps / 2 * np.abs(y) + 1e-38
    if out_dt == "fp16":
        tol = tol + 2.0 ** -25                              # FP16 subnormals
    err = np.abs(got - y)
    assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(err > tol)[:4].tolist())


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 24, 25, 61, 130])
@pytest.mark.parametrize("N,K,dt,out", [(64, 256, "bf16", "bf16"), (300, 1040, "fp16", "fp32"),
                                        (2880, 2880, "bf16", "fp16")])
def test_linear_tokens(orc, T, N, K, dt, out):
    rng = np.random.default_rng(T + N)
    q, sc = weights(rng, N, K)
    check(orc, rows(rng, T, K, dt).to(G.DEV), q, sc, 0.0031, out)


@pytest.mark.parametrize("N,K", [(1, 16), (1, 64), (3, 48), (17, 32), (5, 16384), (149, 80), (1000, 2064), (20000, 64)])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_linear_odd_sizes(orc, N, K, T):
    rng = np.random.default_rng(N + K)
    q, sc = weights(rng, N, K, lo=0, hi=0x7E)
    check(orc, rows(rng, T, K, "bf16").to(G.DEV), q, sc, 1.0, "fp32")


@pytest.mark.parametrize("T,N,K,dt,out", [
    (33, 3000, 4096, "bf16", "bf16"), (128, 128, 64, "fp16", "fp32"), (129, 140, 192, "bf16", "fp16"),
    (256, 256, 2048, "bf16", "bf16"), (600, 2880, 656, "fp16", "bf16"), (1025, 5000, 320, "bf16", "fp32"),
    (700, 20000, 80, "bf16", "bf16")])
def test_linear_many_rows(orc, T, N, K, dt, out):
    """Every token tile width, clusters that split K and tiles that wrap around the SMs."""
    rng = np.random.default_rng(T * N)
    q, sc = weights(rng, N, K)
    check(orc, rows(rng, T, K, dt).to(G.DEV), q, sc, 0.0031, out)


@pytest.mark.parametrize("T", [1, 9, 70])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_linear_strides(orc, T, dt):
    """Rows inside a wider tensor whose padding holds NaN; an output inside a wider tensor, whose
    padding stays as it was (row pitch of no particular alignment)."""
    rng = np.random.default_rng(T)
    N, K = 203, 544
    q, sc = weights(rng, N, K)
    wide = torch.full((T, K + 24), float("nan"), dtype=DT[dt], device=G.DEV)
    wide[:, :K] = rows(rng, T, K, dt).to(G.DEV)
    dst = torch.full((T, N + 3), 7.0, dtype=torch.float32, device=G.DEV)
    check(orc, wide[:, :K], q, sc, 0.02, "fp32", dst[:, :N])
    assert torch.all(dst[:, N:] == 7.0)


@pytest.mark.parametrize("T", [1, 6, 33])
def test_linear_wide_rows(orc, T):
    """BF16 rows spanning more binades than FP16 holds: one element at 2^60 facing a zero code must
    not cost the small ones their bits; BF16 subnormals; all-zero rows."""
    rng = np.random.default_rng(100 + T)
    N, K = 96, 512
    q, sc = weights(rng, N, K)
    q[:, 0] &= 0xF0                                          # element 0 of every weight row is +0
    x = rows(rng, T, K, "bf16")
    x[0, 0] = 2.0 ** 60
    x[0, 1:] *= 2.0 ** -20
    if T > 1:
        x[1] = 0.0
        x[2] = rows(rng, 1, K, "bf16", spread=True)[0]
        x[3] = 2.0 ** -130                                   # subnormals
    check(orc, x.to(G.DEV), q, sc, 0.5, "fp32")


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** -18, 2.0 ** 9, 2.0 ** 30])
def test_linear_rows_of_other_magnitudes(orc, scale):
    """Rows outside the range that the first conversion holds exactly."""
    rng = np.random.default_rng(8)
    q, sc = weights(rng, 130, 608)
    check(orc, (rows(rng, 5, 608, "bf16") * scale).to(G.DEV), q, sc, 0.125, "fp32")


def test_linear_nonfinite_propagates(orc):
    rng = np.random.default_rng(5)
    q, sc = weights(rng, 40, 128)
    q |= 0x11                                                # no zero codes
    x = rows(rng, 4, 128, "bf16").to(G.DEV)
    x[1, 3] = float("inf")
    x[2, 100] = float("nan")
    sc[7, 2] = 0x7F                                          # a NaN scale
    y = nv4.linear_w4a16(x, G.u8_dev(q), G.u8_dev(sc), torch.ones(1, device=G.DEV), dtype=torch.float32).cpu()
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, 7]).all()
    keep = [n for n in range(40) if n != 7]
    assert torch.isinf(y[1, keep]).all() and torch.isfinite(y[0, keep]).all() and torch.isfinite(y[3, keep]).all()


def test_linear_rows_do_not_depend_on_the_batch():
    """The same call twice gives the same bits; an empty batch is a no-op."""
    rng = np.random.default_rng(6)
    q, sc = (G.u8_dev(a) for a in weights(rng, 500, 1024))
    x = rows(rng, 20, 1024, "bf16").to(G.DEV)
    s2 = torch.full((1,), 0.01, device=G.DEV)
    a, b = (nv4.linear_w4a16(x, q, sc, s2, dtype=torch.float32) for _ in range(2))
    assert torch.equal(a, b)
    assert nv4.linear_w4a16(x[:0], q, sc, s2).shape == (0, 500)


def test_linear_streams_and_graph():
    """Two streams at once, and a captured call replayed on new inputs."""
    rng = np.random.default_rng(7)
    q, sc = (G.u8_dev(a) for a in weights(rng, 1024, 2048))
    s2 = torch.full((1,), 0.01, device=G.DEV)
    xs = [rows(rng, 3, 2048, "bf16").to(G.DEV) for _ in range(4)]
    want = [nv4.linear_w4a16(x, q, sc, s2) for x in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [nv4.linear_w4a16(x, q, sc, s2, stream=st[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xin, out = xs[0].clone(), torch.empty_like(want[0])
    nv4.nv4_linear_w4a16(xin, q, sc, s2, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv4.nv4_linear_w4a16(xin, q, sc, s2, out)
    for x, w in zip(xs, want):
        xin.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_one_row_of_a_matrix_with_an_odd_pitch():
    """The distance to a next row that is not there is no reason to refuse a call."""
    gen = torch.Generator(device=G.DEV).manual_seed(3)
    big = torch.randn((3, 133), generator=gen, device=G.DEV).to(torch.bfloat16)
    q = torch.randint(0, 256, (40, 64), generator=gen, dtype=torch.uint8, device=G.DEV)
    sc = torch.full((40, 8), 0x38, dtype=torch.uint8, device=G.DEV)
    s2 = torch.ones(1, device=G.DEV)
    assert torch.equal(nv4.linear_w4a16(big[:1, :128], q, sc, s2), nv4.linear_w4a16(big[:1, :128].clone(), q, sc, s2))
    sm = nv4.mma_scales(torch.full((40, 4), 127, dtype=torch.uint8, device=G.DEV))
    assert torch.equal(nv4.linear_mxfp4(big[:1, :128], q, sm), nv4.linear_mxfp4(big[:1, :128].clone(), q, sm))
    with pytest.raises(nv4.NV4Error):
        nv4.linear_w4a16(big[:2, :128], q, sc, s2)


@pytest.mark.parametrize("T,N", [(17, 100), (20, 2048), (64, 2500), (128, 700), (129, 1290)])
@pytest.mark.parametrize("K", [528, 1280, 2576, 8208])
def test_linear_split_k(orc, T, N, K):
    """Few tiles and long K: clusters of every size share a tile's K, with uneven parts."""
    rng = np.random.default_rng(T + K)
    q, sc = weights(rng, N, K)
    check(orc, rows(rng, T, K, "bf16").to(G.DEV), q, sc, 0.0031, "bf16")
