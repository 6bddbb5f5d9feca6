"""GPU parity of the MXFP4 x MXFP4 product and of the quantizer that feeds it.

Codes and scales are bit-exact.  Product: e2m1 * e2m1 * 2^e is exact; the FP32 accumulation adds
K/64 MMA partial sums, each of 64 products that the tensor core adds with a relative error below
2^-23 of their absolute sum: (K/64 + 4) * 2^-23 * sum|a||b|, plus one rounding to BF16 (2^-8).
"""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu


def operand(rng, rows, K, lo=110, hi=140):
    return (rng.integers(0, 256, (rows, K // 2), dtype=np.uint8), rng.integers(lo, hi + 1, (rows, K // 32), dtype=np.uint8))


def check(orc, qa, ea, qb, eb, dtypes=(torch.float32, torch.bfloat16), out=None):
    K = 2 * qa.shape[1]
    D, Dabs = orc.gemm_mxfp4(qa, ea, qb, eb)
    args = [G.u8_dev(qa), nv4.mma_scales(G.u8_dev(ea)), G.u8_dev(qb), nv4.mma_scales(G.u8_dev(eb))]
    for dt in dtypes:
        f = G.flags_dev()
        if out is None:
            got = nv4.gemm_mxfp4(*args, dtype=dt, d_flags=f)
        else:
            nv4.nv4_gemm_mxfp4(*args, out, f)
            got = out
        torch.cuda.synchronize()
        assert f.item() == 0
        tol = (K / 64 + 4) * 2.0 ** -23 * Dabs + torch.finfo(got.dtype).eps / 2 * np.abs(D) + 1e-38
        err = np.abs(got.double().cpu().numpy() - D)
        assert np.all(err <= tol), (dt, float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2880), (127, 96), (128, 128), (129, 160), (300, 1056), (1001, 2880)])
def test_quant_mma_matches_oracle(orc, dt, rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = (rng.laplace(size=(rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, cols // 32)).repeat(32, 1))).astype(np.float32)
    x[0, :32] = 0.0
    x[-1, -32:] = 2.0 ** -140 if dt == "fp32" else 0.0
    t = torch.from_numpy(x).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    wide = torch.full((rows, cols + 8), float("nan"), dtype=t.dtype, device=G.DEV)
    wide[:, :cols] = t.to(G.DEV)
    f = G.flags_dev()
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=G.DEV)
    n = nv4.nv4_mxfp4_mma_scale_bytes(rows, cols)
    sf = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device=G.DEV)
    nv4.nv4_mxfp4_quant_mma(wide[:, :cols], q, sf, f)
    torch.cuda.synchronize()
    xo = G.host(t.to(G.DEV)) if dt == "bf16" else t.numpy()
    oq, oe, _ = orc.mxfp4_quant(np.ascontiguousarray(xo))
    assert f.item() == 0 and np.array_equal(G.host(q), oq)
    assert np.array_equal(G.host(sf[:n]), orc.scales_to_mma_layout(oe)) and torch.all(sf[n:] == 0xAB)


def test_quant_mma_flags_nonfinite():
    x = torch.ones((2, 64), dtype=torch.bfloat16, device=G.DEV)
    x[1, 40] = float("inf")
    f = G.flags_dev()
    _, sf = nv4.mxfp4_quant_mma(x, d_flags=f)
    assert f.item() == nv4.FLAG_NONFINITE and sf[16 + 1].item() == 0xFF and sf[16].item() == 125


@pytest.mark.parametrize("M", [1, 5, 16, 17, 64, 100, 128, 129, 256, 300])
@pytest.mark.parametrize("N,K", [(1, 32), (130, 96), (256, 256), (77, 1184), (513, 2880)])
def test_gemm_sizes(orc, M, N, K):
    rng = np.random.default_rng(M * N + K)
    check(orc, *operand(rng, M, K), *operand(rng, N, K))


def test_gemm_many_tiles(orc):
    """Several tiles per CTA pair, odd numbers of stages and of scale atoms."""
    rng = np.random.default_rng(1)
    check(orc, *operand(rng, 2200, 416), *operand(rng, 4100, 416), dtypes=(torch.float32,))


def test_gemm_small_integers_exact(orc):
    """Scales 1: every product is a multiple of 1/4 and the sums are small: exact in FP32, so the
    scale of each step and each K position is pinned."""
    rng = np.random.default_rng(2)
    for M, N, K in ((40, 70, 608), (300, 260, 608)):
        qa, ea = operand(rng, M, K, 127, 127)
        qb, eb = operand(rng, N, K, 127, 127)
        # one block at a time carries a scale of its own: a wrong scale byte cannot cancel
        ea[:, :] = 120 + (np.arange(K // 32) % 5)
        D, _ = orc.gemm_mxfp4(qa, ea, qb, eb)
        got = nv4.gemm_mxfp4(G.u8_dev(qa), nv4.mma_scales(G.u8_dev(ea)), G.u8_dev(qb), nv4.mma_scales(G.u8_dev(eb)),
                             dtype=torch.float32)
        assert np.array_equal(got.double().cpu().numpy(), D)


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gemm_output_strides(orc, M, dt):
    """An output inside a wider tensor, with row pitches that keep 16-byte alignment and not."""
    rng = np.random.default_rng(3)
    qa, ea = operand(rng, M, 288)
    qb, eb = operand(rng, 203, 288)
    for pad in (5, 3):                                       # 208: aligned, 206: not
        dst = torch.full((M, 203 + pad), 9.0, dtype=dt, device=G.DEV)
        check(orc, qa, ea, qb, eb, dtypes=(dt,), out=dst[:, :203])
        assert torch.all(dst[:, 203:] == 9.0)


@pytest.mark.parametrize("M,N,pad", [(517, 515, 0), (517, 515, 5), (300, 769, 0), (517, 514, 2), (259, 512, 1)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gemm_unaligned_rows_of_tall_products(orc, M, N, pad, dt):
    """Several tiles of the tall kernel with an odd row pitch, a ragged last tile, or both; what lies
    between the rows stays as it was."""
    rng = np.random.default_rng(M + N + pad)
    dst = torch.full((M, N + pad), 9.0, dtype=dt, device=G.DEV)
    check(orc, *operand(rng, M, 288), *operand(rng, N, 288), dtypes=(dt,), out=dst[:, :N])
    assert torch.all(dst[:, N:] == 9.0)


@pytest.mark.parametrize("N,pad", [(2565, 0), (2560, 8), (2562, 1)])
def test_gemm_unaligned_rows_of_many_tiles(orc, N, pad):
    """As above with more tiles than SMs."""
    rng = np.random.default_rng(N)
    qa, ea = operand(rng, 2050, 96)
    qb, eb = operand(rng, N, 96)
    for dt in (torch.float32, torch.bfloat16):
        dst = torch.full((2050, N + pad), 9.0, dtype=dt, device=G.DEV)
        check(orc, qa, ea, qb, eb, dtypes=(dt,), out=dst[:, :N])
        assert torch.all(dst[:, N:] == 9.0)


@pytest.mark.parametrize("M,N", [(1, 100), (16, 2048), (100, 2500), (129, 700), (257, 1290), (513, 384)])
@pytest.mark.parametrize("K", [512, 1056, 2560, 8224])
def test_gemm_split_k(orc, M, N, K):
    """Few tiles and long K: clusters of every size share a tile's K, with uneven parts."""
    rng = np.random.default_rng(M + K)
    check(orc, *operand(rng, M, K), *operand(rng, N, K))


@pytest.mark.parametrize("M", [4, 260])
def test_gemm_nan_scales_stay_in_their_rows(orc, M):
    rng = np.random.default_rng(4)
    qa, ea = operand(rng, M, 352)
    qb, eb = operand(rng, 300, 352)
    ea[2, 10] = 255                                          # the last block of an odd number of atoms
    eb[7, 0] = 255
    got = nv4.gemm_mxfp4(G.u8_dev(qa), nv4.mma_scales(G.u8_dev(ea)), G.u8_dev(qb), nv4.mma_scales(G.u8_dev(eb)),
                         dtype=torch.float32).cpu()
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[2], want[:, 7] = True, True
    assert torch.equal(nan, want)


def test_linear_mxfp4_run(orc):
    """Quantize and multiply as a user does; twice the same bits; streams; a replayed graph."""
    rng = np.random.default_rng(5)
    w = (0.02 * rng.standard_normal((520, 736))).astype(np.float32)
    qw, ew, _ = orc.mxfp4_quant(w)
    dq, ds = G.u8_dev(qw), nv4.mma_scales(G.u8_dev(ew))
    for M in (1, 7, 16, 33, 270):
        xs = [torch.from_numpy(rng.laplace(size=(M, 736)).astype(np.float32)).to(torch.bfloat16).to(G.DEV) for _ in range(3)]
        want = []
        for x in xs:
            q, e, _ = orc.mxfp4_quant(G.host(x))
            D, Dabs = orc.gemm_mxfp4(q, e, qw, ew)
            y = nv4.linear_mxfp4(x, dq, ds)
            tol = (736 / 64 + 4) * 2.0 ** -23 * Dabs + 2.0 ** -8 * np.abs(D)
            assert np.all(np.abs(y.double().cpu().numpy() - D) <= tol)
            assert torch.equal(y, nv4.linear_mxfp4(x, dq, ds))
            want.append(y)
        st = [torch.cuda.Stream() for _ in range(2)]
        got = [nv4.linear_mxfp4(x, dq, ds, stream=st[i % 2]) for i, x in enumerate(xs)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        xin, out = xs[0].clone(), torch.empty_like(want[0])
        q = torch.empty((M, 368), dtype=torch.uint8, device=G.DEV)
        sf = torch.empty(nv4.nv4_mxfp4_mma_scale_bytes(M, 736), dtype=torch.uint8, device=G.DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv4.nv4_mxfp4_quant_mma(xin, q, sf)
            nv4.nv4_gemm_mxfp4(q, sf, dq, ds, out)
        nb = nv4.nv4_linear_mxfp4_work_bytes(M, 736)
        work = torch.full((nb,), 0xFF, dtype=torch.uint8, device=G.DEV) if nb else None
        graph2, out2 = torch.cuda.CUDAGraph(), torch.empty_like(out)
        with torch.cuda.graph(graph2):
            nv4.nv4_linear_mxfp4(xin, dq, ds, out2, work)
        for x, y in zip(xs, want):
            xin.copy_(x)
            graph.replay()
            graph2.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, y) and torch.equal(out2, y)
    assert nv4.linear_mxfp4(xs[0][:0], dq, ds).shape == (0, 520)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 40, 32), (3, 130, 288), (15, 300, 2880), (16, 128, 4128), (5, 2000, 544), (2, 64, 16384)])
def test_linear_quantizes_within_the_product(orc, dt, M, N, K):
    """Up to 16 rows: the same codes and scales as the quantizer's (the product of its output is
    the same to the bit), rows inside a wider tensor whose padding holds NaN, zero blocks, blocks
    far apart in scale."""
    rng = np.random.default_rng(M * N)
    x = (rng.laplace(size=(M, K)) * np.exp2(rng.integers(-20, 20, (M, K // 32))).repeat(32, 1)).astype(np.float32)
    x[:, :32] = 0.0
    wide = torch.full((M, K + 8), float("nan"), dtype=dt, device=G.DEV)
    wide[:, :K] = torch.from_numpy(x).to(dt).to(G.DEV)
    xs = wide[:, :K]
    qw, ew = operand(rng, N, K)
    dq, ds = G.u8_dev(qw), nv4.mma_scales(G.u8_dev(ew))
    for out_dt in (torch.float32, torch.bfloat16):
        f = G.flags_dev()
        y = nv4.linear_mxfp4(xs, dq, ds, out_dt, f)
        q, sf = nv4.mxfp4_quant_mma(xs)
        assert torch.equal(y, nv4.gemm_mxfp4(q, sf, dq, ds, out_dt)) and f.item() == 0
    q, e, _ = orc.mxfp4_quant(np.ascontiguousarray(G.host(xs.contiguous())))
    D, Dabs = orc.gemm_mxfp4(q, e, qw, ew)
    got = nv4.linear_mxfp4(xs, dq, ds, torch.float32).double().cpu().numpy()
    assert np.all(np.abs(got - D) <= (K / 64 + 4) * 2.0 ** -23 * Dabs + 2.0 ** -24 * np.abs(D) + 1e-38)
    xs[M - 1, K - 1] = float("inf")                          # flagged, its row NaN, the others not
    f = G.flags_dev()
    y = nv4.linear_mxfp4(xs, dq, ds, torch.float32, f)
    assert f.item() == nv4.FLAG_NONFINITE and torch.isnan(y[M - 1]).all() and torch.isfinite(y[:M - 1]).all()


@pytest.mark.parametrize("M", [1, 16])
def test_linear_mxfp4_of_a_wide_layer(orc, M):
    """More than 2^25 weights: quantized within the product without a workspace, in front of it with
    one; the same bits either way, and the oracle's values."""
    rng = np.random.default_rng(8)
    N, K = 34000, 992
    qw, ew = operand(rng, N, K)
    dq, ds = G.u8_dev(qw), nv4.mma_scales(G.u8_dev(ew))
    x = torch.from_numpy(rng.laplace(size=(M, K)).astype(np.float32)).to(G.DEV)
    without = torch.empty((M, N), dtype=torch.float32, device=G.DEV)
    nv4.nv4_linear_mxfp4(x, dq, ds, without)
    y = nv4.linear_mxfp4(x, dq, ds, dtype=torch.float32)
    assert torch.equal(y, without)
    q, e, _ = orc.mxfp4_quant(x.cpu().numpy())
    D, Dabs = orc.gemm_mxfp4(q, e, qw, ew)
    tol = (K / 64 + 4) * 2.0 ** -23 * Dabs + 2.0 ** -24 * np.abs(D) + 1e-38
    assert np.all(np.abs(y.double().cpu().numpy() - D) <= tol)
    with pytest.raises(nv4.NV4Error):
        nv4.nv4_linear_mxfp4(x, dq, ds, without, torch.empty(1 << 17, dtype=torch.uint8, device=G.DEV)[8:])
