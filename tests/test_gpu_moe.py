"""GPU parity of the mixture-of-experts layer on NVFP4 expert weights.

Routing: ids equal the oracle's (the logits are FP64 on both sides; the inputs are random, so no
two logits agree to 1e-13, apart from planted exact ties); weights to 2^-22 (one rounding to
FP32).  Experts: the oracle's FP64 result with its first-order error bound dev per relative error
u.  u covers: a sum of K products in the MMA, at most (K/16 + 40) * 2^-23 for K = max(H, I); silu
in FP32 with expf and a division, 2^-20; the hidden value's FP16 rounding 2^-11 (half a step of 11
bits, relative to the value; values 2^-29 below their row's largest add at most 2^-40 of it,
inside the same bound by its K = I terms).  The hidden rounding enters dev with |h|, the others
with the full first-order term, so u = 2^-11 * (|D||h| part) is bounded by u * dev as a whole.
"""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def experts(rng, E, rows, cols):
    return (rng.integers(0, 256, (E, rows, cols // 2), dtype=np.uint8),
            rng.integers(0x20, 0x48, (E, rows, cols // 16), dtype=np.uint8),
            (rng.uniform(0.5, 1.5, E) * 2e-3 / np.sqrt(cols)).astype(np.float32))


def layer(rng, E, H, I):
    return experts(rng, E, I, H), experts(rng, E, I, H), experts(rng, E, H, I)


def dev3(w):
    return G.u8_dev(w[0]), G.u8_dev(w[1]), G.f32_dev(w[2])


def tokens(rng, T, H, dt="bf16"):
    x = rng.laplace(size=(T, H)).astype(np.float32)
    x[:, rng.integers(0, H, max(1, H // 200))] *= 50.0
    return torch.from_numpy(x).to(DT[dt]).to(G.DEV)


def check(orc, x, ids, weights, gate, up, down, out_dt="bf16", out=None):
    f = G.flags_dev()
    di, dw = torch.from_numpy(ids.astype(np.int32)).to(G.DEV), G.f32_dev(weights)
    g, u, d = dev3(gate), dev3(up), dev3(down)
    if out is None:
        out = nv4.moe_experts(x, di, dw, g, u, d, dtype=DT[out_dt], d_flags=f)
    else:
        work = torch.full((nv4.nv4_moe_work_bytes(*ids.shape, x.shape[1], gate[0].shape[1]),), 0xFF, dtype=torch.uint8, device=G.DEV)
        nv4.nv4_moe_experts(x, di, dw, g, u, d, out, work, f)
    torch.cuda.synchronize()
    assert f.item() == 0
    y, bound = orc.moe_experts(x.double().cpu().numpy(), ids, weights.astype(np.float64), gate, up, down)
    K = max(x.shape[1], gate[0].shape[1])
    u_rel = (K / 16 + 40) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -11
    tol = u_rel * bound + torch.finfo(DT[out_dt]).eps / 2 * np.abs(y) + (2.0 ** -25 if out_dt == "fp16" else 1e-38)
    err = np.abs(out.double().cpu().numpy() - y)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())
    return out


def random_ids(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,H,k", [(1, 4, 16, 1), (1, 64, 4096, 8), (3, 32, 2880, 4), (5, 7, 144, 7), (9, 512, 256, 32),
                                     (48, 64, 1040, 8), (64, 33, 512, 3)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(orc, dt, T, E, H, k, renorm):
    rng = np.random.default_rng(T * E + H)
    x = tokens(rng, T, H, dt)
    wr = torch.from_numpy((rng.standard_normal((E, H)) / (6 * np.sqrt(H))).astype(np.float32)).to(DT[dt]).to(G.DEV)
    ids, w = nv4.moe_route(x, wr, k, renorm)
    oi, ow = orc.moe_route(x.double().cpu().numpy(), wr.double().cpu().numpy(), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), oi)
    assert np.all(np.abs(w.cpu().numpy() - ow) <= 2.0 ** -22 * ow + 1e-38)


def test_route_ties_and_nonfinite():
    """Equal logits go to the lower index; a NaN logit ranks last and sets the flag."""
    H, E = 64, 40
    x = torch.zeros((3, H), dtype=torch.bfloat16, device=G.DEV)
    x[0, 0] = 1.0
    x[2, 1] = 1.0
    wr = torch.zeros((E, H), dtype=torch.bfloat16, device=G.DEV)
    wr[[5, 37, 12], 0] = 2.0                                  # token 0: three equal logits
    f = G.flags_dev()
    ids, w = nv4.moe_route(x, wr, 5, d_flags=f)
    assert f.item() == 0
    assert ids[0].tolist() == [5, 12, 37, 0, 1] and ids[1].tolist() == [0, 1, 2, 3, 4]
    assert torch.allclose(w[1].cpu(), torch.full((5,), 0.2))
    wr[0, 1] = float("nan")
    ids, _ = nv4.moe_route(x, wr[:32], 32, d_flags=f)         # every expert of 32 (top_k is 32 at most)
    assert f.item() == nv4.FLAG_NONFINITE and ids[2, -1].item() == 0 and sorted(ids[2].tolist()) == list(range(32))


@pytest.mark.parametrize("T,E,k,H,I,dt,out", [
    (1, 8, 2, 256, 256, "bf16", "bf16"), (1, 1, 1, 16, 16, "bf16", "fp32"), (2, 4, 4, 48, 80, "fp16", "fp32"),
    (1, 64, 8, 1024, 512, "bf16", "fp32"), (3, 32, 4, 2880, 288, "bf16", "fp16"), (7, 16, 2, 1040, 304, "bf16", "bf16"),
    (8, 5, 3, 512, 1536, "fp16", "bf16"), (20, 16, 4, 272, 64, "bf16", "fp32"), (64, 40, 8, 256, 128, "bf16", "fp32"),
    (64, 12, 12, 64, 64, "fp16", "fp32"), (5, 3, 2, 4096, 64, "bf16", "fp32"), (2, 3, 2, 64, 4096, "bf16", "fp32")])
def test_experts(orc, T, E, k, H, I, dt, out):
    rng = np.random.default_rng(T + E + H)
    check(orc, tokens(rng, T, H, dt), random_ids(rng, T, E, k), rng.uniform(0, 1, (T, k)).astype(np.float32),
          *layer(rng, E, H, I), out_dt=out)


@pytest.mark.parametrize("T", [9, 30, 64])
def test_experts_one_expert_takes_all(orc, T):
    """Every token on the same two experts: more tokens than one pass multiplies."""
    rng = np.random.default_rng(T)
    ids = np.tile(np.array([[3, 1]], np.int32), (T, 1))
    check(orc, tokens(rng, T, 528), ids, rng.uniform(0, 1, (T, 2)).astype(np.float32), *layer(rng, 5, 528, 272), out_dt="fp32")


def test_experts_padding_duplicates_and_strides(orc):
    """Ids outside the range add nothing, a token without experts is 0, an id named twice counts
    with both weights; rows inside wider tensors, the workspace full of NaN."""
    rng = np.random.default_rng(3)
    T, E, k, H, I = 6, 9, 4, 320, 144
    ids = random_ids(rng, T, E, k)
    ids[1] = [-1, 4, 1 << 30, 4]
    ids[2] = -1
    ids[3] = [2, 2, 2, 2]
    ids[5, 0] = E
    wide = torch.full((T, H + 8), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    wide[:, :H] = tokens(rng, T, H)
    dst = torch.full((T, H + 5), 3.0, dtype=torch.float32, device=G.DEV)
    out = check(orc, wide[:, :H], ids, rng.uniform(0, 1, (T, k)).astype(np.float32), *layer(rng, E, H, I), out_dt="fp32",
                out=dst[:, :H])
    assert torch.all(out[2] == 0) and torch.all(dst[:, H:] == 3.0)


def test_experts_wide_rows_and_large_hidden(orc):
    """A token whose values span more binades than FP16 holds next to ordinary ones, and hidden
    values far above FP16's range (their rows are scaled)."""
    rng = np.random.default_rng(4)
    T, E, k, H, I = 4, 4, 2, 256, 128
    gate, up, down = layer(rng, E, H, I)
    gate[0][:, :, 0] &= 0xF0                                  # element 0 meets zero codes
    up[0][:, :, 0] &= 0xF0
    x = tokens(rng, T, H)
    x[1, 0] = 2.0 ** 50
    x[2] *= 2.0 ** 12
    check(orc, x, random_ids(rng, T, E, k), rng.uniform(0, 1, (T, k)).astype(np.float32), gate, up, down, out_dt="fp32")


def test_layer_run(orc):
    """Quantized weights end to end: RTN-quantized experts, router and experts in one call, equal
    to its two parts; twice the same bits; a captured call replayed on other tokens."""
    rng = np.random.default_rng(8)
    T, E, k, H, I = 4, 16, 4, 512, 256

    def quantized(rows, cols):
        parts = [orc.rtn_quant((0.02 * rng.standard_normal((rows, cols))).astype(np.float32), 0.1)[:3] for _ in range(E)]
        return tuple(np.stack([np.asarray(q[i]) for q in parts]) for i in range(2)) + (
            np.array([q[2] for q in parts], np.float32),)

    gate, up, down = quantized(I, H), quantized(I, H), quantized(H, I)
    g, u, d = dev3(gate), dev3(up), dev3(down)
    wr = torch.from_numpy((rng.standard_normal((E, H)) / (6 * np.sqrt(H))).astype(np.float32)).to(torch.bfloat16).to(G.DEV)
    xs = [tokens(rng, T, H) for _ in range(3)]
    want = []
    for x in xs:
        out, ids, w = nv4.moe_layer(x, wr, g, u, d, k)
        oi, _ = orc.moe_route(x.double().cpu().numpy(), wr.double().cpu().numpy(), k)
        assert np.array_equal(ids.cpu().numpy(), oi)
        assert torch.equal(out, nv4.moe_experts(x, ids, w, g, u, d))
        check(orc, x, ids.cpu().numpy(), w.cpu().numpy(), gate, up, down)
        want.append(out)
    xin, out = xs[0].clone(), torch.empty_like(want[0])
    ids = torch.empty((T, k), dtype=torch.int32, device=G.DEV)
    w = torch.empty((T, k), device=G.DEV)
    work = torch.empty(nv4.nv4_moe_work_bytes(T, k, H, I), dtype=torch.uint8, device=G.DEV)
    nv4.nv4_moe_layer(xin, wr, g, u, d, ids, w, out, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv4.nv4_moe_layer(xin, wr, g, u, d, ids, w, out, work)
    for x, y in zip(xs, want):
        xin.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [nv4.moe_layer(x, wr, g, u, d, k, stream=st[i % 2])[0] for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert nv4.moe_layer(xs[0][:0], wr, g, u, d, k)[0].shape == (0, H)
