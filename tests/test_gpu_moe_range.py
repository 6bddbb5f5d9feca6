"""The mixture-of-experts layer over its whole declared range, and against the bound of its FP32 sums.

u, per unit of the oracle's first-order term dev: the sums, at most (K/16 + 64) * 2^-23 for K = max(H, I) (16
products per MMA; beside them the chains', the warps' and up to 32 experts' additions and five multiplications); silu by
expf and a division, 2^-20; the two FP16 parts of a hidden value, 2^-22.  Then half a step of the output.
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


def check(orc, rng, T, E, H, I, ids, dt="bf16", out_dt="fp32"):
    gate, up, down = experts(rng, E, I, H), experts(rng, E, I, H), experts(rng, E, H, I)
    x = torch.from_numpy(rng.laplace(size=(T, H)).astype(np.float32)).to(DT[dt])
    w = rng.uniform(0, 1, ids.shape).astype(np.float32)
    dev3 = lambda m: (G.u8_dev(m[0]), G.u8_dev(m[1]), G.f32_dev(m[2]))  # noqa: E731
    f = G.flags_dev()
    dst = torch.full((T, H + 3), 5.0, dtype=DT[out_dt], device=G.DEV)
    work = torch.full((nv4.nv4_moe_work_bytes(*ids.shape, H, I),), 0xFF, dtype=torch.uint8, device=G.DEV)
    nv4.nv4_moe_experts(x.to(G.DEV), torch.from_numpy(ids.astype(np.int32)).to(G.DEV), G.f32_dev(w), dev3(gate), dev3(up),
                        dev3(down), dst[:, :H], work, f)
    y, dev = orc.moe_experts(x.double().numpy(), ids, w.astype(np.float64), gate, up, down)
    u = (max(H, I) / 16 + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22
    tol = u * dev + torch.finfo(DT[out_dt]).eps / 2 * np.abs(y) + 1e-38
    err = np.abs(dst[:, :H].double().cpu().numpy() - y)
    assert f.item() == 0 and torch.all(dst[:, H:] == 5.0)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


def random_ids(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)])


@pytest.mark.parametrize("T,E,k,H,I,dt,out", [
    (1, 64, 8, 1024, 512, "bf16", "fp32"), (3, 8, 4, 2880, 288, "bf16", "bf16"), (7, 16, 2, 1040, 304, "fp16", "fp32"),
    (24, 16, 4, 272, 576, "bf16", "fp32"), (64, 16, 8, 256, 128, "bf16", "fp32"), (48, 9, 3, 512, 528, "fp16", "bf16")])
def test_ordinary_sizes(orc, T, E, k, H, I, dt, out):
    rng = np.random.default_rng(T + E + I)
    check(orc, rng, T, E, H, I, random_ids(rng, T, E, k), dt, out)


@pytest.mark.parametrize("I", [16, 48])
def test_most_experts_pairs_and_sublists(orc, I):
    """64 tokens of 32 experts, 2048 pairs, of 512 experts: each chosen about four times; 192 of them nine times and 320
    once (704 groups of up to eight tokens, the most there can be); 32 of them by every token."""
    rng = np.random.default_rng(I)
    T, E, k, H = 64, 512, 32, 48
    check(orc, rng, T, E, H, I, random_ids(rng, T, E, k))
    copies = np.repeat(rng.permutation(E)[:192], 9)
    once = np.setdiff1d(np.arange(E), copies)
    pairs = np.concatenate([copies, rng.permutation(once)])
    ids = np.ascontiguousarray(pairs.reshape(32, 64).T)        # copies of one expert go to consecutive tokens
    assert all(np.unique(r).size == k for r in ids) and sum(-(-c // 8) for c in np.bincount(pairs)) == 704
    check(orc, rng, T, E, H, I, ids)
    check(orc, rng, T, E, H, I, np.tile(rng.permutation(E)[:32], (T, 1)))


@pytest.mark.parametrize("T,E,k,H,I", [(3, 2, 2, 32768, 16), (64, 2, 1, 32768, 32), (2, 2, 1, 64, 32768), (33, 3, 2, 32, 16384),
                                       (5, 3, 2, 6000, 272), (9, 2, 1, 9488, 64), (64, 4, 3, 4752, 48), (1, 1, 1, 20000, 16)])
def test_widest_layers(orc, T, E, k, H, I):
    """Up to 222 output rows per CTA, tiles that leave warps without one, sums of 32768."""
    rng = np.random.default_rng(H + I)
    check(orc, rng, T, E, H, I, random_ids(rng, T, E, k))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,H,k", [(64, 512, 64, 32), (1, 512, 4096, 32), (9, 3, 32768, 3), (2, 512, 32768, 1), (64, 32, 16, 32)])
def test_route_at_its_limits(orc, dt, T, E, H, k):
    rng = np.random.default_rng(T + E + H)
    x = torch.from_numpy(rng.laplace(size=(T, H)).astype(np.float32)).to(DT[dt])
    wr = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(DT[dt])
    for renorm in (True, False):
        ids, w = nv4.moe_route(x.to(G.DEV), wr.to(G.DEV), k, renorm)
        oi, ow = orc.moe_route(x.double().numpy(), wr.double().numpy(), k, renorm)
        assert np.array_equal(ids.cpu().numpy(), oi)
        assert np.all(np.abs(w.cpu().numpy() - ow) <= 2.0 ** -22 * ow + 1e-38)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_token_alone_and_among_others(orc, dt):
    """The weight-only layer gives a row the same values, to the bound of the sums, whatever batch it is in."""
    rng = np.random.default_rng(5)
    N, K = 200, 1024
    q, sc = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(0x20, 0x49, (N, K // 16), dtype=np.uint8)
    x = torch.from_numpy(rng.laplace(size=(300, K)).astype(np.float32)).to(DT[dt])
    x[7] *= 2.0 ** 9                                           # another scale than its neighbours'
    y, yabs = orc.linear_w4a16(x.double().numpy(), q, sc, 0.5)
    tol = (K / 16 + 40) * 2.0 ** -23 * yabs + 2.0 ** -24 * np.abs(y)
    for a, b in ((0, 1), (0, 5), (3, 16), (0, 17), (7, 8), (5, 70), (0, 300)):
        got = nv4.linear_w4a16(x[a:b].to(G.DEV), G.u8_dev(q), G.u8_dev(sc), torch.full((1,), 0.5, device=G.DEV), dtype=torch.float32)
        assert np.all(np.abs(got.double().cpu().numpy() - y[a:b]) <= tol[a:b])
