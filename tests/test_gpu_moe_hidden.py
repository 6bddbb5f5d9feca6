"""The hidden values between the products of the mixture-of-experts layer.

All inputs are whole numbers times powers of two, chosen so that every step is exact in FP32: a gate
sum g from 20 to 240 makes silu(g) = g, as 1 + exp(-g) is 1 in FP32; with an up sum u of at most 480, both
multiples of 1/2, h = g u is a whole number of quarters below 2^19; a down row adds three of them times at most
4: below 2^24 eighths.  What comes out is then equal to the whole-number result, bit for bit, if the hidden
values keep 19 bits.
"""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def whole_number_layer(rng, E, H, I):
    """Codes and values (half units) of gate (positive), up (of both signs) and down (three entries a row);
    all block scales are 1."""
    gate = rng.integers(1, 4, (E, I, H))                       # 0.5, 1, 1.5
    up = rng.integers(0, 6, (E, I, H)) | (rng.integers(0, 2, (E, I, H)) << 3)
    down = np.zeros((E, H, I), np.int64)
    for e in range(E):
        for r in range(H):
            at = rng.permutation(I)[:3]
            down[e, r, at] = rng.integers(1, 7, at.size) | (rng.integers(0, 2, at.size) << 3)
    val = lambda c: np.where(c >= 8, -1, 1) * (2 * E2M1[c & 7]).astype(np.int64)  # noqa: E731
    ones = lambda r, c: np.full((E, r, c // 16), 0x38, np.uint8)  # noqa: E731
    return ((pack(gate), ones(I, H)), (pack(up), ones(I, H)), (pack(down), ones(H, I))), (val(gate), val(up), val(down))


def tokens(rng, T, H):
    """40 values of 1, 2 or 4 (one of them per token) among zeros: 40 to 480 half units in the gate, up to 960 in up."""
    x = np.zeros((T, H), np.int64)
    for t in range(T):
        x[t, rng.permutation(H)[:40]] = 1 << rng.integers(0, 3)
    return x


def dev(w, s2):
    return G.u8_dev(w[0]), G.u8_dev(w[1]), torch.full((w[0].shape[0],), s2, dtype=torch.float32, device=G.DEV)


def expected(x, ids, weights, vals):
    """In units of 1/8: half units of the down codes times quarter units of h; weights are whole numbers."""
    gate, up, down = vals
    out = np.zeros((x.shape[0], down.shape[1]), np.int64)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            h = (gate[e] @ x[t]) * (up[e] @ x[t])
            assert np.abs(h).max() < 1 << 19 and (gate[e] @ x[t]).min() >= 40
            out[t] += weights[t, j] * (down[e] @ h)
    return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,H,I", [(1, 2, 64, 32), (1, 2, 400, 272), (4, 1, 80, 560), (5, 1, 96, 48), (8, 1, 64, 1040),
                                     (9, 1, 64, 304), (30, 3, 160, 528), (64, 2, 2400, 80)])
def test_hidden_values_keep_their_bits(dt, T, E, H, I):
    """Up to 4, up to 8 and more tokens of an expert, one expert a token."""
    rng = np.random.default_rng(T + H)
    codes, vals = whole_number_layer(rng, E, H, I)
    x = tokens(rng, T, H)
    ids = rng.integers(0, E, (T, 1))
    w = 1 << rng.integers(0, 2, (T, 1))
    g, u, d = (dev(c, 1.0) for c in codes)
    y = nv4.moe_experts(torch.from_numpy(x.astype(np.float32)).to(dt).to(G.DEV), torch.from_numpy(ids.astype(np.int32)).to(G.DEV),
                        G.f32_dev(w.astype(np.float32)), g, u, d, dtype=torch.float32)
    want = expected(x, ids, w, vals) / 8.0
    assert np.array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("T", [2, 7])
@pytest.mark.parametrize("s_up,s_down", [(-80, -55), (80, 40), (-60, 30), (0, 0), (110, -60)])
def test_scales_far_from_one(T, s_up, s_down):
    """Hidden values and scale_2 of extreme magnitudes whose product is an ordinary number: the sum is exact, the
    routing weight times scale_2 is exact (0.7 times a power of two), so one rounding is left, 2^-24, or 2^-150 where the
    result is subnormal; from 2^128 on the result is an Inf.  (I is one chunk of 256: one warp forms the whole sum.)"""
    rng = np.random.default_rng(T)
    E, H, I = 2, 64, 240
    codes, vals = whole_number_layer(rng, E, H, I)
    x = tokens(rng, T, H)
    ids = rng.integers(0, E, (T, 1))
    w = np.float32(0.7)
    g, u, d = dev(codes[0], 1.0), dev(codes[1], 2.0 ** s_up), dev(codes[2], 2.0 ** s_down)
    y = nv4.moe_experts(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(G.DEV),
                        torch.from_numpy(ids.astype(np.int32)).to(G.DEV), torch.full((T, 1), 0.7, device=G.DEV), g, u, d,
                        dtype=torch.float32).double().cpu().numpy()
    want = expected(x, ids, np.ones((T, 1), np.int64), vals) / 8.0 * float(w) * 2.0 ** (s_up + s_down)
    big = np.abs(want) >= 2.0 ** 128
    assert np.array_equal(y[big], np.copysign(np.inf, want[big]))
    y, want = y[~big], want[~big]
    assert np.all(np.abs(y - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -150)
