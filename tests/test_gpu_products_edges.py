"""Inputs at the ends of their types' ranges, and calls without any expert."""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(3, 70, 96), (40, 300, 1056), (300, 260, 608), (2100, 2600, 288)])
@pytest.mark.parametrize("ea,eb", [(3, 251), (251, 3), (0, 250), (130, 0), (64, 64), (190, 188)])
def test_gemm_mxfp4_scales_at_the_ends(orc, M, N, K, ea, eb):
    """Block scales near 2^-127 and 2^127: their product, not each by itself, has to fit.  The operands' blocks take
    three neighbouring codes.  Bound as for ordinary scales, (K/64 + 4) * 2^-23 of the sum of magnitudes and 2^-24 of the
    value; a partial sum below 2^-126 is off by at most 2^-149 per addition, K + 4 of them.  With codes 190 and 188 terms reach
    36 * 2^(192 + 190 - 254), beyond FP32: only sums of magnitudes below 2^127, of which no part can leave it, are bounded."""
    rng = np.random.default_rng(M + ea)
    qa, qb = (rng.integers(0, 256, (r, K // 2), dtype=np.uint8) for r in (M, N))
    sa, sb = (rng.integers(e, e + 3, (r, K // 32), dtype=np.uint8) for r, e in ((M, ea), (N, eb)))
    f = G.flags_dev()
    y = nv4.gemm_mxfp4(G.u8_dev(qa), nv4.mma_scales(G.u8_dev(sa)), G.u8_dev(qb), nv4.mma_scales(G.u8_dev(sb)),
                       dtype=torch.float32, d_flags=f).double().cpu().numpy()
    D, Dabs = orc.gemm_mxfp4(qa, sa, qb, sb)
    tol = (K / 64 + 4) * 2.0 ** -23 * Dabs + 2.0 ** -24 * np.abs(D) + (K + 4) * 2.0 ** -149
    fits = Dabs < 2.0 ** 127
    assert f.item() == 0 and np.all(np.abs(y - D)[fits] <= tol[fits]) and (ea == 190 or fits.all())


@pytest.mark.parametrize("T", [2, 12, 30, 150])
@pytest.mark.parametrize("dt,low", [(torch.float16, -24), (torch.bfloat16, -133)])
def test_linear_w4a16_subnormal_rows(orc, T, dt, low):
    """Rows of subnormal values alone, and beside ordinary ones: none is flushed."""
    rng = np.random.default_rng(T)
    N, K = 90, 528
    q, sc = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(0x30, 0x49, (N, K // 16), dtype=np.uint8)
    x = rng.integers(-20, 21, (T, K)).astype(np.float64) * 2.0 ** low
    x[1] = rng.standard_normal(K)
    dx = torch.from_numpy(x).to(dt)
    s2 = 2.0 ** 20
    y, yabs = orc.linear_w4a16(dx.double().numpy(), q, sc, s2)
    got = nv4.linear_w4a16(dx.to(G.DEV), G.u8_dev(q), G.u8_dev(sc), torch.full((1,), s2, device=G.DEV), dtype=torch.float32)
    # a partial sum below 2^-126 (before s2) is off by at most 2^-149 per addition
    tol = (K / 16 + 40) * 2.0 ** -23 * yabs + 2.0 ** -24 * np.abs(y) + (K + 40) * 2.0 ** -149 * s2
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= tol)


@pytest.mark.parametrize("T,k", [(1, 1), (5, 3), (64, 8)])
def test_moe_experts_without_any_expert(T, k):
    """Every id is padding: zeros, whatever the tokens and the workspace hold."""
    E, H, I = 8, 272, 48
    w = lambda r, c: (torch.full((E, r, c // 2), 0x77, dtype=torch.uint8, device=G.DEV),  # noqa: E731
                      torch.full((E, r, c // 16), 0x38, dtype=torch.uint8, device=G.DEV), torch.ones(E, device=G.DEV))
    x = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=G.DEV)
    ids[0, 0] = E
    out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=G.DEV)
    work = torch.full((nv4.nv4_moe_work_bytes(T, k, H, I),), 0xFF, dtype=torch.uint8, device=G.DEV)
    f = G.flags_dev()
    nv4.nv4_moe_experts(x, ids, torch.full((T, k), float("nan"), device=G.DEV), w(I, H), w(I, H), w(H, I), out, work, f)
    assert torch.all(out == 0) and f.item() == 0
