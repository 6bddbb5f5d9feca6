"""The weight-only linear layer at sizes on both sides of the choice between token tiles of 128 and 256.

Tolerance as for its other sizes: FP32 sums of K exact products, 16 per MMA and at most 40 additions beside
them, (K/16 + 40) * 2^-23 of the sum of magnitudes; half a step of the output.
"""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("T,N,K,dt,out", [
    (300, 9500, 272, "bf16", "bf16"), (800, 2885, 528, "fp16", "fp32"), (1000, 2880, 1040, "bf16", "fp16"),
    (600, 4096, 1024, "fp16", "bf16"), (600, 4096, 64, "bf16", "fp32"), (129, 19000, 512, "bf16", "bf16"),
    (257, 9473, 1040, "bf16", "bf16")])
def test_linear_either_width(orc, T, N, K, dt, out):
    rng = np.random.default_rng(T + N)
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    sc = rng.integers(0x20, 0x49, (N, K // 16), dtype=np.uint8)
    x = torch.from_numpy(rng.laplace(size=(T, K)).astype(np.float32)).to(DT[dt])
    got = nv4.linear_w4a16(x.to(G.DEV), G.u8_dev(q), G.u8_dev(sc), torch.full((1,), 0.0031, device=G.DEV), dtype=DT[out])
    y, yabs = orc.linear_w4a16(x.double().numpy(), q, sc, float(np.float32(0.0031)))
    tol = (K / 16 + 40) * 2.0 ** -23 * yabs + torch.finfo(DT[out]).eps / 2 * np.abs(y) + (2.0 ** -25 if out == "fp16" else 1e-38)
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= tol)
