"""Router logits of BF16 values whose products leave FP32's range, and their order."""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 9])
@pytest.mark.parametrize("ex,ew", [(70, 70), (-100, -60), (-75, -70), (120, -120), (0, 0)])
def test_products_outside_fp32(orc, T, ex, ew):
    """Products near 2^140, 2^-160 and 2^-145 (subnormal in FP32): the order and the weights of the exact logits.
    The logits are sums of 32 products of whole numbers below 2^8, times one power of two: exact in FP64."""
    rng = np.random.default_rng(T)
    E, H, k = 24, 64, 6
    x, w = rng.integers(-127, 128, (T, H)).astype(np.float64), rng.integers(-127, 128, (E, H)).astype(np.float64)
    x[:, 32:] = 0.0
    x, w = x * 2.0 ** (ex - 7), w * 2.0 ** (ew - 7)
    w[5] = w[3]                                                # an exact tie
    dx, dw = (torch.from_numpy(a).to(torch.bfloat16).to(G.DEV) for a in (x, w))
    assert np.array_equal(dx.double().cpu().numpy(), x) and np.array_equal(dw.double().cpu().numpy(), w)
    f = G.flags_dev()
    ids, weights = nv4.moe_route(dx, dw, k, d_flags=f)
    oi, ow = orc.moe_route(x, w, k)
    assert f.item() == 0 and np.array_equal(ids.cpu().numpy(), oi)
    assert np.all(np.abs(weights.cpu().numpy() - ow) <= 2.0 ** -22 * ow + 1e-38)
