"""NaN and Inf through the products on FP4 weights: which outputs they reach, and the flag."""
import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def weights(rng, N, K):
    """Codes without zeros, so that an Inf stays one; scales 2^-3 to 2^0."""
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8) | 0x11
    return G.u8_dev(q), G.u8_dev(rng.integers(0x20, 0x39, (N, K // 16), dtype=np.uint8))


# few rows alone and in clusters that split K, the tensor-memory kernel split and not, more tiles than SMs
SIZES = [(1, 100, 128), (3, 300, 8192), (16, 200, 4096), (20, 200, 4096), (40, 150, 64), (200, 1000, 528), (300, 9000, 80)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_linear_w4a16_flags_what_it_propagates(T, N, K, dt, out):
    rng = np.random.default_rng(T + N)
    q, sc = weights(rng, N, K)
    s2 = torch.full((1,), 0.01, device=G.DEV)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(DT[dt]).to(G.DEV)

    def run(x, sc=sc, s2=s2):
        f = G.flags_dev()
        y = nv4.linear_w4a16(x, q, sc, s2, dtype=out, d_flags=f)
        nv4.linear_w4a16(x, q, sc, s2, dtype=out)             # without a flag word
        return torch.isfinite(y), f.item()

    ok, f = run(x)
    assert ok.all() and f == 0
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = x.clone()
        bad[T - 1, K - 3] = value                             # the whole row, no other
        ok, f = run(bad)
        assert not ok[T - 1].any() and ok[:T - 1].all() and f == nv4.FLAG_NONFINITE
    bad = sc.clone()
    bad[N - 1, K // 16 - 1] = 0x7F                            # a NaN scale: the whole column, no other
    ok, f = run(x, bad)
    assert not ok[:, N - 1].any() and ok[:, :N - 1].all() and f == nv4.FLAG_NONFINITE
    ok, f = run(x, sc, torch.full((1,), float("inf"), device=G.DEV))
    assert not ok.any() and f == nv4.FLAG_NONFINITE


@pytest.mark.parametrize("T", [2, 30])
def test_an_output_beyond_its_type_is_not_flagged(T):
    """FP16 has no value for 10^6: the output is Inf, but nothing that was read or summed."""
    q = torch.full((20, 32), 0x22, dtype=torch.uint8, device=G.DEV)           # ones
    sc = torch.full((20, 4), 0x38, dtype=torch.uint8, device=G.DEV)
    f = G.flags_dev()
    y = nv4.linear_w4a16(torch.full((T, 64), 1000.0, dtype=torch.float16, device=G.DEV), q, sc,
                         torch.full((1,), 16.0, device=G.DEV), d_flags=f)
    assert torch.isinf(y).all() and f.item() == 0
