"""Refusals of the products on FP4 weights (no GPU: the checks come before any launch) and pins
of their oracle."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_numerics_b200 import binding
    from nvfp4_block_numerics_b200.build import build_library

    build_library()
    return binding.lib()


FAKE = 0x1000


def test_linear_w4a16_refusals(L):
    def f(x=FAKE, dt=0, T=4, K=64, ldx=64, q=FAKE, s=FAKE, s2=FAKE, N=8, odt=0, out=FAKE, ldd=8):
        return L.nv4_linear_w4a16(x, dt, T, K, ldx, q, s, s2, N, odt, out, ldd, None, None)

    assert f(dt=2) == 4 and f(odt=3) == 4                    # FP32 rows; unknown output type
    assert f(K=40, ldx=40) == 2 and f(ldx=56) == 2 and f(ldd=7) == 2 and f(T=-1) == 2 and f(K=0) == 2
    assert f(T=0) == 0 and f(N=0, ldd=0) == 0
    assert f(x=None) == 1 and f(q=None) == 1 and f(s=None) == 1 and f(s2=None) == 1 and f(out=None) == 1
    assert f(x=FAKE + 8) == 3 and f(ldx=68) == 3 and f(q=FAKE + 8) == 3 and f(out=FAKE + 4) == 3 and f(s=FAKE + 4) == 3
    assert f(K=65552, ldx=65552) == 6 and f(T=1 << 31) == 6


def test_linear_w4a16_oracle_is_the_dequantized_product(orc):
    """Against the oracle's own element decoders, entry by entry."""
    rng = np.random.default_rng(1)
    q = rng.integers(0, 256, (3, 16), dtype=np.uint8)
    sc = rng.integers(0, 0x7F, (3, 2), dtype=np.uint8)
    x = rng.standard_normal((2, 32))
    y, _ = orc.linear_w4a16(x, q, sc, 0.25)
    for t in range(2):
        for n in range(3):
            s = 0.0
            for k in range(32):
                c = (int(q[n, k // 2]) >> (4 * (k % 2))) & 15
                s += x[t, k] * orc.e2m1_value(c) * orc.e4m3_value(int(sc[n, k // 16])) * 0.25
            assert abs(s - y[t, n]) < 1e-9 * (1 + abs(s))
