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


def test_moe_refusals(L):
    import ctypes as C

    from nvfp4_block_numerics_b200 import binding as b

    def route(x=FAKE, dt=0, T=2, H=64, ldx=64, wr=FAKE, E=8, k=2, ids=FAKE, w=FAKE):
        return L.nv4_moe_route(x, dt, T, H, ldx, wr, E, k, 1, ids, w, None, None)

    assert route(dt=2) == 4
    assert route(H=40, ldx=40) == 2 and route(ldx=48) == 2 and route(k=9) == 2 and route(k=0) == 2 and route(E=0) == 2
    assert route(T=65) == 6 and route(E=513) == 6 and route(E=64, k=33) == 6 and route(H=32784, ldx=32784) == 6
    assert route(x=None) == 1 and route(wr=None) == 1 and route(ids=None) == 1 and route(w=None) == 1
    assert route(x=FAKE + 2) == 3 and route(ldx=68) == 3 and route(wr=FAKE + 8) == 3 and route(ids=FAKE + 2) == 3
    assert route(T=0) == 0

    ok = b.ExpertWeights(FAKE, FAKE, FAKE)

    def experts(x=FAKE, dt=0, T=2, H=64, ldx=64, ids=FAKE, w=FAKE, k=2, E=8, I=32, g=ok, u=ok, d=ok, odt=0, out=FAKE,
                ldd=64, work=FAKE, wb=1 << 20):
        P = lambda v: None if v is None else C.byref(v)  # noqa: E731
        return L.nv4_moe_experts(x, dt, T, H, ldx, ids, w, k, E, I, P(g), P(u), P(d), odt, out, ldd, work, wb, None, None)

    assert experts(dt=2) == 4 and experts(odt=5) == 4
    assert experts(I=24) == 2 and experts(I=0) == 2 and experts(ldd=63) == 2 and experts(k=9) == 2
    assert experts(I=32784) == 6 and experts(T=65) == 6 and experts(wb=L.nv4_moe_work_bytes(2, 2, 64, 32) - 1) == 6
    assert experts(g=None) == 1 and experts(u=b.ExpertWeights(None, FAKE, FAKE)) == 1 and experts(work=None) == 1
    assert experts(d=b.ExpertWeights(FAKE, FAKE + 4, FAKE)) == 3 and experts(work=FAKE + 8) == 3 and experts(out=FAKE + 2) == 3
    assert experts(T=0) == 0
    assert L.nv4_moe_work_bytes(3, 4, 64, 32) >= 3 * 4 * 32 * 6 + 3 * 64 * 2 and L.nv4_moe_work_bytes(0, 4, 64, 32) == 0
    # the whole layer refuses before it launches anything
    assert L.nv4_moe_layer(FAKE, 0, 2, 64, 64, FAKE, 8, 2, 1, 24, C.byref(ok), C.byref(ok), C.byref(ok), FAKE, FAKE, 0, FAKE,
                           64, FAKE, 1 << 20, None, None) == 2


def test_moe_oracle_small(orc):
    """One expert of weight 1 is the plain gated MLP; two experts add with their weights; an id
    outside the range adds nothing."""
    rng = np.random.default_rng(2)
    mk = lambda E, r, c: (rng.integers(0, 256, (E, r, c // 2), dtype=np.uint8),  # noqa: E731
                          rng.integers(0x30, 0x40, (E, r, c // 16), dtype=np.uint8), np.full(E, 0.01, np.float32))
    gate, up, down = mk(3, 32, 16), mk(3, 32, 16), mk(3, 16, 32)
    x = rng.standard_normal((1, 16))
    one = lambda e: orc.moe_experts(x, np.array([[e]]), np.ones((1, 1)), gate, up, down)[0]  # noqa: E731
    W = [orc._dequant_exact(w[0][1], w[1][1], float(w[2][1])) for w in (gate, up, down)]
    g, u = W[0] @ x[0], W[1] @ x[0]
    assert np.allclose(one(1)[0], W[2] @ (g / (1 + np.exp(-g)) * u), rtol=1e-12)
    two, _ = orc.moe_experts(x, np.array([[2, 0]]), np.array([[0.25, 0.5]]), gate, up, down)
    assert np.allclose(two, 0.25 * one(2) + 0.5 * one(0), rtol=1e-12)
    assert np.all(one(-1) == 0) and np.all(one(3) == 0)
    ids, w = orc.moe_route(np.array([[1.0, 0.0]]), np.array([[0.0, 1.0], [2.0, 0.0], [2.0, 0.0]]), 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, 0.5)


def test_mxfp4_product_refusals(L):
    def quant(x=FAKE, dt=0, rows=4, cols=64, ld=64, q=FAKE, s=FAKE):
        return L.nv4_mxfp4_quant_mma(x, dt, rows, cols, ld, q, s, None, None)

    assert quant(dt=1) == 4 and quant(cols=48, ld=48) == 2 and quant(ld=32) == 2
    assert quant(x=None) == 1 and quant(s=None) == 1 and quant(s=FAKE + 8) == 3 and quant(ld=68) == 3
    assert quant(rows=0) == 0 and quant(rows=1 << 30, cols=1 << 12, ld=1 << 12) == 6

    def gemm(qa=FAKE, sa=FAKE, qb=FAKE, sb=FAKE, M=4, N=8, K=64, dt=0, out=FAKE, ldd=8):
        return L.nv4_gemm_mxfp4(qa, sa, qb, sb, M, N, K, dt, out, ldd, None, None)

    assert gemm(dt=1) == 4 and gemm(K=48) == 2 and gemm(ldd=7) == 2 and gemm(K=0) == 2 and gemm(M=-1) == 2
    assert gemm(qa=None) == 1 and gemm(sb=None) == 1 and gemm(out=None) == 1
    assert gemm(qb=FAKE + 8) == 3 and gemm(sa=FAKE + 4) == 3 and gemm(out=FAKE + 8) == 3
    assert gemm(M=0) == 0 and gemm(N=0, ldd=0) == 0 and gemm(M=1 << 31) == 6

    def linear(x=FAKE, dt=0, M=20, K=64, ldx=64, qw=FAKE, sw=FAKE, N=8, odt=0, out=FAKE, ldd=8, work=FAKE, wb=1 << 20):
        return L.nv4_linear_mxfp4(x, dt, M, K, ldx, qw, sw, N, odt, out, ldd, work, wb, None, None)

    for M in (4, 20):                                        # within the product, and with a workspace
        assert linear(M=M, dt=1) == 4 and linear(M=M, odt=1) == 4 and linear(M=M, K=48, ldx=48) == 2 and linear(M=M, ldx=32) == 2
        assert linear(M=M, x=None) == 1 and linear(M=M, qw=None) == 1 and linear(M=M, out=FAKE + 8) == 3
        assert linear(M=M, x=FAKE + 8) == 3 and linear(M=M, ldx=68) == 3 and linear(M=M, ldd=7) == 2 and linear(M=M, K=0) == 2
    assert linear(work=None) == 1 and linear(work=FAKE + 8) == 3 and linear(M=0) == 0
    assert linear(wb=L.nv4_linear_mxfp4_work_bytes(20, 64) - 1) == 6
    assert L.nv4_linear_mxfp4_work_bytes(20, 64) == 512 + 20 * 32 and L.nv4_linear_mxfp4_work_bytes(16, 64) == 0
    assert L.nv4_mxfp4_mma_scale_bytes(200, 288) == 256 * 12 and L.nv4_mxfp4_mma_scale_bytes(1, 32) == 512
    assert L.nv4_mxfp4_mma_scale_bytes(4, 48) == 0 and L.nv4_mxfp4_mma_scale_bytes(0, 32) == 0


def test_mxfp4_product_oracle_small(orc):
    """Against the oracle's dequantizer, which is pinned to the format."""
    rng = np.random.default_rng(3)
    qa, qb = rng.integers(0, 256, (3, 32), dtype=np.uint8), rng.integers(0, 256, (5, 32), dtype=np.uint8)
    ea, eb = rng.integers(100, 150, (3, 2), dtype=np.uint8), rng.integers(100, 150, (5, 2), dtype=np.uint8)
    D, Dabs = orc.gemm_mxfp4(qa, ea, qb, eb)
    A, B = (orc.mxfp4_dequant(q, e, "fp32").astype(np.float64) for q, e in ((qa, ea), (qb, eb)))
    assert np.allclose(D, A @ B.T, rtol=1e-12) and np.allclose(Dabs, np.abs(A) @ np.abs(B).T, rtol=1e-12)
