"""The products on FP4 weights as a program runs them: on several streams at once, captured before
any other call, with nothing to do."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def layers(seed):
    """Calls of every kernel of these products, as functions of (index of an input, stream)."""
    gen = torch.Generator(device=G.DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=G.DEV)
    code = lambda *s: torch.randint(0, 256, s, generator=gen, dtype=torch.uint8, device=G.DEV)
    scale = lambda *s: torch.randint(0x20, 0x40, s, generator=gen, dtype=torch.uint8, device=G.DEV)
    one = torch.full((1,), 0.01, device=G.DEV)
    calls = []
    for T, N, K in ((3, 700, 1040), (40, 1100, 2080), (500, 2500, 512)):
        xs, q, sc = [rnd(T, K).to(torch.bfloat16) for _ in range(2)], code(N, K // 2), scale(N, K // 16)
        calls.append(lambda i, s, xs=xs, q=q, sc=sc: nv4.linear_w4a16(xs[i], q, sc, one, stream=s))
    for M, N, K in ((5, 1000, 2080), (90, 1300, 4160), (2100, 2600, 288)):
        xs, q = [rnd(M, K).to(torch.bfloat16) for _ in range(2)], code(N, K // 2)
        sf = nv4.mma_scales(torch.randint(110, 130, (N, K // 32), generator=gen, dtype=torch.uint8, device=G.DEV))
        calls.append(lambda i, s, xs=xs, q=q, sf=sf: nv4.linear_mxfp4(xs[i], q, sf, stream=s))
    E, H, I, k, T = 8, 512, 160, 2, 6
    xs, wr, s2 = [rnd(T, H).to(torch.bfloat16) for _ in range(2)], rnd(E, H).to(torch.bfloat16), torch.full((E,), 0.01, device=G.DEV)
    g, u, d = ((code(E, I, H // 2), scale(E, I, H // 16), s2), (code(E, I, H // 2), scale(E, I, H // 16), s2),
               (code(E, H, I // 2), scale(E, H, I // 16), s2))
    calls.append(lambda i, s: nv4.moe_layer(xs[i], wr, g, u, d, k, stream=s)[0])
    return calls


def test_streams_at_once():
    """Every product on four streams, in another order on each: the bits of the calls by themselves."""
    calls = layers(1)
    want = [[f(i, None) for i in range(2)] for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for turn in range(6):
        for j, s in enumerate(streams):
            for n in range(len(calls)):
                c, i = (n * (2 * j + 1) + turn + j) % len(calls), (turn + j) & 1
                got.append((c, i, calls[c](i, s)))
    torch.cuda.synchronize()
    for c, i, y in got:
        assert torch.equal(y, want[c][i]), c


def test_captured_before_any_other_call():
    """A process whose first call of each product is captured, then replayed on other inputs."""
    code = (
        "import sys, torch\n"
        "sys.path[:0] = [%r, %r]\n"
        "import test_gpu_products_together as t\n"
        "calls = t.layers(2)\n"
        "for f in calls:\n"
        "    g = torch.cuda.CUDAGraph()\n"
        "    with torch.cuda.graph(g):\n"
        "        y = f(0, None)\n"
        "    g.replay(); torch.cuda.synchronize()\n"
        "    assert torch.equal(y, f(0, None))\n"
        "print('captured', len(calls))\n" % (ROOT, os.path.join(ROOT, "tests")))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured 7" in r.stdout, r.stdout + r.stderr


def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=G.DEV)
    q, sc, s2 = (torch.zeros(s, dtype=t, device=G.DEV) for s, t in (((24, 32), torch.uint8), ((24, 4), torch.uint8), ((1,), torch.float32)))
    assert nv4.linear_w4a16(e(0, 64), q, sc, s2).shape == (0, 24)
    sf = nv4.mma_scales(torch.zeros((24, 2), dtype=torch.uint8, device=G.DEV))
    assert nv4.linear_mxfp4(e(0, 64), q, sf).shape == (0, 24)
    w = lambda r, c: (torch.zeros((4, r, c // 2), dtype=torch.uint8, device=G.DEV),
                      torch.zeros((4, r, c // 16), dtype=torch.uint8, device=G.DEV), torch.ones(4, device=G.DEV))
    y, ids, weights = nv4.moe_layer(e(0, 64), e(4, 64), w(32, 64), w(32, 64), w(64, 32), 2)
    assert y.shape == (0, 64) and ids.shape == weights.shape == (0, 2)


def test_nan_scales_in_many_tiles():
    """One NaN scale of either operand reaches its row or column only, in the kernel of many tiles."""
    M, N, K = 2050, 2565, 352
    rng = np.random.default_rng(3)
    qa, qb = (G.u8_dev(rng.integers(0, 256, (r, K // 2), dtype=np.uint8)) for r in (M, N))
    ea, eb = (np.full((r, K // 32), 127, dtype=np.uint8) for r in (M, N))
    ea[2049, 10] = eb[2560, 0] = 255
    got = nv4.gemm_mxfp4(qa, nv4.mma_scales(G.u8_dev(ea)), qb, nv4.mma_scales(G.u8_dev(eb)), dtype=torch.float32)
    want = torch.zeros((M, N), dtype=torch.bool, device=G.DEV)
    want[2049], want[:, 2560] = True, True
    assert torch.equal(torch.isnan(got), want)


@pytest.mark.parametrize("T", [1, 6, 16, 20])
def test_longest_rows(orc, T):
    """K at its limit, where shared memory does not hold 16 rows."""
    rng = np.random.default_rng(T)
    N, K = 170, 65536
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16)
    q, sc = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(0x20, 0x49, (N, K // 16), dtype=np.uint8)
    got = nv4.linear_w4a16(x.to(G.DEV), G.u8_dev(q), G.u8_dev(sc), torch.full((1,), 0.5, device=G.DEV), dtype=torch.float32)
    y, yabs = orc.linear_w4a16(x.double().numpy(), q, sc, 0.5)
    tol = (K / 16 + 40) * 2.0 ** -23 * yabs + 2.0 ** -24 * np.abs(y)
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= tol)
