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


def experts(rng, E, rows, cols):
    q, sc = weights(rng, E * rows, cols)
    return q.view(E, rows, cols // 2), sc.view(E, rows, cols // 16), torch.full((E,), 0.02, device=G.DEV)


@pytest.mark.parametrize("T,E,k,H,I", [(2, 4, 2, 256, 64), (5, 3, 1, 64, 304), (40, 4, 2, 336, 256), (64, 6, 3, 2400, 48)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_moe_experts_flags_what_it_propagates(orc, T, E, k, H, I, dt):
    """A NaN or Inf in a token reaches all its outputs and no other token's, which stay within the bound of
    their sums; a NaN scale reaches the tokens that chose its expert."""
    rng = np.random.default_rng(T)
    gate, up, down = experts(rng, E, I, H), experts(rng, E, I, H), experts(rng, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DT[dt]).to(G.DEV)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).to(G.DEV)
    w = torch.from_numpy(rng.uniform(0.1, 1, (T, k)).astype(np.float32)).to(G.DEV)
    host = lambda m: tuple(t.cpu().numpy() for t in m)  # noqa: E731
    want, dev = orc.moe_experts(x.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy(), host(gate), host(up), host(down))
    # FP32 sums and silu as for ordinary tokens, two roundings of 2^-11 of the hidden values, routing weight and scales
    tol = ((max(H, I) / 16 + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22) * dev + 2.0 ** -24 * np.abs(want) + 1e-38

    def run(x, ids=ids, down=down, up=up):
        f = G.flags_dev()
        y = nv4.moe_experts(x, ids, w, gate, up, down, dtype=torch.float32, d_flags=f)
        nv4.moe_experts(x, ids, w, gate, up, down, dtype=torch.float32)       # without a flag word
        return y.double().cpu().numpy(), f.item()

    y, f = run(x)
    assert f == 0 and np.all(np.abs(y - want) <= tol)
    t = T // 2
    others = [i for i in range(T) if i != t]
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = x.clone()
        bad[t, H - 3] = value
        y, f = run(bad)
        assert f == nv4.FLAG_NONFINITE and not np.isfinite(y[t]).any()
        assert np.all(np.abs(y[others] - want[others]) <= tol[others])
        none = ids.clone()
        none[t] = -1                                          # a token without experts is 0, whatever is in it
        y, f = run(bad, none)
        assert f == 0 and np.all(y[t] == 0) and np.all(np.abs(y[others] - want[others]) <= tol[others])
    e = int(ids[t, 0])
    chose = (ids == e).any(1).cpu().numpy()
    for which in ("up", "down"):
        m = up if which == "up" else down
        sc = m[1].clone()
        sc[e, 3, 0] = 0x7F
        y, f = run(x, **{which: (m[0], sc, m[2])})
        assert f == nv4.FLAG_NONFINITE and np.all(np.abs(y[~chose] - want[~chose]) <= tol[~chose])
        if which == "up":                                     # one hidden value, and so every output
            assert not np.isfinite(y[chose]).any()
        else:                                                 # one output
            assert not np.isfinite(y[chose, 3]).any() and np.isfinite(np.delete(y[chose], 3, 1)).all()


def test_moe_layer_flags_what_it_propagates():
    rng = np.random.default_rng(1)
    T, E, H, I = 3, 4, 64, 32
    gate, up, down = experts(rng, E, I, H), experts(rng, E, I, H), experts(rng, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(G.DEV)
    wr = torch.from_numpy(rng.standard_normal((E, H)).astype(np.float32)).to(torch.bfloat16).to(G.DEV)
    f = G.flags_dev()
    nv4.moe_layer(x, wr, gate, up, down, 2, d_flags=f)
    assert f.item() == 0
    down[1][:, 0, 0] = 0x7F
    nv4.moe_layer(x, wr, gate, up, down, 2, d_flags=f)
    assert f.item() == nv4.FLAG_NONFINITE
