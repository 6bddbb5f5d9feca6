"""Cases of the products and of the mixture-of-experts layer on FP4 weights.

Three operators, each in its plain form (elementary torch operations) and as the library's
call:

  w4a16   y = x @ W^T with BF16 / FP16 rows x and NVFP4 weights (16-element blocks of E2M1
          codes, an E4M3 scale per block, one FP32 scale per tensor)
  mxfp4   y = Q(x) @ W^T with both operands MXFP4 (32-element blocks, E8M0 scales); x is
          quantized within the call
  moe     a mixture-of-experts layer for a few tokens: router, softmax, top k, and the chosen
          experts' gate, up and down products on NVFP4 weights
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoded token through a 2048 x 2048 projection: the smallest call, latency
        {"name": "w4a16_1x2048x2048", "op": "w4a16", "T": 1, "N": 2048, "K": 2048, "dtype": "bf16"},
        # a few sequences decoding through a 16384 -> 2048 down projection
        {"name": "w4a16_5x2048x16384", "op": "w4a16", "T": 5, "N": 2048, "K": 16384, "dtype": "bf16"},
        # a ragged batch of decoding sequences, sizes that no tile divides, FP16 rows
        {"name": "w4a16_61x2880x2880", "op": "w4a16", "T": 61, "N": 2880, "K": 2880, "dtype": "fp16"},
        # a prompt of 4096 tokens through the 2048 -> 16384 gate projection
        {"name": "w4a16_4096x16384x2048", "op": "w4a16", "T": 4096, "N": 16384, "K": 2048, "dtype": "bf16"},
        # one token through one 2880 x 2880 expert matrix
        {"name": "mxfp4_1x2880x2880", "op": "mxfp4", "M": 1, "N": 2880, "K": 2880},
        # a decode batch of 16 through a 2048 -> 16384 projection
        {"name": "mxfp4_16x16384x2048", "op": "mxfp4", "M": 16, "N": 16384, "K": 2048},
        # an odd number of tokens through a 2880 x 2880 matrix
        {"name": "mxfp4_1001x2880x2880", "op": "mxfp4", "M": 1001, "N": 2880, "K": 2880},
        # prompts: four sequences of 4096 tokens, 2048 -> 16384
        {"name": "mxfp4_16384x16384x2048", "op": "mxfp4", "M": 16384, "N": 16384, "K": 2048},
        # one token through 64 experts of 1536 x 4096, eight of them chosen
        {"name": "moe_1x64x4096x1536", "op": "moe", "T": 1, "E": 64, "k": 8, "H": 4096, "I": 1536, "norm": True},
        # three tokens, 32 experts of 2880 x 2880, four chosen, softmax weights as they are
        {"name": "moe_3x32x2880x2880", "op": "moe", "T": 3, "E": 32, "k": 4, "H": 2880, "I": 2880, "norm": False},
        # small experts of odd widths, seven tokens
        {"name": "moe_7x16x1040x304", "op": "moe", "T": 7, "E": 16, "k": 2, "H": 1040, "I": 304, "norm": True},
        # a decode batch of 48: nearly every expert is chosen by a few tokens
        {"name": "moe_48x64x4096x1536", "op": "moe", "T": 48, "E": 64, "k": 8, "H": 4096, "I": 1536, "norm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4a16", "mxfp4", "moe"])
    if op == "w4a16":
        N, K = _log(rng, 48, 16384), 16 * _log(rng, 4, 1024)
        T = min(_log(rng, 1, 4096), max(1, 4096 * 16384 * 2048 // (N * K)))
        return {"op": op, "T": T, "N": N, "K": K, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "mxfp4":
        N, K = _log(rng, 48, 16384), 32 * _log(rng, 2, 512)
        M = min(_log(rng, 1, 16384), max(1, 16384 * 16384 * 2048 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K}
    E = _log(rng, 4, 64)
    return {"op": op, "T": _log(rng, 1, 48), "E": E, "k": rng.randint(1, min(8, E)), "H": 16 * _log(rng, 16, 256),
            "I": 16 * _log(rng, 8, 96), "norm": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _laplace(gen, rows, cols):
    """Activations: Laplace(1) with 0.5% outlier channels x 50."""
    u = torch.rand((rows, cols), generator=gen, device=DEV) - 0.5
    x = -u.sign() * torch.log1p((-2.0 * u.abs()).clamp(min=-1.0 + 2.0 ** -24))
    n = max(1, cols // 200)
    x[:, torch.randperm(cols, generator=gen, device=DEV)[:n]] *= 50.0
    return x


def _student(gen, rows, cols, std):
    """Weights with Student-t(4) tails."""
    z = torch.randn((rows, cols), generator=gen, device=DEV)
    e = torch.empty((rows, cols), device=DEV)
    v = e.exponential_(generator=gen).clone() + e.exponential_(generator=gen)
    return z * torch.sqrt(2.0 / v) * (std / math.sqrt(2.0))


def _pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _codes(y):
    """E2M1 codes of values already divided by their scale, nearest with ties to even, saturating."""
    a = y.abs()
    r = torch.where(a < 2.0, torch.round(a * 2.0) * 0.5, torch.where(a < 4.0, torch.round(a), 2.0 * torch.round(a * 0.5)))
    r = r.clamp(max=6.0)
    mag = torch.where(r < 2.0, r * 2.0, torch.where(r < 4.0, r + 2.0, r * 0.5 + 4.0))
    return mag.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)


def _nvfp4(w):
    """Weights as round-to-nearest NVFP4: packed codes, E4M3 bytes, the tensor's scale."""
    rows, cols = w.shape
    b = w.view(rows, cols // 16, 16)
    s2 = w.abs().amax() / 2688.0
    sc = (b.abs().amax(-1) / (6.0 * s2)).to(torch.float8_e4m3fn)
    S = (sc.float() * s2).clamp(min=1e-30)
    return _pack(_codes(b / S[..., None]).view(rows, cols)), sc.view(torch.uint8), s2


def _pow2(k):
    """2^k in 32 bits for whole k from -127 to 127, exactly (pow() is not)."""
    return torch.where(k > -127, (k.clamp(min=-126) + 127) << 23, 1 << 22).int().view(torch.float32)


def _pow2_64(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mx_scale(x):
    """E8M0 codes of 32-element blocks: floor(log2 amax) - 2."""
    b = x.view(x.shape[0], -1, 32)
    a = b.abs().amax(-1)
    return torch.where(a > 0, (torch.frexp(a).exponent - 3).clamp(min=-127), -127) + 127


def _mxfp4(x):
    e = _mx_scale(x)
    y = x.view(x.shape[0], -1, 32) * _pow2(127 - e)[..., None]
    return _codes(y).view(x.shape), e.to(torch.uint8)


def _mma_layout(sc):
    """Block-scale bytes [rows, blocks] as the atoms (128 rows x 4 scales, 512 bytes) that the
    block-scaled tensor-core product reads; rows and blocks padded with zeros."""
    rows, kb = sc.shape
    p = torch.zeros((-(-rows // 128) * 128, -(-kb // 4) * 4), dtype=torch.uint8, device=sc.device)
    p[:rows, :kb] = sc
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _experts(gen, E, rows, cols):
    qs, ss, s2s = [], [], []
    for _ in range(E):
        q, s, s2 = _nvfp4(_student(gen, rows, cols, 0.015))
        qs.append(q)
        ss.append(s)
        s2s.append(s2)
    return torch.stack(qs), torch.stack(ss), torch.stack(s2s).float()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "w4a16":
        st["x"] = _laplace(gen, case["T"], case["K"]).to(DTYPES[case["dtype"]])
        q, s, s2 = _nvfp4(0.02 * torch.randn((case["N"], case["K"]), generator=gen, device=DEV))
        st["q"], st["s"], st["s2"] = q, s, s2.view(1)
    elif case["op"] == "mxfp4":
        st["x"] = _laplace(gen, case["M"], case["K"]).to(torch.bfloat16)
        c, e = _mxfp4(0.02 * torch.randn((case["N"], case["K"]), generator=gen, device=DEV))
        st["q"], st["s"], st["s_mma"] = _pack(c), e, _mma_layout(e)
    else:
        E, H, I = case["E"], case["H"], case["I"]
        st["x"] = _laplace(gen, case["T"], H).to(torch.bfloat16)
        st["router"] = (torch.randn((E, H), generator=gen, device=DEV) / (6.0 * math.sqrt(H))).to(torch.bfloat16)
        st["gate"], st["up"] = _experts(gen, E, I, H), _experts(gen, E, I, H)
        st["down"] = _experts(gen, E, H, I)
    return st


# ------------------------------------------------------------------ the plain forms
def _values(q):
    """E2M1 values of packed codes [..., n / 2] -> [..., n]."""
    tab = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    return torch.stack([tab[(q & 15).int()], tab[(q >> 4).int()]], dim=-1).flatten(-2)


def _nv_weights(q, s):
    """e2m1 * e4m3 of NVFP4 weights, without the tensor's scale: exact in 32 bits."""
    v = _values(q)
    return (v.unflatten(-1, (-1, 16)) * s.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_w4a16(st):
    y = (st["x"].float() @ _nv_weights(st["q"], st["s"]).T) * st["s2"]
    return y.to(st["x"].dtype)


def _plain_mxfp4(st):
    x = st["x"].float()
    c, e = _mxfp4(x)
    a = (_values(_pack(c)).unflatten(-1, (-1, 32)) * _pow2(e.int() - 127)[..., None]).flatten(-2)
    w = (_values(st["q"]).unflatten(-1, (-1, 32)) * _pow2(st["s"].int() - 127)[..., None]).flatten(-2)
    return (a @ w.T).to(torch.bfloat16)


def _plain_moe(st):
    x, k = st["x"], st["k"]
    logits = x.double() @ st["router"].double().T          # the choice is a border: 64 bits
    top, ids = (v[:, :k] for v in torch.sort(logits, dim=-1, descending=True, stable=True))
    ex = torch.exp(top - top[:, :1])
    w = ex / (ex.sum(-1, keepdim=True) if st["norm"] else torch.exp(logits - top[:, :1]).sum(-1, keepdim=True))
    w = w.float()
    xf = x.float()
    (gq, gs, g2), (uq, us, u2), (dq, ds, d2) = st["gate"], st["up"], st["down"]
    if x.shape[0] * k <= gq.shape[0]:                       # fewer pairs than experts: gather the chosen ones
        f = ids.flatten()
        xe = xf.repeat_interleave(k, 0)[:, :, None]
        g = (_nv_weights(gq[f], gs[f]) @ xe).squeeze(-1) * g2[f][:, None]
        u = (_nv_weights(uq[f], us[f]) @ xe).squeeze(-1) * u2[f][:, None]
        h = g / (1.0 + torch.exp(-g)) * u * w.flatten()[:, None]
        y = ((_nv_weights(dq[f], ds[f]) @ h[:, :, None]).squeeze(-1) * d2[f][:, None]).view(x.shape[0], k, -1).sum(1)
    else:                                                   # every expert on every token, weighted by 0 where not chosen
        dense = torch.zeros(logits.shape, device=x.device).scatter_(1, ids, w)
        g = (xf @ _nv_weights(gq, gs).transpose(1, 2)) * g2[:, None, None]
        u = (xf @ _nv_weights(uq, us).transpose(1, 2)) * u2[:, None, None]
        h = g / (1.0 + torch.exp(-g)) * u * dense.T[:, :, None]
        y = ((h @ _nv_weights(dq, ds).transpose(1, 2)) * d2[:, None, None]).sum(0)
    return {"y": y.to(x.dtype), "ids": ids.int(), "weights": w}


def run(st):
    op = st["op"]
    if own:
        from nvfp4_block_numerics_b200 import binding as nv4

        if op == "w4a16":
            return nv4.linear_w4a16(st["x"], st["q"], st["s"], st["s2"])
        if op == "mxfp4":
            return nv4.linear_mxfp4(st["x"], st["q"], st["s_mma"])
        y, ids, w = nv4.moe_layer(st["x"], st["router"], st["gate"], st["up"], st["down"], st["k"], renormalize=st["norm"])
        return {"y": y, "ids": ids, "weights": w}
    return {"w4a16": _plain_w4a16, "mxfp4": _plain_mxfp4, "moe": _plain_moe}[op](st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "w4a16":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": 2 * T * K + N * K // 2 + N * K // 16 + 4 + 2 * T * N, "flops": 2 * T * N * K}
    if case["op"] == "mxfp4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K // 2 + N * K // 32 + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    active = E * (1.0 - (1.0 - k / E) ** T)                 # experts that some token chooses, expected
    return {"bytes": 4 * T * H + 2 * E * H + 8 * T * k + active * 3 * H * I * 9 / 16,
            "flops": 2 * T * E * H + 6 * T * k * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits
def _dec64(q, scale, n):
    """Values of packed E2M1 codes times their blocks' scales (one per n values), by the format's
    fields: sign, two exponent bits with bias 1, one mantissa bit."""
    c = torch.empty(q.shape[:-1] + (2 * q.shape[-1],), dtype=torch.int64, device=q.device)
    c[..., 0::2] = q & 15
    c[..., 1::2] = q >> 4
    ex, m = ((c >> 1) & 3), (c & 1).double()
    mag = torch.where(ex == 0, 0.5 * m, (1.0 + 0.5 * m) * _pow2_64(ex - 1))
    v = torch.where(c >= 8, -mag, mag)
    return v * scale.repeat_interleave(n, dim=-1)


def _e4m3_64(b):
    c = b.long()
    ex, m = (c >> 3) & 15, (c & 7).double()
    return torch.where(ex == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * _pow2_64(ex - 7))


def _exact_w4a16(st):
    w = _dec64(st["q"], _e4m3_64(st["s"]), 16) * st["s2"].double()
    return st["x"].double() @ w.T


def _exact_mxfp4(st):
    x = st["x"].double()
    M, K = x.shape
    a = x.view(M, K // 32, 32).abs().amax(-1)
    log2 = (a.view(torch.int64) >> 52) - 1023               # floor(log2 a) of a normal number, from its exponent field
    e = torch.where(a > 0, log2 - 2, -127).clamp(min=-127)
    s = _pow2_64(e).repeat_interleave(32, dim=-1)
    r = x.abs() / s
    # the nearest grid value; a value on a midpoint goes to the neighbour with the even code
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    up = torch.bucketize(r, mid, right=True)                # midpoints at or below r
    down = torch.bucketize(r, mid)                          # midpoints below r
    k = torch.where((up != down) & (down % 2 == 0), down, up)
    xq = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[k] * s * torch.sign(x)
    w = _dec64(st["q"], _pow2_64(st["s"].long() - 127), 32)
    return xq @ w.T


def _exact_moe(st):
    x, k = st["x"].double(), st["k"]
    T = x.shape[0]
    logits = (x[:, None, :] * st["router"].double()[None]).sum(-1)
    y = torch.zeros((T, st["H"]), dtype=torch.float64, device=x.device)
    ids = torch.zeros((T, k), dtype=torch.int32, device=x.device)
    wts = torch.zeros((T, k), dtype=torch.float64, device=x.device)
    left = logits.clone()
    for j in range(k):
        best = (left == left.amax(-1, keepdim=True)).double().argmax(-1)      # the lowest index of the largest
        ids[:, j] = best.int()
        wts[:, j] = logits[torch.arange(T, device=x.device), best]
        left[torch.arange(T, device=x.device), best] = -math.inf
    p = torch.softmax(logits, -1).gather(1, ids.long())
    wts = p / p.sum(-1, keepdim=True) if st["norm"] else p
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        dec = [_dec64(st[n][0][e], _e4m3_64(st[n][1][e]), 16) * st[n][2][e].double() for n in ("gate", "up", "down")]
        g, u = x[t] @ dec[0].T, x[t] @ dec[1].T
        y.index_add_(0, t, ((g * torch.sigmoid(g) * u) @ dec[2].T) * wts[t, j][:, None])
    return {"y": y, "ids": ids, "weights": wts}


def exact(case, seed):
    st = prepare(case, seed)
    return {"w4a16": _exact_w4a16, "mxfp4": _exact_mxfp4, "moe": _exact_moe}[case["op"]](st)
