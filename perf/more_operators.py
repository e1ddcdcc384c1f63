"""Cases for the operators of a key-value cache held in NVFP4: the norms and the
rotation of queries and keys, the cache's quantization as it is written and its
reading back, and the attention that reads it.

A cache is uint8 [pages, Hkv, P / 16, 18 D]: page p holds P tokens of every KV head,
in tiles of 16 tokens.  A tile is the keys' codes [16, D/2] (two e2m1 codes a byte,
element 2j in the low nibble), their E4M3 scales [16, D/16] (one per 16 elements),
then the values' codes and scales.  A global amax A (one, or one a KV head) gives
the decode scale 1 / min(6 * bound / A, FLT_MAX).  Slot s is token s % P of page
s / P.
"""
import math
import random

import torch

own = False

BOUND = 448.0
FLT_MAX = 3.4028234663852886e38
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token, norms and rotation of its heads: the call's latency
        {"name": "rope 1 token", "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "x": "bf16",
         "norm": True, "layout": "half", "base": 1e6, "far": 4096, "magnitude": 1.0},
        # a long prompt, the heads taken out of one product of queries, keys and values
        {"name": "rope 16384 tokens", "op": "rope", "T": 16384, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "x": "bf16",
         "norm": True, "layout": "half", "base": 1e6, "far": 16384, "magnitude": 1.0},
        # fp32, odd sizes, part of the head in neighbouring pairs, far positions of a stretched context
        {"name": "rope 1003 f32 part", "op": "rope", "T": 1003, "Hq": 9, "Hkv": 3, "D": 256, "rot": 64, "x": "f32",
         "norm": False, "layout": "interleaved", "base": 1e4, "far": 1 << 20, "magnitude": 1.2},
        # a decode batch's new tokens into the cache, and out again
        {"name": "cache 64 tokens", "op": "cache", "T": 64, "Hkv": 8, "D": 128, "P": 64, "x": "bf16", "amax": "head"},
        # a long prompt's
        {"name": "cache 16384 tokens", "op": "cache", "T": 16384, "Hkv": 8, "D": 128, "P": 64, "x": "bf16",
         "amax": "none"},
        # fp32, odd sizes, small pages
        {"name": "cache 517 f32", "op": "cache", "T": 517, "Hkv": 5, "D": 64, "P": 16, "x": "f32", "amax": "tensor"},
        # one sequence at its beginning: the call's latency
        {"name": "attend 1 of 200", "op": "attend", "B": 1, "n": 1, "lo": 200, "hi": 200, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 64, "x": "bf16", "amax": "none", "causal": True, "window": 0, "sinks": False, "shape": 1},
        # one sequence with a long past: the work is in one axis
        {"name": "attend 1 of 131072", "op": "attend", "B": 1, "n": 1, "lo": 131072, "hi": 131072, "Hq": 32, "Hkv": 8,
         "D": 128, "P": 64, "x": "bf16", "amax": "head", "causal": True, "window": 0, "sinks": False, "shape": 1},
        # a decode batch of sequences of very different lengths
        {"name": "attend 64 ragged", "op": "attend", "B": 64, "n": 1, "lo": 512, "hi": 32768, "Hq": 64, "Hkv": 8,
         "D": 128, "P": 64, "x": "bf16", "amax": "head", "causal": True, "window": 0, "sinks": False, "shape": 5},
        # fp32, a few tokens a sequence to be checked at once, odd heads, a window, sinks, small pages
        {"name": "attend 13 odd f32", "op": "attend", "B": 13, "n": 5, "lo": 1, "hi": 5003, "Hq": 15, "Hkv": 3, "D": 64,
         "P": 16, "x": "f32", "amax": "tensor", "causal": True, "window": 1000, "sinks": True, "shape": 7},
        # large heads, every query seeing every key
        {"name": "attend 9 large heads", "op": "attend", "B": 9, "n": 3, "lo": 700, "hi": 9000, "Hq": 16, "Hkv": 4,
         "D": 256, "P": 32, "x": "bf16", "amax": "none", "causal": False, "window": 0, "sinks": False, "shape": 11},
        # pieces of two prompts on what the cache holds of them
        {"name": "attend 2 prompts", "op": "attend", "B": 2, "n": 2048, "lo": 16384, "hi": 16384, "Hq": 32, "Hkv": 8,
         "D": 128, "P": 64, "x": "bf16", "amax": "head", "causal": True, "window": 0, "sinks": False, "shape": 13},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope", "cache", "attend", "attend"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        while True:
            T, Hkv, D = log_int(1, 16384), rng.randint(1, 16), rng.choice([64, 80, 128, 192, 256])
            Hq = Hkv * rng.randint(1, 8)
            if T * (Hq + Hkv) * D * (2 if x == "f32" else 1) <= 16384 * 40 * 128:
                break
        return {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D // 2 // 16 * 16]), "x": x,
                "norm": rng.random() < 0.6, "layout": rng.choice(["half", "interleaved"]),
                "base": rng.choice([1e4, 5e5, 1e6]), "far": log_int(T, 1 << 20),
                "magnitude": rng.choice([1.0, 1.0, 1.15])}
    D = rng.choice([64, 128, 128, 256])
    P = rng.choice([16, 32, 64, 128])
    amax = rng.choice(["none", "tensor", "head"])
    if op == "cache":
        while True:
            T, Hkv = log_int(1, 16384), rng.randint(1, 16)
            if T * Hkv * D * (2 if x == "f32" else 1) <= 16384 * 8 * 128:
                break
        return {"op": op, "T": T, "Hkv": Hkv, "D": D, "P": P, "x": x, "amax": amax}
    while True:
        B, n, hi = log_int(1, 64), rng.choice([1, 1, rng.randint(2, 8), log_int(9, 2048)]), log_int(1, 131072)
        Hkv = rng.randint(1, 8)
        Hq = Hkv * rng.randint(1, 8)
        lo = log_int(1, hi)
        if B * hi * Hkv * D <= 64 * 32768 * 8 * 128 // 2 and B * n * Hq * hi * D <= 2 * 2048 * 32 * 16384 * 128 // 4:
            break
    return {"op": op, "B": B, "n": n, "lo": lo, "hi": hi, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "x": x, "amax": amax,
            "causal": rng.random() < 0.8, "window": log_int(1, hi) if rng.random() < 0.3 else 0,
            "sinks": rng.random() < 0.3, "shape": rng.randrange(1 << 30)}


def sequences(case):
    """(queries, keys) of each sequence of an attention, drawn from the case alone: the keys hold the queries' own."""
    r = random.Random(case["shape"])
    out = []
    for _ in range(case["B"]):
        keys = int(round(math.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"])))))
        n = case["n"] if case["n"] == 1 or case["n"] > 1024 else r.randint(1, case["n"])
        out.append((n, max(n, keys)))
    return out


# ---- inputs -----------------------------------------------------------------------------------
def _codes(v):
    """e2m1 code of each value, ties to the even code."""
    a = v.abs()
    k = (a > 0.25).to(torch.uint8)
    k += a >= 0.75
    k += a > 1.25
    k += a >= 1.75
    k += a > 2.5
    k += a >= 3.5
    k += a > 5.0
    return k | torch.signbit(v).to(torch.uint8) << 3


def _enc(amax):
    return torch.clamp(torch.full_like(amax, 6.0 * BOUND) / amax, max=FLT_MAX)


def _quantize(y, amax):
    """Codes [..., D/2] and scale bytes [..., D/16] of fp32 y [T, H, D]; amax None, [1] or [H]."""
    g = y.reshape(*y.shape[:2], -1, 16)
    b = g.abs().amax(dim=3)
    s = b / torch.full_like(b, 6.0)
    if amax is not None:
        enc = _enc(amax).reshape(1, -1, 1)
        s = s * enc
    s = s.clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float()
    if amax is not None:
        d = d * (torch.ones_like(enc) / enc)
    c = _codes(g / torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(3))
    c = torch.where(d.unsqueeze(3) > 0, c, torch.zeros_like(c)).reshape(*y.shape[:2], -1, 2)
    return c[..., 0] | c[..., 1] << 4, s.view(torch.uint8)


def _parts(cache):
    """Views of a cache: keys' codes [pages, H, tiles, 16, D/2] and scales [.., 16, D/16], values' the same."""
    D = cache.shape[3] // 18
    at = [0, 8 * D, 9 * D, 17 * D, 18 * D]
    return [cache[..., a:b].unflatten(3, (16, (b - a) // 16)) for a, b in zip(at, at[1:])]


def _place(slots, P):
    """Indexes into those views: [n, H, width] for slots [n]."""
    return slots // P, slice(None), slots % P // 16, slots % 16


def _write(cache, k, v, slots, k_amax, v_amax):
    P = cache.shape[2] * 16
    at = _place(slots, P)
    kc, ks, vc, vs = _parts(cache)
    kc[at], ks[at] = _quantize(k.float(), k_amax)
    vc[at], vs[at] = _quantize(v.float(), v_amax)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    s = {"case": dict(case), "grid": torch.tensor(grid + [-g for g in grid], device=dev)}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "rope":
        T, Hq, Hkv, D, rot = case["T"], case["Hq"], case["Hkv"], case["D"], case["rot"]
        qkv = (3.0 * normal(T, Hq + 2 * Hkv, D)).to(DTYPES[case["x"]])      # one product, cut into heads
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1.0 + 0.1 * normal(D)).to(DTYPES[case["x"]]) for _ in range(2))
        s["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device=dev)
        freq = [case["base"] ** (-2 * i / rot) for i in range(rot // 2)]
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        turns = [int(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]      # of a position, in 2^-64
        s["phases"] = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], device=dev)
        return s
    Hkv, D, P = case["Hkv"], case["D"], case["P"]
    s["k_amax"] = s["v_amax"] = None
    if case["amax"] != "none":
        n = Hkv if case["amax"] == "head" else 1
        s["k_amax"], s["v_amax"] = 60.0 + 10.0 * torch.rand(n, generator=gen, device=dev), 5.0 + torch.rand(
            n, generator=gen, device=dev)

    def keys(T):
        """Normal values with one channel in 50 ten times as large."""
        return normal(T, Hkv, D) * torch.where(torch.rand(Hkv, D, generator=gen, device=dev) < 0.02, 10.0, 1.0)

    if case["op"] == "cache":
        T = case["T"]
        pages = -(-T // P) + 3
        s["cache"] = torch.zeros(pages, Hkv, P // 16, 18 * D, dtype=torch.uint8, device=dev)
        s["slots"] = torch.randperm(pages * P, generator=gen, device=dev)[:T]
        s["k"], s["v"] = keys(T).to(DTYPES[case["x"]]), normal(T, Hkv, D).to(DTYPES[case["x"]])
        return s
    seqs = sequences(case)
    counts = [-(-m // P) for _, m in seqs]
    width, total = max(counts), sum(counts)
    s["cache"] = torch.empty(total + 2, Hkv, P // 16, 18 * D, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 28) // (Hkv * D * P))               # pages filled at once
    for p in range(0, total + 2, step):
        part = s["cache"][p:p + step]
        t = part.shape[0] * P
        _write(part, keys(t), normal(t, Hkv, D), torch.arange(t, device=dev), s["k_amax"], s["v_amax"])
    order = torch.randperm(total + 2, generator=gen, device=dev)[:total].int()
    s["pages"] = torch.zeros(case["B"], width, dtype=torch.int32, device=dev)
    inside = torch.arange(width, device=dev) < torch.tensor(counts, device=dev)[:, None]
    s["pages"][inside] = order
    s["lengths"] = torch.tensor([m for _, m in seqs], device=dev)
    s["offsets"] = None if case["n"] == 1 else torch.tensor([0] + [n for n, _ in seqs], device=dev).cumsum(0)
    s["most"] = max(n for n, _ in seqs)
    T = sum(n for n, _ in seqs)
    s["q"] = (1.5 * normal(T, case["Hq"], D)).to(DTYPES[case["x"]])
    s["sinks"] = normal(case["Hq"]) if case["sinks"] else None
    return s


# ---- plain forms ------------------------------------------------------------------------------
def _rotated(x, weight, cos, sin, layout):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(dim=2, keepdim=True) + 1e-6) * weight.float()
    half = cos.shape[2]
    turned, rest = y[..., :2 * half], y[..., 2 * half:]
    if layout == "half":
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2)
    return torch.cat([turned, rest], dim=2).to(x.dtype)


def _rope_plain(s):
    c = s["case"]
    angle = (s["positions"].double()[:, None] * s["freq"])[:, None]
    cos, sin = (angle.cos() * c["magnitude"]).float(), (angle.sin() * c["magnitude"]).float()
    return {"q": _rotated(s["q"], s["q_weight"], cos, sin, c["layout"]),
            "k": _rotated(s["k"], s["k_weight"], cos, sin, c["layout"])}


def _values(codes, scales, amax, grid):
    """fp32 values [..., H, D] of codes [..., H, D/2] and scale bytes [..., H, D/16]."""
    q = grid[torch.stack([codes & 15, codes >> 4], dim=-1).int()]
    d = scales.view(torch.float8_e4m3fn).float()
    y = q.reshape(*d.shape, 16) * d.unsqueeze(-1)
    if amax is not None:
        enc = _enc(amax).reshape(-1, 1, 1)
        y = y * (torch.ones_like(enc) / enc)
    return y.flatten(-2)


def _cache_plain(s):
    _write(s["cache"], s["k"], s["v"], s["slots"], s["k_amax"], s["v_amax"])
    kc, ks, vc, vs = (p[_place(s["slots"], s["case"]["P"])] for p in _parts(s["cache"]))
    dt = s["k"].dtype
    return {"k": _values(kc, ks.contiguous(), s["k_amax"], s["grid"]).to(dt),
            "v": _values(vc, vs.contiguous(), s["v_amax"], s["grid"]).to(dt)}


def _attend_plain(s):
    """Every sequence padded to the most queries and the most keys, one batched softmax."""
    c = s["case"]
    B, P, H, D = c["B"], c["P"], c["Hkv"], c["D"]
    dev, q, most = s["q"].device, s["q"], s["most"]
    G, T = c["Hq"] // H, q.shape[0]
    off = torch.arange(B + 1, device=dev) if s["offsets"] is None else s["offsets"]
    n, keys = off[1:] - off[:-1], s["lengths"]
    at = off[:-1, None] + torch.arange(most, device=dev)
    j = torch.arange(s["pages"].shape[1] * P, device=dev)
    page = s["pages"].long()[:, j // P]
    kc, ks, vc, vs = (p[page, :, (j % P // 16).expand_as(page), (j % 16).expand_as(page)] for p in _parts(s["cache"]))
    k = _values(kc, ks.contiguous(), s["k_amax"], s["grid"])
    qq = q.float()[at.clamp(max=T - 1)].reshape(B, most, H, G, D)
    x = torch.einsum("bnhgd,blhd->bhgnl", qq, k) * D ** -0.5
    del k
    pos = (keys - n)[:, None] + torch.arange(most, device=dev)      # of each query
    see = (j < keys[:, None])[:, None].expand(B, most, -1)
    if c["causal"]:
        see = see & (j <= pos[:, :, None])
    if c["window"]:
        see = see & (j > pos[:, :, None] - c["window"])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    top = x.amax(dim=4, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].reshape(1, H, G, 1, 1)
        top = torch.maximum(top, sink)
    e = torch.exp(x - top.clamp(min=-FLT_MAX))
    del x
    total = e.sum(dim=4, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - top)
    v = _values(vc, vs.contiguous(), s["v_amax"], s["grid"])
    o = torch.einsum("bhgnl,blhd->bnhgd", e, v) / total.clamp(min=1e-30).permute(0, 3, 1, 2, 4)
    row = torch.arange(T, device=dev)
    b = torch.searchsorted(off[1:].contiguous(), row, right=True)
    return o[b, row - off[b]].reshape(T, c["Hq"], D).to(q.dtype)


def run(state):
    case = state["case"]
    if not own:
        return {"rope": _rope_plain, "cache": _cache_plain, "attend": _attend_plain}[case["op"]](state)
    import nvfp4_block_quantization_quantize_gb300 as nv
    if case["op"] == "rope":
        return nv.nvfp4_qk_norm_rope(state["q"], state["k"], state["positions"], state["phases"],
                                     q_weight=state["q_weight"], k_weight=state["k_weight"], eps=1e-6,
                                     layout=case["layout"], magnitude=case["magnitude"])
    if case["op"] == "cache":
        nv.nvfp4_cache_write(state["cache"], state["k"], state["v"], state["slots"], k_gamax=state["k_amax"],
                             v_gamax=state["v_amax"])
        k, v = nv.nvfp4_cache_read(state["cache"], state["slots"], k_gamax=state["k_amax"], v_gamax=state["v_amax"],
                                   out_dtype=case["x"])
        return {"k": k, "v": v}
    return nv.nvfp4_cache_attention(state["q"], state["cache"], state["pages"], state["lengths"],
                                    offsets=state["offsets"], k_gamax=state["k_amax"], v_gamax=state["v_amax"],
                                    causal=case["causal"], window=case["window"], sinks=state["sinks"],
                                    out_dtype=case["x"])


# ---- what a pass needs, and its exact result --------------------------------------------------
def _seen(case, n, keys):
    """(pairs of a query and a key it sees, keys that some query sees) of one sequence."""
    pairs, first, last = 0, keys, 0
    for i in range(n):
        pos = keys - n + i
        end = pos + 1 if case["causal"] else keys
        begin = max(0, pos - case["window"] + 1) if case["window"] else 0
        if end > begin:
            pairs += end - begin
            first, last = min(first, begin), max(last, end)
    return pairs, max(0, last - first)


def work(case):
    e = {"f32": 4, "bf16": 2}[case["x"]]
    D, H = case["D"], case["Hkv"]
    if case["op"] == "rope":
        n = case["T"] * (case["Hq"] + H) * D
        return {"bytes": 2 * n * e + 8 * case["T"] + 4 * case["rot"] + (2 * D * e if case["norm"] else 0),
                "flops": n * (7 if case["norm"] else 3)}
    if case["op"] == "cache":
        n = 2 * case["T"] * H * D                            # values in, 9/16 of a byte each out and in, values out
        return {"bytes": 2 * n * e + 2 * n * 9 // 16 + 16 * case["T"], "flops": 4 * n}
    seqs = [(n, *_seen(case, n, keys)) for n, keys in sequences(case)]
    T = sum(n for n, _, _ in seqs)
    pairs, keys = (sum(q[i] for q in seqs) for i in (1, 2))
    return {"bytes": keys * H * D * 9 // 8 + 2 * T * case["Hq"] * D * e + 4 * (keys // case["P"]) + 8 * case["B"],
            "flops": 4 * pairs * case["Hq"] * D}


def _nearest(v, bits, low, top):
    """v rounded to `bits` bits after the leading one, ties to even; steps end at exponent `low`, values at `top`."""
    m = torch.frexp(v)[0].abs()                             # v / m is a power of two, exactly
    step = torch.where(m > 0, v.abs() / m / 2.0, torch.zeros_like(v)).clamp(min=2.0 ** low) / 2.0 ** bits
    return (torch.round(v / step) * step).clamp(-top, top)


def _quantized64(y, amax):
    """What 16 elements with one scale are held as, in 64 bits."""
    g = y.double().reshape(*y.shape[:2], -1, 16)
    enc = 1.0 if amax is None else (6.0 * BOUND / amax.double()).reshape(1, -1, 1)
    b = g.abs().amax(dim=3)                             # over a tensor of sixes: a plain 6.0 is taken as its inverse
    s = _nearest(b / torch.full_like(b, 6.0) * enc, 3, -6.0, 448.0) / enc
    q = _nearest(g / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(3), 1, 0.0, 6.0)
    return (q * s.unsqueeze(3)).reshape(y.shape)


def _values64(codes, scales, amax):
    """Values in 64 bits from the fields of each code and scale byte: [n, D] of one head."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(torch.int16)
    e, m = (c >> 1) & 3, c & 1
    mag = torch.where(e > 0, (2 + m) * torch.pow(2.0, (e - 2).double()), m * 0.5)
    q = torch.where(c > 7, -mag, mag)
    b = scales.to(torch.int16)
    e, m = (b >> 3) & 15, b & 7
    d = torch.where(e > 0, (8 + m) * torch.pow(2.0, (e - 10).double()), m * 2.0 ** -9)
    v = q * d.repeat_interleave(16, dim=-1)
    return v if amax is None else v / (6.0 * BOUND / amax.double())


def _rope64(s):
    c = s["case"]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if c["norm"]:
            x = x / torch.sqrt(x.square().sum(dim=2, keepdim=True) / c["D"] + 1e-6) * s[name + "_weight"].double()
        half = c["rot"] // 2
        i = torch.arange(half, device=x.device)
        first, second = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.polar(torch.full_like(s["freq"], c["magnitude"]).expand(c["T"], half),
                        s["positions"].double()[:, None] * s["freq"])
        p = torch.complex(x[..., first], x[..., second]) * z[:, None]
        y = x.clone()
        y[..., first], y[..., second] = p.real, p.imag
        out[name] = y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope64(s)
    if case["op"] == "cache":
        return {"k": _quantized64(s["k"], s["k_amax"]), "v": _quantized64(s["v"], s["v_amax"])}
    H, P, D, G = case["Hkv"], case["P"], case["D"], case["Hq"] // case["Hkv"]
    seqs = sequences(case)
    if sum(_seen(case, *q)[0] for q in seqs) * case["Hq"] * D > 1 << 41:
        return None
    views = _parts(s["cache"])
    out, row = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device), 0
    for b, (n, keys) in enumerate(seqs):
        pages = s["pages"][b, :-(-keys // P)].long()
        pos = torch.arange(keys - n, keys, device=out.device)[:, None]
        j = torch.arange(keys, device=out.device)
        for h in range(H):
            kc, ks, vc, vs = (p[pages, h].flatten(0, 2)[:keys] for p in views)
            k, v = (_values64(x, y, None if a is None else a.expand(H)[h])
                    for x, y, a in ((kc, ks, s["k_amax"]), (vc, vs, s["v_amax"])))
            for r in range(0, n, 512):
                p = pos[r:r + 512]
                q = s["q"][row + r:row + r + p.shape[0], h * G:(h + 1) * G].double()
                x = torch.matmul(q.transpose(0, 1), k.t()) / math.sqrt(D)
                hidden = torch.zeros(p.shape[0], keys, dtype=torch.bool, device=out.device)
                if case["causal"]:
                    hidden |= j > p
                if case["window"]:
                    hidden |= j <= p - case["window"]
                x = x.masked_fill(hidden, -math.inf)
                if s["sinks"] is not None:
                    sink = s["sinks"].double()[h * G:(h + 1) * G].reshape(G, 1, 1).expand(G, p.shape[0], 1)
                    x = torch.cat([x, sink], dim=2)
                w = torch.softmax(x, dim=2)[..., :keys]
                out[row + r:row + r + p.shape[0], h * G:(h + 1) * G] = torch.matmul(w, v).transpose(0, 1)
        row += n
    return out
