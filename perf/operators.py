"""Cases for the serving operators on NVFP4 weights: the fused residual-add
RMS norm with an 8-bit block-scaled output, the product of a few tokens with
an NVFP4 weight, and the products grouped by expert with ragged sizes.

An NVFP4 tensor [rows, K] is codes [rows, K/2] (two e2m1 codes a byte, element
2j in the low nibble), one E4M3 scale byte per 16 elements and an optional
fp32 global amax A with decode scale 1 / min(6 * bound / A, FLT_MAX).  An
MXFP8 tensor is E4M3 codes [rows, K] and one E8M0 byte (2^(byte - 127)) per 32
elements; the last group of a row may hold 16.
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
        # a small projection of one decoded token: the call's latency
        {"name": "mv 1 x 1024x1024", "op": "mv", "M": 1, "N": 1024, "K": 1024, "x": "bf16", "amax": "none",
         "out": "bf16"},
        # the feed-forward weight [14336, 4096] on one decoded token
        {"name": "mv 1 x 14336x4096", "op": "mv", "M": 1, "N": 14336, "K": 4096, "x": "bf16", "amax": "tensor",
         "out": "bf16"},
        # the way back, [4096, 14336], on a decode batch whose activations the norm left in 8 bits
        {"name": "mv 8 mxfp8 x 4096x14336", "op": "mv", "M": 8, "N": 4096, "K": 14336, "x": "mxfp8",
         "amax": "tensor", "out": "bf16"},
        # odd sizes, fp32 activations, a row-scaled weight
        {"name": "mv 13 f32 x 5003x2064", "op": "mv", "M": 13, "N": 5003, "K": 2064, "x": "f32", "amax": "row",
         "out": "f32"},
        # the last projection to a vocabulary, for a few sequences
        {"name": "mv 4 x 65536x8192", "op": "mv", "M": 4, "N": 65536, "K": 8192, "x": "bf16", "amax": "tensor",
         "out": "f32"},
        # one decoded token's norm: the call's latency
        {"name": "norm 1x4096", "op": "norm", "M": 1, "K": 4096, "x": "bf16", "hidden": True, "weight": "bf16"},
        # the activations of a long prompt
        {"name": "norm 16384x4096", "op": "norm", "M": 16384, "K": 4096, "x": "bf16", "hidden": True,
         "weight": "bf16"},
        # odd rows, a last group of 16, fp32, nothing to add
        {"name": "norm 517x7152 f32", "op": "norm", "M": 517, "K": 7152, "x": "f32", "hidden": False,
         "weight": "f32"},
        # a single token sent to 2 of 8 small experts: the call's latency
        {"name": "grouped 2 of 8", "op": "grouped", "E": 8, "T": 2, "N": 1024, "K": 1024, "a_amax": "none",
         "b_amax": False, "out": "bf16", "routing": 3},
        # decode: 8 tokens to 8 of 64 experts each
        {"name": "grouped 64 of 64", "op": "grouped", "E": 64, "T": 64, "N": 2048, "K": 4096, "a_amax": "tensor",
         "b_amax": True, "out": "bf16", "routing": 5},
        # ragged rows, sizes off the tiles, empty experts, row-scaled activations
        {"name": "grouped 1999 of 13 odd", "op": "grouped", "E": 13, "T": 1999, "N": 1430, "K": 2112,
         "a_amax": "row", "b_amax": True, "out": "f32", "routing": 7},
        # prompt tokens through 8 experts of [14336, 4096]
        {"name": "grouped 8192 of 8", "op": "grouped", "E": 8, "T": 8192, "N": 14336, "K": 4096,
         "a_amax": "tensor", "b_amax": True, "out": "bf16", "routing": 11},
    ]


def draw(rng):
    def log_int(lo, hi, step=1):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))

    op = rng.choice(["mv", "norm", "grouped"])
    if op == "mv":
        while True:
            N, K = log_int(64, 65536), log_int(256, 16384, 16)
            if N * K <= 65536 * 8192:
                break
        return {"op": op, "M": rng.randint(1, 16), "N": N, "K": K, "x": rng.choice(["f32", "bf16", "mxfp8"]),
                "amax": rng.choice(["none", "tensor", "row"]), "out": rng.choice(["f32", "bf16"])}
    if op == "norm":
        while True:
            M, K = log_int(1, 16384), log_int(64, 16384, 16)
            if M * K <= 16384 * 4096:
                break
        x = rng.choice(["f32", "bf16"])
        if x == "f32" and M * K > 8192 * 4096:
            M = max(1, M // 2)
        return {"op": op, "M": M, "K": K, "x": x, "hidden": rng.random() < 0.7,
                "weight": rng.choice(["f32", "bf16"])}
    while True:
        E, T = rng.randint(1, 64), log_int(1, 8192)
        N, K = log_int(64, 14336), log_int(64, 8192, 64)
        if E * N * K <= 8 * 14336 * 4096 and T * N * K <= 8192 * 14336 * 4096:
            break
    return {"op": op, "E": E, "T": T, "N": N, "K": K, "a_amax": rng.choice(["none", "tensor", "row"]),
            "b_amax": rng.random() < 0.5, "out": rng.choice(["f32", "bf16"]), "routing": rng.randrange(1 << 30)}


def counts(case):
    """Rows of each expert: a skewed routing, drawn from the case alone."""
    r = random.Random(case["routing"])
    p = [math.exp(r.gauss(0.0, 0.7)) for _ in range(case["E"])]
    n = [0] * case["E"]
    for e in r.choices(range(case["E"]), p, k=case["T"]):
        n[e] += 1
    return n


# ---- inputs -----------------------------------------------------------------------------------
def _codes(v):
    """e2m1 code of each value, ties to the even code."""
    a = v.abs()
    k = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                     (5.0, False)):
        k += (a >= edge) if up else (a > edge)
    return k | (v < 0).to(torch.uint8) << 3


def _nvfp4(y, amax):
    """Codes and scale bytes of fp32 y [rows, K]; amax broadcasts over rows, or None."""
    rows, K = y.shape
    enc = 1.0 if amax is None else (6.0 * BOUND / amax).reshape(-1, 1)
    b = y.reshape(rows, K // 16, 16).abs().amax(dim=2)
    s = (b / 6.0 * enc).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() / enc
    v = y.reshape(rows, K // 16, 16) / torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(2)
    c = _codes(v).reshape(rows, K // 2, 2)
    return c[..., 0] | c[..., 1] << 4, s.view(torch.uint8)


def _mxfp8(y):
    rows, K = y.shape
    pad = -K % 32
    g = torch.nn.functional.pad(y, (0, pad)).reshape(rows, -1, 32)
    m, k = torch.frexp(g.abs().amax(dim=2))
    e = torch.where(m > 0.875, k - 8, k - 9).clamp(min=-127)
    e = torch.where(m > 0, e, torch.full_like(e, -127))
    q = torch.ldexp(g, -e.unsqueeze(2)).to(torch.float8_e4m3fn).reshape(rows, K + pad)[:, :K]
    return q.contiguous(), (e + 127).to(torch.uint8)


def _mma_layout(s):
    """Scale bytes [E, rows, cols] in the tensor cores' layout: 128 x 4 tiles of
    512 bytes, byte (r, c) of a tile at (r % 32) * 16 + (r / 32) * 4 + c."""
    E, rows, cols = s.shape
    s = torch.nn.functional.pad(s, (0, -cols % 4, 0, -rows % 128))
    R, C = s.shape[1:]
    return s.reshape(E, R // 128, 4, 32, C // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, R, C).contiguous()


def _activations(gen, M, K, dev):
    """Normal values with one channel in 500 twenty times as large."""
    x = torch.randn(M, K, generator=gen, device=dev)
    return x * torch.where(torch.rand(K, generator=gen, device=dev) < 0.002, 20.0, 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    s = {"case": dict(case), "grid": torch.tensor(grid + [-g for g in grid], device=dev)}
    if case["op"] == "mv":
        M, N, K = case["M"], case["N"], case["K"]
        w = torch.randn(N, K, generator=gen, device=dev) * 0.02
        s["amax"] = {"none": lambda: None, "tensor": lambda: w.abs().amax().reshape(1),
                     "row": lambda: w.abs().amax(dim=1)}[case["amax"]]()
        s["codes"], s["scales"] = _nvfp4(w, s["amax"])
        x = _activations(gen, M, K, dev)
        s["x_scales"] = None
        if case["x"] == "mxfp8":
            q, s["x_scales"] = _mxfp8(x)
            s["x"] = q.view(torch.uint8)
        else:
            s["x"] = x.to(DTYPES[case["x"]])
        return s
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        s["x"] = _activations(gen, M, K, dev).to(DTYPES[case["x"]])
        s["hidden"] = _activations(gen, M, K, dev).to(DTYPES[case["x"]]) if case["hidden"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(K, generator=gen, device=dev)).to(DTYPES[case["weight"]])
        return s
    E, T, N, K = case["E"], case["T"], case["N"], case["K"]
    n = counts(case)
    s["offsets"] = torch.tensor([0] + n, device=dev).cumsum(0)
    s["most"] = max(n)
    w = torch.randn(E, N, K, generator=gen, device=dev) * 0.02
    s["b_amax"] = w.abs().amax(dim=(1, 2)) if case["b_amax"] else None
    per_row = None if s["b_amax"] is None else s["b_amax"].repeat_interleave(N)
    c, b = _nvfp4(w.reshape(E * N, K), per_row)
    del w
    s["b_codes"], s["b_scales"] = c.reshape(E, N, K // 2), b.reshape(E, N, K // 16)
    s["b_scales_mma"] = _mma_layout(s["b_scales"])
    x = _activations(gen, T, K, dev)
    s["a_amax"] = {"none": lambda: None, "tensor": lambda: x.abs().amax().reshape(1),
                   "row": lambda: x.abs().amax(dim=1)}[case["a_amax"]]()
    s["a_codes"], s["a_scales"] = _nvfp4(x, s["a_amax"])
    return s


# ---- plain forms ------------------------------------------------------------------------------
def _values(codes, scales, grid):
    """fp32 values of NVFP4 codes [..., K/2] and scale bytes [..., K/16], without the global scale."""
    q = grid[torch.stack([codes & 15, codes >> 4], dim=-1).int()]
    d = scales.view(torch.float8_e4m3fn).float()
    return (q.reshape(*d.shape, 16) * d.unsqueeze(-1)).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _dec(amax):
    return 1.0 / (6.0 * BOUND / amax).clamp(max=FLT_MAX)


def _mv_plain(s):
    x = s["x"]
    if s["x_scales"] is not None:
        g = torch.pow(2.0, s["x_scales"].float() - 127.0).repeat_interleave(32, dim=1)[:, :x.shape[1]]
        x = x.view(torch.float8_e4m3fn).float() * g
    y = x.float() @ _values(s["codes"], s["scales"], s["grid"]).t()
    if s["amax"] is not None:
        y = y * _dec(s["amax"])
    return y.to(DTYPES[s["case"]["out"]])


def _norm_plain(s):
    h = s["x"].float()
    if s["hidden"] is not None:
        h = h + s["hidden"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * s["weight"].float()
    q, e = _mxfp8(y)
    out = {"codes": q, "scales": e.view(torch.float8_e8m0fnu)}
    if s["hidden"] is not None:
        out["hidden"] = h.to(s["hidden"].dtype)
    return out


def _grouped_plain(s):
    """The experts' rows padded to the longest, one batched product, the rows taken back."""
    off, T = s["offsets"], s["a_codes"].shape[0]
    a = _values(s["a_codes"], s["a_scales"], s["grid"])
    if s["a_amax"] is not None:
        a = a * _dec(s["a_amax"]).reshape(-1, 1)
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)
    y = torch.bmm(a[at.clamp(max=T - 1)], _values(s["b_codes"], s["b_scales"], s["grid"]).transpose(1, 2))
    if s["b_amax"] is not None:
        y = y * _dec(s["b_amax"]).reshape(-1, 1, 1)
    row = torch.arange(T, device=off.device)
    e = torch.searchsorted(off[1:], row, right=True)
    return y[e, row - off[e]].to(DTYPES[s["case"]["out"]])


def run(state):
    case = state["case"]
    if not own:
        return {"mv": _mv_plain, "norm": _norm_plain, "grouped": _grouped_plain}[case["op"]](state)
    import nvfp4_block_quantization_quantize_gb300 as nv
    if case["op"] == "mv":
        return nv.nvfp4_mv(state["x"], state["codes"], state["scales"], x_scales=state["x_scales"],
                           gamax=state["amax"], out_dtype=case["out"])
    if case["op"] == "norm":
        r = nv.nvfp4_rmsnorm(state["x"], state["weight"], hidden=state["hidden"], eps=1e-6)
        out = {"codes": r["codes"].view(torch.float8_e4m3fn), "scales": r["scales"].view(torch.float8_e8m0fnu)}
        if state["hidden"] is not None:
            out["hidden"] = r["hidden"]
        return out
    return nv.nvfp4_grouped_mm(state["a_codes"], state["a_scales"], state["offsets"], state["b_codes"],
                               state["b_scales_mma"], gamax_a=state["a_amax"], gamax_b=state["b_amax"],
                               out_dtype=case["out"])


# ---- what a pass needs, and its exact result --------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "mv":
        M, N, K = case["M"], case["N"], case["K"]
        x = M * K * size[case["x"]] if case["x"] != "mxfp8" else M * (K + -(-K // 32))
        amax = {"none": 0, "tensor": 4, "row": 4 * N}[case["amax"]]
        return {"bytes": N * K * 9 // 16 + x + amax + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        e = size[case["x"]]
        return {"bytes": M * K * (e * (3 if case["hidden"] else 1) + 1) + M * -(-K // 32) + K * size[case["weight"]],
                "flops": 8 * M * K}
    E, T, N, K = case["E"], case["T"], case["N"], case["K"]
    used = sum(1 for n in counts(case) if n)
    amax = {"none": 0, "tensor": 4, "row": 4 * T}[case["a_amax"]] + (4 * used if case["b_amax"] else 0)
    return {"bytes": used * N * K * 9 // 16 + T * K * 9 // 16 + 8 * (E + 1) + amax + T * N * size[case["out"]],
            "flops": 2 * T * N * K}


def _values64(codes, scales, amax):
    """NVFP4 values in 64 bits from the fields of each code and scale byte; amax broadcasts over the rows."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(torch.int16)
    e, m = (c >> 1) & 3, c & 1
    mag = torch.where(e > 0, (2 + m) * torch.pow(2.0, (e - 2).double()), m * 0.5)
    q = torch.where(c > 7, -mag, mag)
    b = scales.to(torch.int16)
    e, m = (b >> 3) & 15, b & 7
    d = torch.where(e > 0, (8 + m) * torch.pow(2.0, (e - 10).double()), m * 2.0 ** -9)
    v = q * d.repeat_interleave(16, dim=-1)
    if amax is not None:
        v = v / (6.0 * BOUND / amax.double()).unsqueeze(-1)
    return v


def _norm64(s):
    h = s["x"].double() + (s["hidden"].double() if s["hidden"] is not None else 0.0)
    M, K = h.shape
    y = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / K + 1e-6) * s["weight"].double()
    y = torch.cat([y, y.new_zeros(M, -K % 32)], dim=1).reshape(M, -1, 32)
    top = y.abs().amax(dim=2, keepdim=True)
    e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-127.0)
    v = y / torch.pow(2.0, e)
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    out = {"codes": (torch.round(v / step) * step).reshape(M, -1)[:, :K], "scales": torch.pow(2.0, e).squeeze(2)}
    if s["hidden"] is not None:
        out["hidden"] = h
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "mv":
        x = s["x"]
        if s["x_scales"] is not None:
            p = torch.pow(2.0, s["x_scales"].double() - 127.0)
            x = x.view(torch.float8_e4m3fn).double() * p[:, torch.arange(x.shape[1], device=x.device) // 32]
        amax = None if s["amax"] is None else s["amax"].expand(case["N"])
        parts = []
        for r in range(0, case["N"], 8192):
            w = _values64(s["codes"][r:r + 8192], s["scales"][r:r + 8192], None if amax is None else amax[r:r + 8192])
            parts.append(x.double() @ w.t())
        return torch.cat(parts, dim=1)
    if case["op"] == "norm":
        return _norm64(s)
    a = _values64(s["a_codes"], s["a_scales"], None if s["a_amax"] is None else s["a_amax"].expand(case["T"]))
    y, at = [], 0
    for e, n in enumerate(counts(case)):
        if n:
            g = None if s["b_amax"] is None else s["b_amax"][e].expand(case["N"])
            y.append(a[at:at + n] @ _values64(s["b_codes"][e], s["b_scales"][e], g).t())
            at += n
    return torch.cat(y, dim=0)
