"""Plain 64-bit forms of the cache operators, for their tests."""
import math

import torch


def parts(cache):
    """Views of a cache: keys' codes [pages, H, tiles, 16, D/2] and scales [.., 16, D/16], values' the same."""
    D = cache.shape[3] // 18
    at = [0, 8 * D, 9 * D, 17 * D, 18 * D]
    return [cache[..., a:b].unflatten(3, (16, (b - a) // 16)) for a, b in zip(at, at[1:])]


def take(part, slots):
    """What slots [n] hold of one of those views: [n, H, width]."""
    P = part.shape[2] * 16
    return part[slots // P, :, slots % P // 16, slots % 16]


def decode_scales(amax, bound=448.0):
    """fp32 decode scale of each amax, as the library derives it, in 64 bits."""
    enc = torch.clamp(torch.full_like(amax, 6.0 * bound) / amax, max=3.4028234663852886e38)
    enc = torch.where((amax > 0) & torch.isfinite(amax), enc, torch.ones_like(enc))
    return (torch.ones_like(enc) / enc).double()


def values(codes, scales, amax=None):
    """64-bit values [n, H, D] of codes and scale bytes; amax [1] or [H]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    grid = torch.cat([grid, -grid])
    q = grid[torch.stack([codes & 15, codes >> 4], dim=-1).long()].flatten(-2)
    d = scales.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1)
    v = q * d
    return v if amax is None else v * decode_scales(amax).reshape(1, -1, 1)


def rotate(x, positions, freq, layout, magnitude):
    """The rotation of x [T, H, D] in 64 bits; freq [R/2] angles a position."""
    x = x.double().clone()
    half = freq.numel()
    i = torch.arange(half, device=x.device)
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    t = (positions.double()[:, None] * freq.double())[:, None]
    u, v = x[..., a].clone(), x[..., b].clone()
    x[..., a] = magnitude * (u * t.cos() - v * t.sin())
    x[..., b] = magnitude * (v * t.cos() + u * t.sin())
    return x


def attention(q, k, v, n, *, scale, causal=True, window=0, sinks=None):
    """(out, log of the denominator, sum of weight * |v|, largest sum of |q||k|) in 64 bits of the n queries q [n, Hq, D]
    of one sequence over k, v [L, Hkv, D]."""
    L, H, D = k.shape
    G = q.shape[1] // H
    qq = q.double().reshape(n, H, G, D)
    x = torch.einsum("nhgd,lhd->hgnl", qq, k) * scale
    most = torch.einsum("nhgd,lhd->hgnl", qq.abs(), k.abs()).amax().item() * abs(scale) if L else 0.0
    pos = torch.arange(L - n, L, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)
    see = torch.ones(n, L, dtype=torch.bool, device=q.device)
    if causal:
        see &= j <= pos
    if window:
        see &= j > pos - window
    x = x.masked_fill(~see, -math.inf)
    if sinks is not None:
        x = torch.cat([x, sinks.double().reshape(H, G, 1, 1).expand(H, G, n, 1)], dim=3)
    lse = torch.logsumexp(x, dim=3) if x.shape[3] else torch.full((H, G, n), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.exp(x - lse.unsqueeze(3))
    w = torch.where(torch.isneginf(lse).unsqueeze(3), torch.zeros_like(w), w)[..., :L]
    out = torch.einsum("hgnl,lhd->nhgd", w, v).reshape(n, H * G, D)
    mass = torch.einsum("hgnl,lhd->nhgd", w, v.abs()).reshape(n, H * G, D)
    return out, lse.permute(2, 0, 1).reshape(n, H * G), mass, most


def tolerance(out, mass, most, biggest, L, D, x, o):
    """How far an output may be off.  delta: a logit's error, from D products summed in fp32 (each step off by at most
    2^-23 of the sum of magnitudes), the query's own rounding and five fp32 roundings; it moves a weight and the
    denominator by that much each.  A weight enters its product as f16 (2^-11 of itself, 2^-25 of the largest
    weight at least) or as two; exp2 and sums of L weights add 2^-22 and L / 16 + 64 roundings of 2^-23; the output is
    rounded once."""
    delta = (D + 8) * 2.0 ** -23 * most
    weight = 2.0 ** -11 if x == torch.bfloat16 else 2.0 ** -21
    floor = 2.0 ** -25 if x == torch.bfloat16 else 2.0 ** -36
    rounding = 2.0 ** -8 if o == torch.bfloat16 else 2.0 ** -24
    return rounding * out.abs() + (2 * delta + weight + 2.0 ** -20 + (L / 16 + 64) * 2.0 ** -23) * mass + L * floor * biggest + 1e-30
