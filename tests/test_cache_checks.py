"""Refusals of the cache operators, checked without a GPU: the C ABI's argument checks run on the host before any CUDA
call, the binding's before the library is called.  And the frequencies of a rotation, which are made on the host."""
import ctypes
import math

import pytest
import torch

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")

NAN, INF = float("nan"), float("inf")


def at(i):
    """A pointer that is never used as an address: every call below is refused or empty."""
    return ctypes.c_void_p(0x1000000 * (i + 1))


ODD = ctypes.c_void_p(0x7000002)
A8 = ctypes.c_void_p(0x7000008)


@pytest.fixture(scope="module")
def lib():
    nv.build()
    return nv.load_library()


def rope(lib, q=at(0), k=at(1), v=None, T=4, Hq=4, Hkv=2, D=64, qs=256, ks=128, vs=0, dtype=1, qw=None, kw=None, wdt=1,
         eps=1e-6, pos=at(2), phases=at(3), rot=64, layout=0, magnitude=1.0, q_out=at(4), k_out=at(5), cache=None, pages=0,
         P=16, slots=None, km=0, kg=None, vm=0, vg=None, bound=448.0):
    return lib.nvfp4_qk_norm_rope(q, k, v, T, Hq, Hkv, D, qs, ks, vs, dtype, qw, kw, wdt, eps, pos, phases, rot, layout,
                                  magnitude, q_out, k_out, cache, pages, P, slots, km, kg, vm, vg, bound, None)


CACHED = dict(v=at(6), vs=128, cache=at(7), pages=4, slots=at(8), k_out=None)
ROPE_BAD = {
    "D not a multiple of 16": dict(D=72),
    "D zero": dict(D=0),
    "D too large": dict(D=528),
    "negative T": dict(T=-1),
    "too many heads": dict(Hq=1 << 15),
    "bad dtype": dict(dtype=2),
    "bad weight dtype": dict(wdt=7),
    "eps negative": dict(eps=-1.0),
    "eps NaN": dict(eps=NAN),
    "magnitude infinite": dict(magnitude=INF),
    "magnitude NaN": dict(magnitude=NAN),
    "bad layout": dict(layout=2),
    "rotary_dim past D": dict(rot=80),
    "rotary_dim odd": dict(rot=24),
    "rotary_dim negative": dict(rot=-16),
    "one weight": dict(qw=at(9)),
    "positions missing": dict(pos=None),
    "phases missing": dict(phases=None),
    "positions misaligned": dict(pos=ODD),
    "q NULL": dict(q=None),
    "k NULL": dict(k=None),
    "q_out NULL": dict(q_out=None),
    "neither k_out nor cache": dict(k_out=None),
    "q misaligned": dict(q=A8),
    "stride of half a piece": dict(qs=260),
    "stride negative": dict(ks=-128),
    "q_out is q": dict(q_out=at(0)),
    "q_out in k": dict(q_out=ctypes.c_void_p(0x2000000 + 512)),
    "k_out is q_out": dict(k_out=at(4)),
    "cache without v": dict(CACHED, v=None),
    "cache without slots": dict(CACHED, slots=None),
    "k_out with a cache": dict(CACHED, k_out=at(5)),
    "a cache of other heads": dict(CACHED, D=80),
    "pages of no tile": dict(CACHED, P=24),
    "half layout, blocks cut": dict(CACHED, rot=48),
    "cache is q": dict(CACHED, cache=at(0)),
    "bad mode": dict(CACHED, km=1, kg=at(9)),
    "gamax NULL": dict(CACHED, vm=3),
    "gamax misaligned": dict(CACHED, vm=3, vg=ODD),
    "bound zero": dict(CACHED, bound=0.0),
    "cache too large": dict(CACHED, pages=(1 << 30) - 1, P=(1 << 29), Hkv=1 << 14),
}


@pytest.mark.parametrize("case", sorted(ROPE_BAD))
def test_rope_rejects(lib, case):
    assert rope(lib, **ROPE_BAD[case]) == nv.EINVAL
    assert lib.nvfp4_last_error() != b""


def write(lib, k=at(0), v=at(1), T=4, Hkv=2, D=64, ks=128, vs=128, dtype=1, cache=at(2), pages=4, P=16, slots=at(3), km=0,
          kg=None, vm=0, vg=None, bound=448.0):
    return lib.nvfp4_cache_write(k, v, T, Hkv, D, ks, vs, dtype, cache, pages, P, slots, km, kg, vm, vg, bound, None)


def read(lib, cache=at(2), pages=4, P=16, Hkv=2, D=64, slots=at(3), T=4, km=0, kg=None, vm=0, vg=None, bound=448.0,
         k=at(0), v=at(1), odt=1):
    return lib.nvfp4_cache_read(cache, pages, P, Hkv, D, slots, T, km, kg, vm, vg, bound, k, v, odt, None)


@pytest.mark.parametrize("call,bad", [(c, b) for c, extra in (
    (write, [dict(dtype=3), dict(ks=4), dict(vs=-8), dict(k=None), dict(v=None), dict(cache=at(0)), dict(k=A8)]),
    (read, [dict(odt=2), dict(k=None, v=None), dict(k=at(2)), dict(k=at(1)), dict(k=A8)])) for b in extra + [
        dict(D=80), dict(D=512), dict(P=0), dict(P=40), dict(pages=-1), dict(T=-1), dict(Hkv=1 << 15), dict(T=1 << 30),
        dict(slots=None), dict(slots=ODD), dict(cache=None), dict(cache=A8), dict(km=2), dict(km=4), dict(vm=9), dict(bound=NAN),
        dict(bound=449.0)]])
def test_write_and_read_reject(lib, call, bad):
    assert call(lib, **bad) == nv.EINVAL
    assert lib.nvfp4_last_error() != b""


def attend(lib, q=at(0), T=4, Hq=4, qs=256, dtype=1, cache=at(1), pages=4, P=16, Hkv=2, D=64, table=at(2), B=4, width=2,
           lengths=at(3), offsets=None, km=0, kg=None, vm=0, vg=None, bound=448.0, scale=0.1, causal=1, window=0, sinks=None,
           out=at(4), odt=1, lse=None, ws=None, ws_bytes=0):
    return lib.nvfp4_cache_attention(q, T, Hq, qs, dtype, cache, pages, P, Hkv, D, table, B, width, lengths, offsets, km, kg,
                                     vm, vg, bound, scale, causal, window, sinks, out, odt, lse, ws, ws_bytes, None)


ATTEND_BAD = {
    "heads not whole": dict(Hq=3, qs=192),
    "no KV heads": dict(Hkv=0),
    "D": dict(D=96),
    "T is not B": dict(T=3),
    "bad dtype": dict(dtype=2),
    "bad out dtype": dict(odt=5),
    "negative T": dict(T=-1, B=-1),
    "negative B": dict(B=-1, offsets=at(5)),
    "too many rows": dict(T=1 << 29, B=1 << 29, Hq=8),
    "width too large": dict(width=1 << 27),
    "page_size": dict(P=8),
    "causal": dict(causal=2),
    "window": dict(window=-1),
    "scale NaN": dict(scale=NAN),
    "scale infinite": dict(scale=INF),
    "stride": dict(qs=260),
    "q NULL": dict(q=None),
    "cache NULL": dict(cache=None),
    "table NULL": dict(table=None),
    "table misaligned": dict(table=ODD),
    "lengths NULL": dict(lengths=None),
    "lengths misaligned": dict(lengths=ODD),
    "offsets misaligned": dict(offsets=ODD),
    "sinks misaligned": dict(sinks=ODD),
    "out NULL": dict(out=None),
    "lse misaligned": dict(lse=ODD),
    "out is q": dict(out=at(0)),
    "out in the cache": dict(out=ctypes.c_void_p(0x2000000 + 1152)),
    "lse is out": dict(lse=at(4)),
    "lse is lengths": dict(lse=at(3)),
    "mode": dict(vm=1, vg=at(6)),
    "gamax NULL": dict(km=4),
    "bound": dict(bound=-1.0),
    "no workspace": dict(width=1000, pages=1000),
    "a workspace too small": dict(width=1000, pages=1000, ws=at(40), ws_bytes=16),
}


@pytest.mark.parametrize("case", sorted(ATTEND_BAD))
def test_attention_rejects(lib, case):
    assert attend(lib, **ATTEND_BAD[case]) == nv.EINVAL
    assert lib.nvfp4_last_error() != b""


def test_workspace_that_is_an_input_is_refused(lib):
    need = lib.nvfp4_cache_attention_workspace(4, 4, 2, 64, 4, 1000, 16, 1, 0)
    assert need > 0
    assert attend(lib, width=1000, pages=1000, ws=at(0), ws_bytes=need) == nv.EINVAL
    assert attend(lib, width=1000, pages=1000, ws=A8, ws_bytes=need) == nv.EINVAL


def test_workspace_sizes(lib):
    """None for what no call may cut, more where offsets allow a sequence many rows, 0 for sizes a call refuses."""
    ws = lib.nvfp4_cache_attention_workspace
    assert ws(1, 4, 2, 64, 1, 32, 16, 1, 0) == 0            # (two groups: no more than run at once anywhere)
    few = ws(4, 8, 1, 128, 4, 1000, 16, 1, 0)
    assert 0 < few < ws(100, 8, 1, 128, 4, 1000, 16, 1, 1)
    assert ws(1, 8, 1, 128, 1, 32, 16, 1, 0) == 0 < ws(100, 8, 1, 128, 1, 32, 16, 1, 1)
    assert ws(10000, 8, 1, 128, 10000, 32, 16, 1, 0) > 0    # more groups than run at once
    for bad in ((-1, 4, 2, 64, 4, 32, 16, 1, 0), (4, 3, 2, 64, 4, 32, 16, 1, 0), (4, 4, 2, 96, 4, 32, 16, 1, 0),
                (4, 4, 2, 64, 4, 1 << 40, 16, 1, 0), (4, 4, 2, 64, 4, 32, 0, 1, 0)):
        assert ws(*bad) == 0


def test_empty_calls_enqueue_nothing(lib):
    assert rope(lib, T=0, q=None, k=None, q_out=None, k_out=None, pos=None, phases=None) == nv.OK
    assert rope(lib, Hq=0, Hkv=0, q=None, k=None, q_out=None, k_out=None) == nv.OK
    assert write(lib, T=0, k=None, v=None, slots=None, cache=None) == nv.OK
    assert write(lib, pages=0, cache=None) == nv.OK
    assert read(lib, T=0, k=None, v=None, slots=None, cache=None) == nv.OK
    assert attend(lib, T=0, B=0, q=None, out=None, lengths=None, table=None, cache=None) == nv.OK
    assert attend(lib, T=0, B=3, offsets=at(5), q=None, out=None) == nv.OK
    assert attend(lib, Hq=0, q=None, out=None) == nv.OK


def test_binding_refuses_host_tensors():
    x, u, i = torch.zeros(2, 4, 64), torch.zeros(1, 4, 1, 18 * 64, dtype=torch.uint8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_qk_norm_rope(x, x, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_cache_write(u, x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_cache_read(u, i)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_cache_attention(x, u, torch.zeros(2, 1, dtype=torch.int32), i)
    for bad in ((4, 24, 2, 64), (4, 16, 2, 80), (-1, 16, 2, 64), (4, 0, 2, 64)):
        with pytest.raises(ValueError, match="nvfp4_cache_empty"):
            nv.nvfp4_cache_empty(*bad, device="cpu")
    assert nv.nvfp4_cache_empty(3, 48, 2, 128, device="cpu").shape == (3, 2, 3, 18 * 128)


# ---- frequencies ----------------------------------------------------------------------------------
def turns(phases):
    """Angles a position of the phases, as floats."""
    return [(int(p) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for p in phases]


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (512, 500000.0)])
def test_frequencies(rot, base):
    """One rounding of the power, one of the division, one to whole 2^-64 turns: 2^-51 of the angle is ample."""
    p = nv.nvfp4_rope_phases(rot, base)
    assert p.dtype == torch.int64 and p.shape == (rot // 2,)
    for i, t in enumerate(turns(p)):
        want = base ** (-2 * i / rot)
        assert abs(t - want) <= 2.0 ** -51 * want + 2 * math.pi * 2.0 ** -64
    for i, t in enumerate(turns(nv.nvfp4_rope_phases(rot, base, factor=4.0))):
        assert abs(t - base ** (-2 * i / rot) / 4) <= 2.0 ** -51


def test_longer_contexts():
    rot, base, f = 64, 10000.0, 8.0
    plain, ntk = turns(nv.nvfp4_rope_phases(rot, base)), turns(nv.nvfp4_rope_phases(rot, base, factor=f, method="ntk"))
    assert ntk[0] == plain[0]                              # the fastest pair stays, the slowest is divided by the factor
    assert abs(ntk[-1] - plain[-1] / f) <= 2.0 ** -40 * ntk[-1] + 2.0 ** -60
    assert all(a <= b for a, b in zip(ntk, plain))
    yarn = turns(nv.nvfp4_rope_phases(rot, base, factor=f, method="yarn", original=4096))
    for i, (y, p) in enumerate(zip(yarn, plain)):
        made = 4096 * p / (2 * math.pi)                    # turns in the original context
        assert p / f * (1 - 1e-12) <= y <= p * (1 + 1e-12)
        if made > 48:
            assert y == p
        if made < 0.6:
            assert abs(y - p / f) <= 1e-12 * p
    given = turns(nv.nvfp4_rope_phases(4, inv_freq=[0.5, 9.0]))
    assert abs(given[0] - 0.5) < 1e-15 and abs(given[1] - (9.0 - 2 * math.pi)) < 1e-14      # whole turns drop out


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=3), dict(factor=0.5), dict(factor=NAN), dict(factor=INF),
                                dict(base=0.0), dict(base=-1.0), dict(method="other"), dict(method="yarn"),
                                dict(method="yarn", original=0), dict(method="yarn", original=4096, beta_fast=1.0),
                                dict(inv_freq=[1.0]), dict(inv_freq=[1.0, INF]), dict(inv_freq=[1.0, 0.5], method="ntk", factor=2.0),
                                dict(method="yarn", original=4096, base=1.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError, match="nvfp4_rope_phases"):
        nv.nvfp4_rope_phases(**{"rotary_dim": 4, **kw})
