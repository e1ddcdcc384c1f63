"""The phases of a rotation against arithmetic of many digits: a far position multiplies what they are off by."""
import pytest

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
mp = pytest.importorskip("mpmath")


def check(phases, freq):
    """Each phase is the nearest whole number of 2^-64 turns (a tie or a last digit may go either way: one unit)."""
    assert len(phases) == len(freq)
    for p, f in zip(phases, freq):
        turns = f / (2 * mp.pi) * mp.mpf(2) ** 64
        d = (int(p) - int(mp.nint(turns))) % (1 << 64)
        assert min(d, (1 << 64) - d) <= 1


@pytest.fixture(autouse=True)
def digits():
    with mp.workdps(120):
        yield


@pytest.mark.parametrize("rot,base", [(2, 1e4), (64, 1e4), (128, 1e6), (128, 500000.0), (96, 1e4), (512, 1e7), (16, 0.1)])
def test_phases_of_a_base(rot, base):
    check(nv.nvfp4_rope_phases(rot, base), [mp.mpf(base) ** (-mp.mpf(2 * i) / rot) for i in range(rot // 2)])


@pytest.mark.parametrize("factor", [1.0, 3.0, 8.0, 31.7])
def test_phases_of_longer_contexts(factor):
    rot, base = 128, 1e6
    f = [mp.mpf(base) ** (-mp.mpf(2 * i) / rot) for i in range(64)]
    check(nv.nvfp4_rope_phases(rot, base, factor=factor), [x / mp.mpf(factor) for x in f])
    raised = mp.mpf(base) * mp.mpf(factor) ** (mp.mpf(64) / 63)
    check(nv.nvfp4_rope_phases(rot, base, factor=factor, method="ntk"), [raised ** (-mp.mpf(2 * i) / rot) for i in range(64)])

    def pair(turns):
        return 64 * mp.log(4096 / (turns * 2 * mp.pi)) / mp.log(base)

    low, high = int(mp.floor(pair(32))), int(mp.ceil(pair(1)))
    keep = [1 - min(max(mp.mpf(i - low) / (high - low), 0), 1) for i in range(64)]
    check(nv.nvfp4_rope_phases(rot, base, factor=factor, method="yarn", original=4096),
          [x * k + x / mp.mpf(factor) * (1 - k) for x, k in zip(f, keep)])


def test_phases_of_given_frequencies():
    """Angles a position of more than a turn: whole turns drop out exactly, of large ones too."""
    freq = [1.0, 0.1, 9.0, 1e-9, 6.283185307179586, 12345.678, 1e15, 1e40]
    check(nv.nvfp4_rope_phases(16, inv_freq=freq), [mp.mpf(f) for f in freq])
    check(nv.nvfp4_rope_phases(16, inv_freq=freq, factor=7.0), [mp.mpf(f) / 7 for f in freq])
