"""What the attention's kernels leave when a wait runs out.  A copy of their sources is built whose waits poll a few times
instead of millions of times, so that they give up while their copies and products are on their way: nothing hangs or
faults, and every row is NaN or as it should be."""
import concurrent.futures as cf
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from test_gpu_cache import Paged, gen, normal

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")
pytestmark = pytest.mark.gpu

build = nv.build.__globals__                               # the build module's names
CHANGED = ["nvfp4_attend.cu", "nvfp4_attend_many.cu"]


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """Libraries by the number of times a wait polls."""
    nv.build()
    nv.load_library()
    top = tmp_path_factory.mktemp("waits")

    def make(limit):
        src = top / str(limit) / "package" / "csrc"        # (next to include/, as the sources name it)
        shutil.copytree(build["CSRC"], src)
        shutil.copytree(build["INCLUDE"], top / str(limit) / "include")
        found = 0
        for f in os.listdir(src):
            text = (src / f).read_text()
            new = text.replace("kWaitLimit = 1L << 22;", f"kWaitLimit = {limit};")
            found += new != text
            (src / f).write_text(new.replace("mbarrier.try_wait.parity", "mbarrier.test_wait.parity"))
        assert found == 1
        out = [str(top / f"{limit}_{f}.o") for f in CHANGED]
        for f, o in zip(CHANGED, out):
            subprocess.run([build["nvcc"](), *build["ARCH"], *build["FLAGS"], "-c", str(src / f), "-o", o], check=True, capture_output=True)
        rest = [os.path.join(build["BUILD_DIR"], f.replace(".cu", ".o")) for f in build["SOURCES"] if f not in CHANGED]
        lib = str(top / f"hasty{limit}.so")
        subprocess.run([build["nvcc"](), *build["ARCH"], "-shared", "-o", lib, *out, *rest, "-cudart", "static"], check=True, capture_output=True)
        return ctypes.CDLL(lib)

    limits = (0, 20, 300)
    with cf.ThreadPoolExecutor() as ex:
        return dict(zip(limits, ex.map(make, limits)))


def call(lib, c, q, off, **opt):
    """nvfp4_cache_attention of `lib` into outputs and a workspace that hold a pattern: (out, lse)."""
    B, T, Hq, D = len(c.lens), q.shape[0], q.shape[1], q.shape[2]
    dt = nv.F32 if q.dtype == torch.float32 else nv.BF16
    i64, f32, P = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    ws = lib.nvfp4_cache_attention_workspace
    ws.restype, ws.argtypes = i64, nv.load_library().nvfp4_cache_attention_workspace.argtypes
    fn = lib.nvfp4_cache_attention
    fn.restype, fn.argtypes = ctypes.c_int32, nv.load_library().nvfp4_cache_attention.argtypes
    need = ws(T, Hq, c.H, D, B, c.pages.shape[1], c.P, dt, int(off is not None))
    work = torch.full((max(need, 16),), 0x3F, dtype=torch.uint8, device="cuda")      # (floats of 0.747)
    out, lse = torch.full(q.shape, 7.0, device="cuda"), torch.full((T, Hq), 7.0, device="cuda")
    p = lambda t: P(0 if t is None else t.data_ptr())      # noqa: E731
    mode = nv.GAMAX_NONE if c.ka is None else nv.GAMAX_ROW_GIVEN
    rc = fn(p(q), T, Hq, Hq * D, dt, p(c.cache), c.cache.shape[0], c.P, c.H, D, p(c.pages), B, c.pages.shape[1], p(c.lengths), p(off),
            mode, p(c.ka), mode, p(c.va), f32(448.0), f32(D ** -0.5), 1, 0, P(0), p(out), nv.F32, p(lse), p(work), need,
            P(torch.cuda.current_stream().cuda_stream))
    assert rc == nv.OK
    torch.cuda.synchronize()
    return out, lse


CASES = [
    # lens, queries of each (None: one, no offsets), Hq, H, D, x
    ([200, 0, 5000, 17], None, 8, 2, 128, "bf16"),         # cut groups and whole ones
    ([30, 900], None, 4, 1, 64, "f32"),                    # a group a CTA
    ([9000], None, 6, 2, 256, "bf16"),
    ([700, 900], [700, 300], 8, 2, 128, "bf16"),           # the tensor-memory kernel
    ([6000, 12, 2000], [300, 5, 257], 8, 2, 64, "bf16"),   # both kernels
    ([20000], [130], 4, 1, 128, "bf16"),                   # one group, cut between all CTAs
]


@pytest.mark.parametrize("limit", [0, 20, 300])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_waits_that_run_out(hasty, i, limit):
    lens, counts, Hq, H, D, x = CASES[i]
    c = Paged(i, lens, H, D, 16, "head")
    n = [1] * len(lens) if counts is None else counts
    q = (2.0 * normal(gen(i), sum(n) + 3 * (counts is not None), Hq, D)).to({"bf16": torch.bfloat16, "f32": torch.float32}[x])
    off = None if counts is None else torch.tensor([0] + counts, device="cuda").cumsum(0)
    want, want_lse = call(nv.load_library(), c, q, off)
    c.check(q, n, want, want_lse)
    got, lse = call(hasty[limit], c, q, off)
    lost = got.isnan().any(dim=2)
    assert torch.equal(got[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
    assert got[lost].isnan().all() and lse[lost].isnan().all()
    assert not lost[sum(n):].any()                         # rows of no sequence stay as they were
    if limit == 0:
        keys = torch.tensor([length > 0 for length, m in zip(lens, n) for _ in range(m)], device="cuda")
        assert lost[:sum(n)][keys].float().mean() > 0.5
    again, again_lse = call(nv.load_library(), c, q, off)
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse)
