"""The serving layers (serving.py): their products against float64 products of the
operators' own quantized values, and the whole against the unquantized layer."""
import numpy as np
import pytest
import torch

import oracle
from parity_helpers import to_np

pytestmark = pytest.mark.gpu

nv = pytest.importorskip("nvfp4_block_quantization_quantize_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.build()
    nv.load_library()


def tensor(rng, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * scale).cuda().to(dtype)


def nvfp4_values(q, gamax):
    """float64 values of nvfp4_quantize's outputs with one amax a row."""
    rows, K = q["codes"].shape[0], q["codes"].shape[1] * 2
    v = oracle.dequantize(to_np(q["codes"]), to_np(q["scales"]), rows, K, out_dtype=oracle.F32).astype(np.float64)
    return v * np.array([oracle.global_scales(float(g), 448.0)[1] for g in gamax], np.float64)[:, None]


@pytest.mark.parametrize("M", [1, 7, 16, 17, 100])
def test_projection(M):
    from nvfp4_block_quantization_quantize_gb300.serving import FP4Projection
    rng = np.random.default_rng(M)
    N, K = 200, 512
    w, nw = tensor(rng, N, K, scale=0.02), tensor(rng, K, dtype=torch.float32)
    x, r = tensor(rng, M, K), tensor(rng, M, K)
    layer = FP4Projection(w, nw)
    y, h = layer(x, r, out_dtype="f32")
    q = nv.nvfp4_quantize(w, gamax_mode="tensor")
    wv = nvfp4_values(q, np.repeat(to_np(q["gamax"]), N))
    if M <= 16:
        n = nv.nvfp4_rmsnorm(x, nw, hidden=r)
        e = torch.from_numpy(to_np(n["codes"])).view(torch.float8_e4m3fn).double().numpy()
        nvv = e * np.repeat(2.0 ** (to_np(n["scales"]).astype(np.float64) - 127), 32, axis=1)
    else:
        n = nv.nvfp4_rmsnorm(x, nw, hidden=r, format="nvfp4", gamax_mode="row")
        nvv = nvfp4_values(n, to_np(n["gamax"]))
    assert torch.equal(h, n["hidden"]) and torch.equal(h, (x.float() + r.float()).to(x.dtype))
    assert (np.abs(to_np(y) - nvv @ wv.T) <= (np.abs(nvv) @ np.abs(wv).T) * 2.0 ** -17).all()


def experts_layer(rng, E, D, F, k):
    from nvfp4_block_quantization_quantize_gb300.serving import FP4Experts
    w = dict(norm_weight=torch.ones(D, device="cuda"), router=tensor(rng, E, D, scale=0.2),
             gate_up=tensor(rng, E, 2 * F, D, scale=D ** -0.5), down=tensor(rng, E, D, F, scale=F ** -0.5))
    return FP4Experts(**w, top_k=k), w


@pytest.mark.parametrize("M,E,D,F,k", [(1, 8, 256, 192, 2), (33, 8, 256, 192, 2), (300, 5, 192, 256, 1),
                                       (64, 6, 128, 64, 6)])
def test_experts_against_the_unquantized_layer(M, E, D, F, k):
    """The two quantized activations are each about a tenth of their norm off (e2m1 has steps of
    a third to a half of a value), and so is each of the two weights: four such errors are
    0.2 of the output's norm, and 0.35 leaves room for small samples."""
    rng = np.random.default_rng(M + E)
    layer, w = experts_layer(rng, E, D, F, k)
    x, r = tensor(rng, M, D), tensor(rng, M, D)
    out, h = layer(x, r)
    assert out.shape == (M, D) and out.dtype == x.dtype
    s = x.double() + r.double()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6)
    got = nv.nvfp4_rmsnorm(x, w["norm_weight"], hidden=r, want_out=True)["out"]
    idx, p = layer.route(got)
    ref = torch.zeros(M, D, dtype=torch.float64, device="cuda")
    for m in range(M):
        for e, q in zip(idx[m].tolist(), p[m].tolist()):
            g, u = (w["gate_up"][e].double() @ n[m]).chunk(2)
            ref[m] += q * (w["down"][e].double() @ (torch.nn.functional.silu(g) * u))
    assert float((out.double() - ref).norm() / ref.norm()) < 0.35


def test_experts_token_by_token_and_in_a_graph():
    """A batch gives each token what it gets alone (the same products, other tiles: within one
    bf16 step of the largest output), and a captured step what an eager one gives."""
    rng = np.random.default_rng(4)
    layer, _ = experts_layer(rng, 8, 256, 192, 2)
    x, r = tensor(rng, 24, 256), tensor(rng, 24, 256)
    out, _ = layer(x, r)
    for m in (0, 11, 23):
        one, _ = layer(x[m:m + 1], r[m:m + 1])
        assert float((one - out[m:m + 1]).abs().max()) <= 2.0 ** -7 * float(out[m].abs().max())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x, r)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _ = layer(x, r)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, out)


def test_layers_refuse():
    from nvfp4_block_quantization_quantize_gb300.serving import FP4Experts
    z = torch.zeros
    with pytest.raises(ValueError):
        FP4Experts(z(64), z(4, 64), z(4, 128, 64), z(4, 64, 128), 2)
    with pytest.raises(ValueError):
        FP4Experts(z(64), z(4, 64), z(4, 128, 64), z(4, 64, 64), 5)
