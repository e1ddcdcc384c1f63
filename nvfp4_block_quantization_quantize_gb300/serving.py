"""Layers of a served model on frozen NVFP4 weights, made of the serving
operators: the norm that adds the residual stream and quantizes, the product of
a few tokens, the products grouped by expert.

The weights are quantized once with the library (1x16 blocks, one global amax a
weight or expert).  Nothing here reads a device value on the host, so a step
of fixed shapes can be captured in a CUDA graph.  No gradient is taken: the results
do not require one, whatever the inputs do.
"""
from __future__ import annotations

import torch

from . import (nvfp4_grouped_mm, nvfp4_grouped_scales_to_mma, nvfp4_mv, nvfp4_quantize, nvfp4_rmsnorm)

MV_ROWS = 16                                    # the most rows nvfp4_mv takes


def _quantize_experts(w: torch.Tensor) -> dict:
    """[E, N, K] -> codes, scales in the product's layout and one amax an expert."""
    E, N, K = w.shape
    q = [nvfp4_quantize(w[e].contiguous(), gamax_mode="tensor") for e in range(E)]
    return {"codes": torch.stack([t["codes"] for t in q]),
            "scales": torch.stack([t["scales"] for t in q]),
            "gamax": torch.cat([t["gamax"] for t in q])}


class FP4Projection:
    """norm(x + hidden) W^T for a weight [N, K], K a multiple of 64.

    activations: "mxfp8" (8 bits; nvfp4_mv, 16 rows at a time), "nvfp4" (4 bits; the FP4
    tensor cores through nvfp4_grouped_mm with one group), or "auto": "mxfp8" for the 16
    rows nvfp4_mv takes at once, "nvfp4" above.  With "auto" the precision of a token's
    result goes by the number of rows it comes with; the other two give it the same at
    any.  [14336, 4096] in a graph: 1 row 10 us, 16 rows 31 us in 8 bits, 64 rows 14 us in 4."""

    def __init__(self, weight: torch.Tensor, norm_weight: torch.Tensor, eps: float = 1e-6, activations: str = "auto"):
        if activations not in ("auto", "mxfp8", "nvfp4"):
            raise ValueError(f"FP4Projection: activations {activations!r}; expected auto, mxfp8 or nvfp4")
        q = _quantize_experts(weight.unsqueeze(0))
        self.norm_weight, self.eps, self.activations = norm_weight, eps, activations
        self.codes, self.scales, self.gamax = q["codes"], q["scales"], q["gamax"]
        self.scales_mma = nvfp4_grouped_scales_to_mma(self.scales)

    def _mv(self, codes, x_scales, out_dtype):
        return nvfp4_mv(codes, self.codes[0], self.scales[0], x_scales=x_scales, gamax=self.gamax, out_dtype=out_dtype)

    def __call__(self, x: torch.Tensor, hidden: torch.Tensor, out_dtype="bf16"):
        """(product [M, N], new hidden [M, K])."""
        M = x.shape[0]
        if self.activations == "mxfp8" or (self.activations == "auto" and M <= MV_ROWS):
            n = nvfp4_rmsnorm(x, self.norm_weight, hidden=hidden, eps=self.eps)
            if M <= MV_ROWS:
                return self._mv(n["codes"], n["scales"], out_dtype), n["hidden"]
            parts = zip(n["codes"].split(MV_ROWS), n["scales"].split(MV_ROWS))
            return torch.cat([self._mv(c, s, out_dtype) for c, s in parts]), n["hidden"]
        n = nvfp4_rmsnorm(x, self.norm_weight, hidden=hidden, eps=self.eps, format="nvfp4", gamax_mode="row")
        offsets = torch.zeros(2, dtype=torch.int64, device=x.device)
        offsets[1:].fill_(M)
        y = nvfp4_grouped_mm(n["codes"], n["scales"], offsets, self.codes, self.scales_mma, gamax_a=n["gamax"],
                             gamax_b=self.gamax, out_dtype=out_dtype)
        return y, n["hidden"]


class FP4Experts:
    """A feed-forward layer of E experts, each token through its top_k by a router:
    sum over them of p * (silu(n Wg^T) * (n Wu^T)) Wd^T with n = norm(x + hidden) and
    p the softmax over the chosen experts' router logits.

    gate_up [E, 2 F, D] (gate rows first), down [E, D, F]; router [E, D] stays as it is;
    D and F multiples of 64."""

    def __init__(self, norm_weight, router, gate_up, down, top_k: int, eps: float = 1e-6):
        if gate_up.dim() != 3 or down.dim() != 3 or gate_up.shape[1] != 2 * down.shape[2]:
            raise ValueError("FP4Experts: gate_up [E, 2 F, D] and down [E, D, F]")
        if not 1 <= top_k <= router.shape[0] == gate_up.shape[0] == down.shape[0]:
            raise ValueError("FP4Experts: router [E, D] and 1 <= top_k <= E")
        self.norm_weight, self.router, self.top_k, self.eps = norm_weight, router, top_k, eps
        self.gate_up, self.down = _quantize_experts(gate_up), _quantize_experts(down)
        for w in (self.gate_up, self.down):
            w["scales"] = nvfp4_grouped_scales_to_mma(w["scales"])

    def route(self, n: torch.Tensor):
        """(chosen experts [M, top_k], their weights [M, top_k]); the lowest index wins a tie."""
        logits = n.float() @ self.router.float().t()
        top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
        return idx[:, :self.top_k], torch.softmax(top[:, :self.top_k], dim=1)

    def __call__(self, x: torch.Tensor, hidden: torch.Tensor):
        """(layer output [M, D] in x's dtype, new hidden [M, D])."""
        M, E, k = x.shape[0], self.router.shape[0], self.top_k
        n = nvfp4_rmsnorm(x, self.norm_weight, hidden=hidden, eps=self.eps, format="nvfp4", gamax_mode="row",
                          want_out=True)
        idx, p = self.route(n["out"])
        experts = idx.reshape(-1)
        order = torch.argsort(experts, stable=True)           # rows sorted by expert
        counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
        counts.scatter_add_(0, experts + 1, torch.ones_like(experts))
        offsets = counts.cumsum(0)
        rows = order // k
        h = nvfp4_grouped_mm(n["codes"][rows], n["scales"][rows], offsets, self.gate_up["codes"],
                             self.gate_up["scales"], gamax_a=n["gamax"][rows], gamax_b=self.gate_up["gamax"],
                             out_dtype="f32")
        gate, up = h.chunk(2, dim=1)
        q = nvfp4_quantize(torch.nn.functional.silu(gate) * up, gamax_mode="row")
        y = nvfp4_grouped_mm(q["codes"], q["scales"], offsets, self.down["codes"], self.down["scales"],
                             gamax_a=q["gamax"], gamax_b=self.down["gamax"], out_dtype="f32")
        # back to token order, then one sum in a fixed order
        back = torch.empty_like(order)
        back[order] = torch.arange(M * k, device=x.device)
        out = (y[back].view(M, k, y.shape[1]) * p.unsqueeze(2)).sum(dim=1)
        return out.to(x.dtype), n["hidden"]
