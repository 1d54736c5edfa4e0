"""A gated expert layer in BF16 with its gradients, on one GPU, through the
calls of ``binding``:

    forward   layout_dispatch -> group_gemm_swiglu -> group_gemm -> combine
              (shared experts: linear, SwiGLU -> linear, the rest as residual)
    backward  combine_backward -> group_gemm_wgrad, group_gemm_swiglu_dgrad
              -> group_gemm_wgrad, group_gemm_dgrad -> combine
              (shared experts: linear_backward twice)

Between two calls everything is held in bf16: the dispatched rows, the
pre-activations, the activated rows, the experts' outputs, and their gradients.
Gradients of weights are float32 or bf16, and may be added to what is there.
"""
from collections import namedtuple

import torch

from . import binding

# what the backward pass needs of a forward pass
Saved = namedtuple("Saved", "x topk_w layout rows z h y shared_z shared_h")
ExpertGrads = namedtuple("ExpertGrads", "dx dtopk_w dw13 dw2 dshared13 dshared2")


class TrainableExpertLayer:
    """Experts ``w13`` [E, 2I, H] (gate rows, then up rows) and ``w2`` [E, H, I]
    in bf16, and optionally one shared expert that every token takes,
    ``shared13`` [2S, H] and ``shared2`` [H, S].  The tensors are used as they
    are at each call: an optimizer may write to them in between."""

    def __init__(self, w13, w2, shared13=None, shared2=None):
        if w13.dim() != 3 or w2.dim() != 3 or tuple(w13.shape) != (w2.shape[0], 2 * w2.shape[2], w2.shape[1]):
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        if (shared13 is None) != (shared2 is None):
            raise ValueError("a shared expert has both shared13 and shared2")
        if shared13 is not None and (shared2.dim() != 2 or shared2.shape[0] != w2.shape[1]
                                     or tuple(shared13.shape) != (2 * shared2.shape[1], shared2.shape[0])):
            raise ValueError("shared13 must be [2S, H] and shared2 [H, S]")
        self.w13, self.w2, self.shared13, self.shared2 = w13, w2, shared13, shared2
        # the device status word of every call made here, on whatever streams
        # (binding.status_read)
        self.status = torch.zeros(1, dtype=torch.int32, device=w13.device)

    def forward(self, x, topk_idx, topk_w):
        """x [T, H] bf16 and its route [T, k] to (out [T, H] bf16, Saved)."""
        if x.dim() != 2 or x.shape[1] != self.w2.shape[1]:
            raise ValueError("x must be [T, H]")
        if topk_idx.dim() != 2 or topk_idx.shape[0] != x.shape[0] or topk_w.shape != topk_idx.shape:
            raise ValueError("topk_idx and topk_w must be [T, k]")
        E, inner = self.w2.shape[0], self.w2.shape[2]
        # the layout zeroes the word that it is given, so it has one of its own
        lay, rows = binding.layout_dispatch(x, topk_idx, E, with_rank_counts=False)
        at = (lay.expert_counts, lay.expert_offsets)
        z = torch.empty(rows.shape[0], 2 * inner, dtype=torch.bfloat16, device=x.device)
        h = binding.group_gemm_swiglu(rows, self.w13, *at, z=z, status=self.status)
        y = binding.group_gemm(h, self.w2, *at, status=self.status)
        out = binding.combine(y, topk_w, lay.dst_row, status=self.status)
        binding.status_merge(lay.status, self.status)
        sz = sh = None
        if self.shared13 is not None:
            sz = torch.empty(x.shape[0], self.shared13.shape[0], dtype=torch.bfloat16, device=x.device)
            sh = binding.linear(x, self.shared13, activation="swiglu", z=sz, status=self.status)
            out = binding.linear(sh, self.shared2, residual=out, out=out, status=self.status)
        return out, Saved(x, topk_w, lay, rows, z, h, y, sz, sh)

    def backward(self, dout, saved, grads=None, dtype=torch.float32):
        """Gradients of a forward pass from ``dout`` [T, H] bf16: of x (bf16), of
        topk_w (float32) and of the weights, in ``dtype``.  ``grads``, an earlier
        call's result, has its gradients of weights added to and returned."""
        if dout.shape != saved.x.shape:
            raise ValueError("dout must be [T, H]")
        lay = saved.layout
        at = (lay.expert_counts, lay.expert_offsets)
        kept = grads if grads is not None else ExpertGrads(*[None] * 6)
        dy, dtopk_w = binding.combine_backward(dout, saved.y, saved.topk_w, lay.dst_row, status=self.status)
        dw2 = binding.group_gemm_wgrad(dy, saved.h, *at, dw=kept.dw2, add=kept.dw2, dtype=dtype, status=self.status)
        dz = binding.group_gemm_swiglu_dgrad(dy, self.w2, saved.z, *at, status=self.status)
        dw13 = binding.group_gemm_wgrad(dz, saved.rows, *at, dw=kept.dw13, add=kept.dw13, dtype=dtype,
                                        status=self.status)
        drows = binding.group_gemm_dgrad(dz, self.w13, *at, status=self.status)
        dx = binding.combine(drows, torch.ones_like(saved.topk_w), lay.dst_row, status=self.status)
        ds13 = ds2 = None
        if self.shared13 is not None:
            second = binding.linear_backward(dout, saved.shared_h, self.shared2, dw=kept.dshared2, add=kept.dshared2,
                                             dtype=dtype, with_dbias=False, status=self.status)
            first = binding.linear_backward(second.dx, saved.x, self.shared13, saved.shared_z, "swiglu",
                                            dw=kept.dshared13, add=kept.dshared13, dtype=dtype, with_dbias=False,
                                            status=self.status)
            dx, ds13, ds2 = dx.add_(first.dx), first.dw, second.dw
        return ExpertGrads(dx, dtopk_w, dw13, dw2, ds13, ds2)
