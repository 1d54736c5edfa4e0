"""A gated expert layer on one GPU, from the router's logits to the combined
hidden states, through the calls of ``binding``:

    route -> moe_few                                            few tokens
    route -> layout_dispatch (FP8) -> group_gemm_swiglu_fp8
          -> group_gemm_fp8 -> combine                          the others

Both paths cast x and the activated hidden rows to FP8, x with quotients that
differ in the last bit (a code may differ by one where a value lies between
two); the second also rounds every expert's output row to bf16 before the
weighted sum.
"""
import torch

from . import binding


class ExpertLayer:
    """Experts held as e4m3 codes with one float32 scale per 128 x 128 block:
    ``w13_q`` [E, 2I, H] (gate rows, then up rows), ``w13_scale`` [E, 2I/128,
    H/128], ``w2_q`` [E, H, I], ``w2_scale`` [E, H/128, I/128].  ``k`` experts
    per token; the keyword arguments are ``binding.route``'s."""

    def __init__(self, w13_q, w13_scale, w2_q, w2_scale, k, *, bias=None, groups=1, groups_per_token=None,
                 scoring="softmax", renormalize=True, scale=1.0):
        if (w13_q.dim() != 3 or w2_q.dim() != 3 or w13_q.shape[1] != 2 * w2_q.shape[2]
                or tuple(w2_q.shape[:2]) != (w13_q.shape[0], w13_q.shape[2])):
            raise ValueError("w13_q must be [E, 2I, H] and w2_q [E, H, I]")
        self.w13_q, self.w13_scale, self.w2_q, self.w2_scale = w13_q, w13_scale, w2_q, w2_scale
        self.E, self.k = w13_q.shape[0], k
        self.routing = dict(bias=bias, groups=groups, groups_per_token=groups_per_token, scoring=scoring,
                            renormalize=renormalize, scale=scale)
        # the device status word of every call made here, on whatever streams
        # (binding.status_read)
        self.status = torch.zeros(1, dtype=torch.int32, device=w13_q.device)

    def __call__(self, x, logits, out=None):
        """x [T, H] bf16 and the router's logits [T, E] to out [T, H] bf16, on
        the current stream."""
        if logits.shape != (x.shape[0], self.E):
            raise ValueError("logits must be [T, E]")
        idx, w = binding.route(logits, self.k, status=self.status, **self.routing)
        return self.experts(x, idx, w, out)

    def few(self, T):
        """Whether T tokens go through ``moe_few``.  It takes widths up to
        ``MOE_FEW_MAX_WIDTH`` and weights on 32 bytes, the longer path any
        width and weights on 16.  Where both take the call: ``moe_few`` saves the five launches of
        the longer path about 10 us, but reads an expert's weights at the full
        rate only for one or two tokens each.  Measured, few against long, in
        us: H 2048, I 1024, E 128, k 8: 16 / 28 (1 token), 103 / 104 (16), 154 /
        140 (48); H 7168, I 2048, E 64, k 8: 69 / 77 (1), 429 / 410 (16), 584 /
        436 (64); H 1024, I 512, E 8, k 2, whose weights are 13 MB: 10 / 21 (1),
        21 / 23 (64)."""
        if T > binding.MOE_FEW_MAX_TOKENS or max(self.w13_q.shape[2], self.w2_q.shape[2]) > binding.MOE_FEW_MAX_WIDTH:
            return False
        if self.w13_q.data_ptr() % 32 or self.w2_q.data_ptr() % 32:
            return False
        return T * self.k <= 2 * self.E or self.w13_q.numel() + self.w2_q.numel() <= 32 << 20

    def experts(self, x, topk_idx, topk_w, out=None):
        """The same for a route that is already at hand."""
        if x.dim() != 2 or x.shape[1] != self.w13_q.shape[2]:
            raise ValueError("x must be [T, H]")
        if topk_idx.dim() != 2 or topk_idx.shape[0] != x.shape[0] or topk_w.shape != topk_idx.shape:
            raise ValueError("topk_idx and topk_w must be [T, k]")
        if out is not None and out.shape != x.shape:
            raise ValueError("out must be [T, H]")
        if self.few(x.shape[0]):
            return binding.moe_few(x, topk_idx, topk_w, self.w13_q, self.w13_scale, self.w2_q, self.w2_scale,
                                   out=out, status=self.status)
        # the layout zeroes the word that it is given, so it has one of its own
        lay, q, s = binding.layout_dispatch(x, topk_idx, self.E, with_rank_counts=False, fp8=True)
        at = (lay.expert_counts, lay.expert_offsets)
        h, hs = binding.group_gemm_swiglu_fp8(q, s, self.w13_q, self.w13_scale, *at, status=self.status)
        y = binding.group_gemm_fp8(h, hs, self.w2_q, self.w2_scale, *at, status=self.status)
        out = binding.combine(y, topk_w, lay.dst_row, out=out, status=self.status)
        binding.status_merge(lay.status, self.status)
        return out
