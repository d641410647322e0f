"""Pre-norm feed-forward blocks on the block-scaled FP8 operators.

FP8BlockMLP  RMS norm of x + residual -> gate/up product -> SiLU * up -> down product
             (the dense layers and the shared expert of a DeepSeek-V3-shaped tower)
FP8BlockMoE  the same per routed expert, with the framework's routing, dispatch and
             combine

Weights are E4M3 codes with one float32 scale per 128x128 block, as such
checkpoints hold them; activations are quantized 1x128 by the operator that
produces them, so no bfloat16 copy of a product's input exists.  Every step is a
kernel of libfp4moe but the router's product, which stays a library call in
float32 (or the caller's, who then passes logits).
"""

from dataclasses import dataclass

import torch

from . import (fp8_block_grouped_gemm, fp8_block_linear, moe_combine, moe_permute, moe_route,
               rms_norm_fp8, swiglu_fp8)


def _check_x(x, dtypes, wanted):
    """Before anything is launched: the products return 16-bit types only, the combine
    bfloat16."""
    if x.dtype not in dtypes:
        raise ValueError(f"x is {x.dtype}; wanted {wanted}")


class FP8BlockMLP:
    """norm [H]; w13 codes [2I, H] (gate rows first), w13_scale [2I/128, H/128]; w2
    codes [H, I], w2_scale [H/128, I/128] (block counts rounded up)."""

    def __init__(self, norm, w13, w13_scale, w2, w2_scale, eps=1e-6):
        self.norm, self.eps = norm, eps
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale

    def forward(self, x, residual=None, stream=None):
        """x, residual [T, H] bfloat16 or float16, of norm's type -> (out [T, H] of x's
        type, the new residual or None)."""
        _check_x(x, (torch.bfloat16, torch.float16), "bfloat16 or float16")
        codes, scales, residual = rms_norm_fp8(x, self.norm, self.eps, residual, stream=stream)
        gate_up = fp8_block_linear(codes, scales, self.w13, self.w13_scale, out_dtype=x.dtype,
                                   stream=stream)
        codes, scales = swiglu_fp8(gate_up, stream=stream)
        return fp8_block_linear(codes, scales, self.w2, self.w2_scale, out_dtype=x.dtype,
                                stream=stream), residual


@dataclass
class FP8BlockMoEConfig:
    E: int                 # routed experts
    n_shared: int          # shared experts (ids E .. E+n_shared-1 in the weight tensors)
    n_group: int
    topk_group: int
    topk: int
    eps: float = 1e-6
    renormalize: bool = True
    routed_scale: float = 1.0


class FP8BlockMoE:
    """norm [H] bfloat16; w13 codes [E+n_shared, 2I, H], w2 codes [E+n_shared, H, I] with
    their block scales; router float32 [E, H] (None: the caller passes logits) and
    its correction bias float32 [E] (or None)."""

    def __init__(self, cfg: FP8BlockMoEConfig, norm, w13, w13_scale, w2, w2_scale, router=None,
                 bias=None):
        self.cfg, self.norm = cfg, norm
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale
        self.router, self.bias = router, bias

    def forward(self, x, residual=None, logits=None, keep=False):
        """x, residual bfloat16 [T, H], logits float32 [T, E] (None: the router's own)
        -> (out bfloat16 [T, H], the new residual or None), on the current stream.
        keep=True: a dict of every intermediate instead."""
        _check_x(x, (torch.bfloat16,), "bfloat16")
        c = self.cfg
        k = c.topk + c.n_shared
        y = torch.empty_like(x) if logits is None else None
        xq, xs, residual = rms_norm_fp8(x, self.norm, c.eps, residual, y=y)
        if logits is None:
            logits = torch.mm(y.float(), self.router.t())
        ids, weights = moe_route(logits, self.bias, c.n_group, c.topk_group, c.topk, c.renormalize,
                                 c.routed_scale)
        # entries of 16 rows while an expert has few, of 128 above (the products cut their
        # own tiles; long lists only cost their lookup)
        block_m = 16 if x.shape[0] * k <= 24 * (c.E + c.n_shared) else 128
        perm = moe_permute(ids, c.E, c.n_shared, block_m)
        gate_up = fp8_block_grouped_gemm(xq, xs, self.w13, self.w13_scale, perm, block_m,
                                         a_row_gather=perm["sorted_pairs"], gather_div=k)
        hq, hs = swiglu_fp8(gate_up, row_count=perm["expert_offsets"][c.E + c.n_shared:])
        down = fp8_block_grouped_gemm(hq, hs, self.w2, self.w2_scale, perm, block_m)
        out = moe_combine(down, perm["pair_pos"], weights, c.topk, c.n_shared)
        if keep:
            return dict(xq=xq, xs=xs, residual=residual, topk_ids=ids, topk_w=weights, perm=perm,
                        block_m=block_m, gate_up=gate_up, hq=hq, hs=hs, down=down, out=out)
        return out, residual
