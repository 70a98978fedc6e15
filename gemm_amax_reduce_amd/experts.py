"""The layers of a mixture of experts in NVFP4: rows grouped by expert, each
group against its own 4-bit weights, activations and gradients as they are.

    forward  y  = x W_e^T     W (axis 1)
    backward dx = dy W_e      W (axis 0)
             dW_e = dy^T x    over the rows of group e

The experts' weights are quantized as one tensor, one maximum for all of them;
with gradients needed, both of its layouts come from a dual-layout call.  Every
quantization and product runs in the HIP library; there is no CPU path.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (NVFP4Error, NVFP4Tensor, nvfp4_dequantize, nvfp4_grouped_matmul, nvfp4_grouped_wgrad,
               nvfp4_quantize, nvfp4_quantize_dual)
from .capture import LateLeafFunction, LeafFunction, refuse_beside
from .head import RMSNorm, _matrix


def group_by_expert(choice: torch.Tensor, experts: int):
    """(order, offsets) of a router's choice [tokens, top] of experts: the
    pairs token * top + place sorted by expert, and where each expert's begin.
    Rows of the grouped layers are x[order // top]; choices outside
    [0, experts) come last and belong to no group."""
    flat = choice.reshape(-1)
    flat = torch.where((flat >= 0) & (flat < experts), flat, experts)
    chosen, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(chosen, torch.arange(experts + 1, device=choice.device, dtype=chosen.dtype))
    return order, offsets


def weighted_sum(parts, share):
    """The sum over a token's experts of share [tokens, top] times parts
    [tokens, top, features], in parts' type; formed in float32, rounded once."""
    return (parts * share[:, :, None]).sum(1).to(parts.dtype)


class NVFP4ExpertsFunction(LeafFunction):
    """y [rows, out] of grouped rows x [rows, in], W [experts, out, in]; rows
    of no group are zeros."""

    @staticmethod
    def forward(ctx, x, weight, offsets):
        x, offsets = _matrix(x), offsets.contiguous()
        stack = weight.contiguous().reshape(-1, weight.shape[2])
        ctx.qw0 = None
        if ctx.needs_input_grad[0]:
            qw, ctx.qw0 = nvfp4_quantize_dual(stack)
        else:
            qw = nvfp4_quantize(stack, axis=1)
        ctx.save_for_backward(x, offsets)
        ctx.w_dtype = weight.dtype
        return nvfp4_grouped_matmul(qw, x, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, offsets = ctx.saved_tensors
        dy = _matrix(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = nvfp4_grouped_matmul(ctx.qw0, dy, offsets, transposed=True)
        if ctx.needs_input_grad[1]:
            dw = nvfp4_grouped_wgrad(dy, x, offsets, ctx.w_dtype)
        return dx, dw, None


class PackedExpertsFunction(LateLeafFunction):
    """The same with weights that are packed already, and frozen: x alone gets a
    gradient, from their decoded values quantized along the other axis, in
    every backward pass (a stack kept in both layouts would take twice the
    memory that packing is for)."""

    @staticmethod
    def forward(ctx, x, packed, offsets):
        offsets = offsets.contiguous()
        ctx.save_for_backward(offsets, packed.codes, packed.scales, packed.meta)
        ctx.outer, ctx.k = packed.outer, packed.k
        return nvfp4_grouped_matmul(packed, _matrix(x), offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        refuse_beside(ctx)
        offsets, codes, scales, meta = ctx.saved_tensors
        stack = nvfp4_dequantize(NVFP4Tensor(codes, scales, meta, ctx.outer, ctx.k))
        return nvfp4_grouped_matmul(nvfp4_quantize(stack, axis=0), _matrix(dy), offsets, transposed=True), None, None


class NVFP4Experts(torch.nn.Module):
    """Bias-free linear layers of several experts on rows grouped by expert,
    weights [experts, out, in] in NVFP4 (see group_by_expert)."""

    def __init__(self, experts: int, in_features: int, out_features: int, device=None, dtype=torch.bfloat16):
        super().__init__()
        if in_features % 16 or out_features % 16:
            raise NVFP4Error("in_features and out_features must be multiples of 16")
        self.weight = torch.nn.Parameter(torch.empty((experts, out_features, in_features), device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, x, offsets, packed: NVFP4Tensor | None = None):
        """x [rows, in] -> [rows, out].  With `packed` (from pack), those
        weights are used, and x alone gets a gradient."""
        if x.dim() != 2 or x.shape[1] != self.weight.shape[2]:
            raise NVFP4Error(f"x must be [rows, {self.weight.shape[2]}], got shape {tuple(x.shape)}")
        if offsets.dim() != 1 or offsets.shape[0] != self.weight.shape[0] + 1:
            raise NVFP4Error(f"offsets must have {self.weight.shape[0] + 1} entries, got shape {tuple(offsets.shape)}")
        if packed is not None:
            return PackedExpertsFunction.apply(x, packed, offsets)
        return NVFP4ExpertsFunction.apply(x, self.weight, offsets)

    @torch.no_grad()
    def pack(self) -> NVFP4Tensor:
        """The weights as they are now, in NVFP4."""
        return nvfp4_quantize(self.weight.detach().contiguous().reshape(-1, self.weight.shape[2]), axis=1)


class NVFP4ExpertBlock(torch.nn.Module):
    """The feed-forward half of a layer with a mixture of experts:

        h = x + residual,  n = rms_norm(h)
        y[t] = sum over t's `top` experts of share * down_e(silu(gate_e(n)) up_e(n))

    with the shares a softmax over the chosen experts' scores.  Returns (y, h),
    the next block's x and residual.
    """

    def __init__(self, experts: int, top: int, features: int, hidden: int, eps: float = 1e-6, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        if not 1 <= top <= experts:
            raise NVFP4Error(f"top must lie between 1 and {experts}, got {top}")
        self.top = top
        self.norm = RMSNorm(features, eps, device, dtype)
        self.router = torch.nn.Parameter(torch.empty((experts, features), device=device, dtype=dtype))
        torch.nn.init.normal_(self.router, std=0.02)
        self.up = NVFP4Experts(experts, features, 2 * hidden, device, dtype)       # gate and up together
        self.down = NVFP4Experts(experts, hidden, features, device, dtype)

    def forward(self, x, residual, packed=None):
        """x, residual [..., features] -> (y, h).  packed: from pack, for
        answers, or training around frozen experts."""
        lead, experts = x.shape[:-1], self.router.shape[0]
        n, h = self.norm(x, residual)
        rows = n.reshape(-1, n.shape[-1])
        scores = torch.nn.functional.linear(rows.float(), self.router.float())
        best, choice = torch.topk(scores, self.top, dim=1)
        share = torch.softmax(best, 1)
        order, offsets = group_by_expert(choice, experts)
        both = self.up(rows[order // self.top], offsets, packed and packed[0])
        gate, up = both.chunk(2, 1)
        out = self.down(torch.nn.functional.silu(gate) * up, offsets, packed and packed[1])
        back = torch.empty_like(order).scatter_(0, order, torch.arange(order.shape[0], device=order.device))
        parts = out[back].reshape(rows.shape[0], self.top, -1)
        y = weighted_sum(parts, share)
        return y.reshape(*lead, -1), h

    @torch.no_grad()
    def pack(self):
        """Both stacks of experts as they are now, in NVFP4."""
        return self.up.pack(), self.down.pack()
