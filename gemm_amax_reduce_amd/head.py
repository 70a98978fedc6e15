"""The end of a model around a 4-bit linear layer: final norm, NVFP4 head, and
the loss on a teacher's best logits, for training; norm and matrix-vector
product with the head's 4-bit weights, for answering a few tokens.

    training   h = layer_norm(x),  logits = NVFP4Linear(h),
               loss_t = tau^2 KL(teacher's top logits || logits_t)
    answering  h = layer_norm(x),  logits = h W^T with W in NVFP4, h as it is

The norm may be an RMS norm instead, and answers may pass through the low-rank
adapter of the request that each token belongs to.

Distillation against the model's own 16-bit form is how a model brought to 4
bits is trained further; the norm in front of a 4-bit layer also knows the
maximum that the layer's quantizer needs.  Every step runs in the HIP library;
there is no CPU path.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (NVFP4Error, NVFP4Tensor, nvfp4_distill_topk, nvfp4_distill_topk_backward, nvfp4_gemm_ws,
               nvfp4_layer_norm, nvfp4_layer_norm_backward, nvfp4_matvec, nvfp4_quantize, nvfp4_quantize_amax,
               nvfp4_rms_norm, nvfp4_rms_norm_backward)
from .adapters import LowRankAdapters
from .capture import LateLeafFunction, LeafFunction, refuse_beside
from .linear import NVFP4Linear

# Up to this many rows are answered by the matrix-vector form, which reads
# the weights once for every 16.
MATVEC_TOKENS = 16


def _matrix(x: torch.Tensor) -> torch.Tensor:
    """x, or a copy of it, as the kernels read a matrix: unit column stride,
    rows that do not overlap (a transposed, expanded or windowed x is copied)."""
    if x.dim() == 2 and (x.stride(1) != 1 or x.stride(0) < x.shape[1]):
        return x.contiguous()
    return x


class LayerNormFunction(LateLeafFunction):
    """y = layer norm of the rows of x [tokens, features], in x's dtype."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps: float):
        x = _matrix(x)
        y, mean, rstd = nvfp4_layer_norm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.has_bias = bias is not None
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        refuse_beside(ctx)
        x, mean, rstd, weight = ctx.saved_tensors
        grad_dtype = weight.dtype if weight is not None else ctx.bias_dtype or torch.float32
        dx, dw, db = nvfp4_layer_norm_backward(dy.contiguous(), x, mean, rstd, weight, grad_dtype=grad_dtype)
        return dx, dw if weight is not None else None, db if ctx.has_bias else None, None


class RMSNormFunction(LeafFunction):
    """y = RMS norm of the rows of x [tokens, features] in x's dtype, or with a
    residual (y, h) of h = x + residual, in the residual's dtype."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps: float):
        x = _matrix(x)
        ctx.x_dtype, ctx.has_residual = x.dtype, residual is not None
        if residual is None:
            y, rstd = nvfp4_rms_norm(x, weight, eps=eps)
            ctx.save_for_backward(x, rstd, weight)
            return y
        y, rstd, h = nvfp4_rms_norm(x, weight, _matrix(residual), eps=eps)
        ctx.save_for_backward(h, rstd, weight)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, rstd, weight = ctx.saved_tensors
        grad_dtype = weight.dtype if weight is not None else torch.float32
        r_dtype = h.dtype
        if ctx.x_dtype == torch.float32 and r_dtype != torch.float32:
            # the kernel writes dx in h's type: beside a bf16 stream a float32 x
            # would get a gradient of 8 bits
            h, dh = h.float(), None if dh is None else dh.float()
        dx, dw = nvfp4_rms_norm_backward(dy.contiguous(), h, rstd, weight, None if dh is None else dh.contiguous(),
                                         grad_dtype=grad_dtype)
        return (dx.to(ctx.x_dtype), dx.to(r_dtype) if ctx.has_residual else None, dw if weight is not None else None,
                None)


class DistillTopKFunction(LateLeafFunction):
    """Per-token distillation losses [tokens] of logits [tokens, vocab]; the
    gradient takes any upstream gradient of the losses."""

    @staticmethod
    def forward(ctx, logits, indices, teacher, temperature: float):
        logits, indices, teacher = _matrix(logits), indices.contiguous(), teacher.contiguous()
        loss, lse = nvfp4_distill_topk(logits, indices, teacher, temperature=temperature)
        ctx.save_for_backward(logits, indices, teacher, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        refuse_beside(ctx)
        logits, indices, teacher, lse = ctx.saved_tensors
        dz = nvfp4_distill_topk_backward(logits, indices, teacher, lse, dloss.contiguous(),
                                         temperature=ctx.temperature)
        return dz, None, None, None


def distill_topk_loss(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                      weight: torch.Tensor | None = None, temperature: float = 1.0) -> torch.Tensor:
    """The sum of the tokens' losses times `weight` (f32 [tokens]), or their
    mean without one; differentiable in the logits."""
    loss = DistillTopKFunction.apply(logits, indices, teacher, temperature)
    return loss.mean() if weight is None else torch.dot(loss, weight)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, weight and bias learned."""

    def __init__(self, features: int, eps: float = 1e-5, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype))
        self.eps = eps

    def forward(self, x):
        if x.dim() < 1 or x.shape[-1] != self.weight.shape[0]:
            raise NVFP4Error(f"x must end in {self.weight.shape[0]} features, got shape {tuple(x.shape)}")
        y = LayerNormFunction.apply(x.reshape(-1, x.shape[-1]), self.weight, self.bias, self.eps)
        return y.reshape(x.shape)


class RMSNorm(torch.nn.Module):
    """RMS norm over the last dimension, weight learned; with a residual, of
    the sum x + residual, which is returned too: (y, sum)."""

    def __init__(self, features: int, eps: float = 1e-6, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.eps = eps

    def forward(self, x, residual=None):
        features = self.weight.shape[0]
        if x.dim() < 1 or x.shape[-1] != features:
            raise NVFP4Error(f"x must end in {features} features, got shape {tuple(x.shape)}")
        if residual is None:
            return RMSNormFunction.apply(x.reshape(-1, features), None, self.weight, self.eps).reshape(x.shape)
        if residual.shape != x.shape:
            raise NVFP4Error(f"residual must have x's shape {tuple(x.shape)}, got {tuple(residual.shape)}")
        y, h = RMSNormFunction.apply(x.reshape(-1, features), residual.reshape(-1, features), self.weight, self.eps)
        return y.reshape(x.shape), h.reshape(x.shape)


class NVFP4Head(torch.nn.Module):
    """Final norm ("layer" or "rms") and NVFP4 output projection.

    forward / loss train it (the token count a multiple of 16); pack lays the
    weights out in NVFP4 once, and answer gives the logits of any number of
    tokens from them without gradients.
    """

    def __init__(self, features: int, vocab: int, eps: float = 1e-5, seed: int = 0, device=None,
                 dtype=torch.bfloat16, norm: str = "layer"):
        super().__init__()
        if norm not in ("layer", "rms"):
            raise NVFP4Error(f"norm must be 'layer' or 'rms', got {norm!r}")
        self.norm = (LayerNorm if norm == "layer" else RMSNorm)(features, eps, device, dtype)
        self.proj = NVFP4Linear(features, vocab, seed=seed, device=device, dtype=dtype)

    def forward(self, x):
        return self.proj(self.norm(x))

    def loss(self, x, indices, teacher, weight=None, temperature: float = 1.0):
        """The distillation loss of x [..., features] against the teacher's
        lists [tokens, top]."""
        logits = self.forward(x)
        return distill_topk_loss(logits.reshape(-1, logits.shape[-1]), indices, teacher, weight, temperature)

    @torch.no_grad()
    def pack(self) -> NVFP4Tensor:
        """The projection's weights as they are now, in NVFP4."""
        return nvfp4_quantize(self.proj.weight.detach().contiguous(), axis=1)

    @torch.no_grad()
    def answer(self, x, packed: NVFP4Tensor, out_dtype=torch.float32, adapters: LowRankAdapters | None = None,
               offsets=None, index=None):
        """Logits [..., vocab] of x [..., features] from packed weights.  Up
        to MATVEC_TOKENS tokens meet them unquantized; more (a prompt) are
        quantized with the maximum that the norm hands over (an RMS norm's
        output is read for it) and multiplied by the NVFP4 GEMM.

        With `adapters`, tokens offsets[i] .. offsets[i + 1] - 1 get adapter
        index[i]'s part added in place (index -1: none)."""
        if adapters is not None and (offsets is None or index is None):
            raise NVFP4Error("adapters need offsets and index")
        lead = x.shape[:-1]
        rows = _matrix(x.reshape(-1, x.shape[-1]))
        w, eps = self.norm.weight.detach(), self.norm.eps
        few = rows.shape[0] <= MATVEC_TOKENS
        amax = None
        if isinstance(self.norm, RMSNorm):
            h, _ = nvfp4_rms_norm(rows, w, eps=eps)
        elif few:
            h, _, _ = nvfp4_layer_norm(rows, w, self.norm.bias.detach(), eps=eps)
        else:
            h, _, _, amax = nvfp4_layer_norm(rows, w, self.norm.bias.detach(), eps=eps, amax=True)
        if few:
            y = nvfp4_matvec(packed, h, out_dtype=out_dtype)
        else:
            q = nvfp4_quantize(h, axis=1) if amax is None else nvfp4_quantize_amax(h, amax, axis=1)
            y = nvfp4_gemm_ws(q, packed, out_dtype)
        if adapters is not None:
            adapters.add(h, y, offsets, index)
        return y.reshape(*lead, packed.outer)
