"""The end of a model around a 4-bit linear layer: final norm, NVFP4 head, and
the loss on a teacher's best logits, for training; norm and matrix-vector
product with the head's 4-bit weights, for answering a few tokens.

    training   h = layer_norm(x),  logits = NVFP4Linear(h),
               loss_t = tau^2 KL(teacher's top logits || logits_t)
    answering  h = layer_norm(x),  logits = h W^T with W in NVFP4, h as it is

Distillation against the model's own 16-bit form is how a model brought to 4
bits is trained further; the norm in front of a 4-bit layer also knows the
maximum that the layer's quantizer needs.  Every step runs in the HIP library;
there is no CPU path.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (NVFP4Error, NVFP4Tensor, nvfp4_distill_topk, nvfp4_distill_topk_backward, nvfp4_gemm_ws,
               nvfp4_layer_norm, nvfp4_layer_norm_backward, nvfp4_matvec, nvfp4_quantize, nvfp4_quantize_amax)
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


class LayerNormFunction(torch.autograd.Function):
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
        x, mean, rstd, weight = ctx.saved_tensors
        grad_dtype = weight.dtype if weight is not None else ctx.bias_dtype or torch.float32
        dx, dw, db = nvfp4_layer_norm_backward(dy.contiguous(), x, mean, rstd, weight, grad_dtype=grad_dtype)
        return dx, dw if weight is not None else None, db if ctx.has_bias else None, None


class DistillTopKFunction(torch.autograd.Function):
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


class NVFP4Head(torch.nn.Module):
    """Final norm and NVFP4 output projection.

    forward / loss train it (the token count a multiple of 16); pack lays the
    weights out in NVFP4 once, and answer gives the logits of any number of
    tokens from them without gradients.
    """

    def __init__(self, features: int, vocab: int, eps: float = 1e-5, seed: int = 0, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        self.norm = LayerNorm(features, eps, device, dtype)
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
    def answer(self, x, packed: NVFP4Tensor, out_dtype=torch.float32):
        """Logits [..., vocab] of x [..., features] from packed weights.  Up
        to MATVEC_TOKENS tokens meet them unquantized; more (a prompt) are
        quantized with the maximum that the norm hands over and multiplied by
        the NVFP4 GEMM."""
        lead = x.shape[:-1]
        rows = _matrix(x.reshape(-1, x.shape[-1]))
        w, b, eps = self.norm.weight.detach(), self.norm.bias.detach(), self.norm.eps
        if rows.shape[0] <= MATVEC_TOKENS:
            h, _, _ = nvfp4_layer_norm(rows, w, b, eps=eps)
            y = nvfp4_matvec(packed, h, out_dtype=out_dtype)
        else:
            h, _, _, amax = nvfp4_layer_norm(rows, w, b, eps=eps, amax=True)
            y = nvfp4_gemm_ws(nvfp4_quantize_amax(h, amax, axis=1), packed, out_dtype)
        return y.reshape(*lead, packed.outer)
