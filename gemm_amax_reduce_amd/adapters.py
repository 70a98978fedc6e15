"""Low-rank adapters of many requests beside a shared, frozen projection.

    y[t] = base[t] + scale_a B_a A_a x[t]    for the tokens t of a request, a its adapter

The shared projection's result comes from any of the linear layers, its 4-bit
weights read once for all requests; training reaches the adapters, x and the
base.  Every step runs in the HIP library; there is no CPU path.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import NVFP4Error, nvfp4_adapters, nvfp4_adapters_backward
from .capture import LeafFunction


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy of it, with unit column stride and rows that do not overlap."""
    return t.contiguous() if t.stride(1) != 1 or t.stride(0) < t.shape[1] else t


class AdaptersFunction(LeafFunction):
    """y [tokens, out] of x [tokens, in] and base [tokens, out] (or None)."""

    @staticmethod
    def forward(ctx, x, a, b, base, scale, offsets, index):
        x, a, b = _rows(x), a.contiguous(), b.contiguous()
        offsets, index = offsets.contiguous(), index.contiguous()
        y, u = nvfp4_adapters(x, a, b, offsets, index, scale, None if base is None else _rows(base))
        ctx.save_for_backward(x, u, a, b, scale, offsets, index)
        ctx.base_dtype = None if base is None else base.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, u, a, b, scale, offsets, index = ctx.saved_tensors
        dx = da = db = None
        if any(ctx.needs_input_grad[:3]):
            dx, da, db = nvfp4_adapters_backward(_rows(dy), x, u, a, b, offsets, index, scale, grad_dtype=a.dtype)
        dbase = dy.to(ctx.base_dtype) if ctx.needs_input_grad[3] else None
        return dx, da, db, dbase, None, None, None


class LowRankAdapters(torch.nn.Module):
    """A set of low-rank adapters of one projection [out, in]; B starts at
    zero, so that an adapter changes nothing before it is trained.

    The tokens come in segments, offsets[i] .. offsets[i + 1] - 1 those of
    request i with adapter index[i] (-1: none); both int32 or both int64 on
    the GPU.
    """

    def __init__(self, adapters: int, in_features: int, out_features: int, rank: int, scale: float = 1.0, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        self.a = torch.nn.Parameter(torch.empty((adapters, rank, in_features), device=device, dtype=dtype))
        self.b = torch.nn.Parameter(torch.zeros((adapters, out_features, rank), device=device, dtype=dtype))
        torch.nn.init.normal_(self.a, std=in_features ** -0.5)
        self.register_buffer("scale", torch.full((adapters,), scale, device=device, dtype=torch.float32))

    def _apply(self, fn, recurse=True):
        # the kernels take the scales in float32: they follow the module to a
        # device, but not to another type
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.scale.device)
        return self

    def forward(self, x, base, offsets, index):
        """base + the adapters' part of x [..., in]; base [..., out], or None
        for the part alone, in x's dtype."""
        features = self.a.shape[2]
        if x.dim() < 1 or x.shape[-1] != features:
            raise NVFP4Error(f"x must end in {features} features, got shape {tuple(x.shape)}")
        out = self.b.shape[1]
        if base is not None and tuple(base.shape) != (*x.shape[:-1], out):
            raise NVFP4Error(f"base must have shape {(*x.shape[:-1], out)}, got {tuple(base.shape)}")
        y = AdaptersFunction.apply(x.reshape(-1, features), self.a, self.b,
                                   None if base is None else base.reshape(-1, out), self.scale, offsets, index)
        return y.reshape(*x.shape[:-1], out)

    @torch.no_grad()
    def add(self, x, y, offsets, index):
        """Adds the adapters' part of x [tokens, in] to y [tokens, out], in place."""
        nvfp4_adapters(x, self.a.detach(), self.b.detach(), offsets, index, self.scale, base=y, out=y)
        return y
