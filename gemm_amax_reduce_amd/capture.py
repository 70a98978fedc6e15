"""What an autograd function asks before it records a graph node under stream
capture.

A leaf has one gradient accumulator for all graphs that it is part of, bound to
the stream of the first.  A backward pass captured while an eager graph of the
same leaf lives would make the captured stream wait for that other stream, and
the process ends inside autograd's worker thread.  So each function here notes
its node and the leaves that it starts from, and refuses to be captured beside
an eager one.  Without gradients no node is recorded, and nothing is refused.
"""
from __future__ import annotations

import weakref

import torch

from . import NVFP4Error

_eager = weakref.WeakSet()            # the nodes recorded outside a capture that still live


def _capturing() -> bool:
    return torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()


def _leaves(args):
    """The leaves among the tensors (or that they are views of) that need a gradient."""
    tensors = [t._base if t._is_view() else t for t in args if isinstance(t, torch.Tensor) and t.requires_grad]
    return [t for t in tensors if t.is_leaf and t.requires_grad]


class LeafFunction(torch.autograd.Function):
    """An autograd function whose nodes are noted; under capture, apply raises
    NVFP4Error if a node noted outside a capture still lives at a leaf of the
    call's."""

    @classmethod
    def apply(cls, *args):
        # (inside forward gradients are always off, and ctx.needs_input_grad tells
        # only what the inputs say)
        leaves = _leaves(args) if torch.is_grad_enabled() else []
        if not leaves:
            return super().apply(*args)
        if _capturing():
            for node in list(_eager):
                noted = [leaf() for leaf in node.leaves]
                if any(t is leaf for t in leaves for leaf in noted):
                    raise NVFP4Error("a graph of this parameter or input, made outside the capture, still lives: "
                                     "delete its outputs before the capture")
            return super().apply(*args)
        out = super().apply(*args)
        node = (out[0] if isinstance(out, tuple) else out).grad_fn
        node.leaves = [weakref.ref(t) for t in leaves]
        _eager.add(node)
        return out
