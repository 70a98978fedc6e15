"""What an autograd function asks before it records a graph node under stream
capture.

A leaf has one gradient accumulator for all graphs that it is part of, bound to
the stream of the first.  A backward pass captured while an eager graph of the
same leaf lives makes that other stream part of the capture, which the default
stream cannot be: the process ends inside autograd's worker thread.  So each
function here notes its node and the leaves that it starts from, and refuses to
be captured beside an eager one of the default stream: some at once, others,
whose forward pass alone may be captured there, in their backward pass.  Without
gradients no node is recorded, and nothing is refused.
"""
from __future__ import annotations

import threading
import weakref

import torch

from . import NVFP4Error, _current_handle

# (node, its leaves) of the nodes that the default stream recorded, or that hold
# an accumulator of its, by weak references; what is dead is swept out when the
# list has doubled, or is looked through.  (A weak set, whose entries are called
# at each node's end, made noting 2 us longer on the host.)
_noted: list = []
_sweep_at = 256
_lock = threading.RLock()             # held by whoever adds to it or looks through it


def _capturing() -> bool:
    return torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()


def _leaves(args) -> list:
    """The leaves among the tensors (or that they are views of) that need a gradient."""
    found = []
    for t in args:
        if isinstance(t, torch.Tensor) and t.requires_grad:
            if t._is_view():
                t = t._base
            if t.is_leaf and t.requires_grad:
                found.append(t)
    return found


def _default_stream(device) -> bool:
    return device.type == "cuda" and _current_handle(device) == 0


def _sweep() -> None:
    global _noted, _sweep_at
    _noted = [e for e in _noted if e[0]() is not None]
    _sweep_at = max(256, 2 * len(_noted))


def _note(node, leaves) -> None:
    entry = (weakref.ref(node), [weakref.ref(t) for t in leaves])
    with _lock:
        if len(_noted) >= _sweep_at:
            _sweep()
        _noted.append(entry)


def _lives_beside(leaves) -> bool:
    """Whether a noted node still lives at one of them."""
    with _lock:
        _sweep()
        entries = list(_noted)
    return any(node() is not None and any(t is leaf() for leaf in noted for t in leaves) for node, noted in entries)


def _refuse():
    raise NVFP4Error("a graph of this parameter or input, made on the default stream, still lives: delete its outputs "
                     "before the capture")


def refuse_beside(ctx) -> None:
    """For the backward pass of a LateLeafFunction."""
    if getattr(ctx, "beside", False) and _capturing():
        _refuse()


class LeafFunction(torch.autograd.Function):
    """An autograd function whose nodes are noted; under capture, apply raises
    NVFP4Error if a node that the default stream recorded still lives at a leaf of
    the call's."""

    late = False

    @classmethod
    def apply(cls, *args):
        # (inside forward gradients are always off, and ctx.needs_input_grad tells
        # only what the inputs say)
        leaves = _leaves(args) if torch.is_grad_enabled() else []
        if not leaves:
            return super().apply(*args)
        capturing = _capturing()
        beside = capturing and _lives_beside(leaves)
        if beside and not cls.late:
            _refuse()
        out = super().apply(*args)
        node = (out[0] if isinstance(out, tuple) else out).grad_fn
        if capturing:
            node.beside = beside
        # (beside another node a node holds the same accumulator, also when that one
        # is gone)
        if beside if capturing else _default_stream(leaves[0].device) or _lives_beside(leaves):
            _note(node, leaves)
        return out


class LateLeafFunction(LeafFunction):
    """The same for a function whose forward pass may be captured beside an eager
    graph; its backward pass begins with refuse_beside."""

    late = True
