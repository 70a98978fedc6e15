"""What an autograd function asks before it records a graph node under stream
capture.

A leaf has one gradient accumulator for all graphs that it is part of, bound to
the stream of the first.  A backward pass captured while an eager graph of the
same leaf lives would make the captured stream wait for that other stream, and
the process ends inside autograd's worker thread.  So each function here notes
its node and the leaves that it starts from, and refuses to be captured beside
an eager one: some at once, others, whose forward pass alone may be captured
there, in their backward pass.  Without gradients no node is recorded, and
nothing is refused.
"""
from __future__ import annotations

import threading
import weakref

import torch

from . import NVFP4Error

# (node, its leaves) of those recorded outside a capture, as weak references;
# what is dead is swept out when the list has doubled.  (With a weak set,
# whose entries are called at each node's end, noting took 6.4 us of a call's
# time on the host, so 4.2.)
_eager: list = []
_sweep_at = 256
_lock = threading.RLock()             # held by whoever adds to it or copies it


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


def _note(node, leaves) -> None:
    global _eager, _sweep_at
    entry = (weakref.ref(node), [weakref.ref(t) for t in leaves])
    with _lock:
        if len(_eager) >= _sweep_at:
            _eager = [e for e in _eager if e[0]() is not None]
            _sweep_at = max(256, 2 * len(_eager))
        _eager.append(entry)


def _lives_beside(leaves) -> bool:
    """Whether a node noted outside a capture still lives at one of them."""
    with _lock:
        entries = list(_eager)
    return any(node() is not None and any(t is leaf() for leaf in noted for t in leaves) for node, noted in entries)


def _refuse():
    raise NVFP4Error("a graph of this parameter or input, made outside the capture, still lives: delete its outputs "
                     "before the capture")


def refuse_beside(ctx) -> None:
    """For the backward pass of a LateLeafFunction."""
    if getattr(ctx, "beside", False) and _capturing():
        _refuse()


class LeafFunction(torch.autograd.Function):
    """An autograd function whose nodes are noted; under capture, apply raises
    NVFP4Error if a node noted outside a capture still lives at a leaf of the
    call's."""

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
            # (the accumulator stays the eager graph's, also where that is gone by
            # the backward pass: this graph holds it)
            node.beside = beside
        else:
            _note(node, leaves)
        return out


class LateLeafFunction(LeafFunction):
    """The same for a function whose forward pass may be captured beside an eager
    graph; its backward pass begins with refuse_beside."""

    late = True
