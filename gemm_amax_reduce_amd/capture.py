"""What an autograd function asks before it records a graph node under stream
capture.

A leaf has one gradient accumulator for all graphs that it is part of, bound to
the stream of the first.  A backward pass captured while an eager graph of the
same leaf lives would make the captured stream wait for that other stream, and
the process ends inside autograd's worker thread.  So each function here notes
its node and the leaves that it starts from, and refuses to be captured beside
an eager one.
"""
from __future__ import annotations

import weakref

import torch

from . import NVFP4Error

_eager = weakref.WeakSet()            # the nodes recorded outside a capture that still live


def note_leaves(ctx, *tensors) -> None:
    """Notes the graph node `ctx` with the leaves among `tensors` (or that they
    are views of) that need a gradient; under capture, raises NVFP4Error if a
    node noted outside a capture still lives at one of them."""
    if not any(ctx.needs_input_grad):
        return
    leaves = [t._base if t._is_view() else t for t in tensors if t is not None]
    leaves = [t for t in leaves if t.is_leaf and t.requires_grad]
    if not leaves:
        return
    if not (torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()):
        ctx.leaves = [weakref.ref(t) for t in leaves]
        _eager.add(ctx)
        return
    for node in list(_eager):
        noted = [leaf() for leaf in node.leaves]
        if any(t is leaf for t in leaves for leaf in noted):
            raise NVFP4Error("a graph of this parameter or input, made outside the capture, still lives: delete its "
                             "outputs before the capture")
