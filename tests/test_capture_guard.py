"""The guard of captured autograd functions, on the CPU: a stand-in function, and
a flag in the place of the stream's state."""
import pytest
import torch

import gemm_amax_reduce_amd as nv
from gemm_amax_reduce_amd import capture


class Twice(capture.LeafFunction):
    @staticmethod
    def forward(ctx, x, w):
        return x * w

    @staticmethod
    def backward(ctx, dy):
        return dy, dy


class LateTwice(capture.LateLeafFunction):
    @staticmethod
    def forward(ctx, x, w):
        return x * w

    @staticmethod
    def backward(ctx, dy):
        capture.refuse_beside(ctx)
        return dy, dy


@pytest.fixture
def default(monkeypatch):
    """Whether eager calls run on the default stream."""
    flag = [True]
    monkeypatch.setattr(capture, "_default_stream", lambda device: flag[0])
    return flag


@pytest.fixture
def capturing(monkeypatch, default):
    flag = [False]
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: flag[0])
    return flag


def test_beside_an_eager_graph(capturing):
    x, w = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    alive = Twice.apply(x, w)
    capturing[0] = True
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        Twice.apply(torch.ones(3), w)
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        Twice.apply(x.view(3, 1), torch.ones(3, 1))
    other = torch.ones(3, requires_grad=True)
    Twice.apply(torch.ones(3), other)                              # another leaf
    del alive
    y = Twice.apply(x, w)
    y.sum().backward()
    assert torch.equal(x.grad, torch.ones(3))


def test_without_gradients(capturing):
    """Parameters need gradients, but no node is recorded."""
    x, w = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    alive = Twice.apply(x, w)
    capturing[0] = True
    with torch.no_grad():
        assert not Twice.apply(x, w).requires_grad
    with torch.inference_mode():
        Twice.apply(x, w)
    assert not Twice.apply(x.detach(), w.detach()).requires_grad
    capturing[0] = False
    with torch.no_grad():
        quiet = Twice.apply(x, w)
    del alive
    capturing[0] = True
    Twice.apply(x, w)                                              # no graph is left beside
    assert quiet.grad_fn is None


def test_forward_alone_beside_an_eager_graph(capturing):
    """The backward pass is what may not be captured there, and that holds when
    the eager graph is gone by then."""
    x, w = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    alive = LateTwice.apply(x, w)
    capturing[0] = True
    y, again = LateTwice.apply(x, w), LateTwice.apply(x, w)
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        y.sum().backward()
    assert x.grad is None
    del alive
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        again.sum().backward()
    capturing[0] = False
    LateTwice.apply(x, w).sum().backward()
    x.grad = w.grad = None
    del y, again
    capturing[0] = True
    LateTwice.apply(x, w).sum().backward()                         # no graph is left beside
    assert torch.equal(x.grad, torch.ones(3))


def test_either_function_sees_the_others_graph(capturing):
    w = torch.ones(3, requires_grad=True)
    alive = LateTwice.apply(torch.ones(3), w)
    capturing[0] = True
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        Twice.apply(torch.ones(3), w)
    del alive
    capturing[0] = False
    alive = Twice.apply(torch.ones(3), w)
    capturing[0] = True
    y = LateTwice.apply(torch.ones(3), w)
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        y.sum().backward()
    assert alive.grad_fn is not None


def test_functions_of_the_package():
    from gemm_amax_reduce_amd import adapters, experts, head, linear
    for function in (adapters.AdaptersFunction, experts.NVFP4ExpertsFunction, head.RMSNormFunction):
        assert issubclass(function, capture.LeafFunction) and not function.late
    for function in (head.LayerNormFunction, head.DistillTopKFunction, linear.NVFP4LinearFunction,
                     experts.PackedExpertsFunction):
        assert issubclass(function, capture.LateLeafFunction)


def test_other_threads_record_meanwhile(capturing):
    """A capture looks through the noted nodes while other threads add to them."""
    import sys
    import threading
    w = torch.ones(3, requires_grad=True)
    kept = [Twice.apply(torch.ones(3, requires_grad=True), torch.ones(3)) for _ in range(2000)]
    stop, failed = threading.Event(), []

    def record():
        try:
            while not stop.is_set():
                capture._note(Node(), [w.detach()])
        except Exception as e:
            failed.append(e)

    class Node:
        pass

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    threads = [threading.Thread(target=record) for _ in range(3)]
    try:
        for t in threads:
            t.start()
        for _ in range(200):
            assert not capture._lives_beside([w])
    finally:
        stop.set()
        for t in threads:
            t.join()
        sys.setswitchinterval(before)
    assert not failed and len(kept) == 2000


def test_nodes_that_are_gone_are_swept_out(capturing):
    w = torch.ones(3, requires_grad=True)
    alive = [Twice.apply(torch.ones(3), w) for _ in range(5)]
    for _ in range(3000):
        Twice.apply(torch.ones(3), w)
    assert len(capture._noted) <= 256 + 2 * 2005                   # (another test's nodes may still live)
    capturing[0] = True
    assert capture._lives_beside([w])
    del alive
    assert not capture._lives_beside([w])


def test_beside_a_graph_of_another_stream(capturing, default):
    """As a warm-up's, whose outputs are often kept: that stream joins the capture."""
    default[0] = False
    w = torch.ones(3, requires_grad=True)
    alive = Twice.apply(torch.ones(3), w), LateTwice.apply(torch.ones(3), w)
    capturing[0] = True
    Twice.apply(torch.ones(3), w).sum().backward()
    LateTwice.apply(torch.ones(3), w).sum().backward()
    capturing[0] = False
    default[0] = True
    first = Twice.apply(torch.ones(3), w)                          # (taken for the default stream's)
    default[0] = False
    second = Twice.apply(torch.ones(3), w)                         # holds the first one's accumulator
    del first
    capturing[0] = True
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        Twice.apply(torch.ones(3), w)
    del second, alive
    Twice.apply(torch.ones(3), w)


def test_a_captured_node_keeps_the_accumulator(capturing):
    w = torch.ones(3, requires_grad=True)
    alive = LateTwice.apply(torch.ones(3), w)
    capturing[0] = True
    kept = LateTwice.apply(torch.ones(3), w)                       # captured beside it
    del alive
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        Twice.apply(torch.ones(3), w)
    del kept
    Twice.apply(torch.ones(3), w)
