"""The workspace that nvfp4_gemm_ws takes by itself: one for each stream, cleared
in that stream's order, and one of its own for every captured call."""
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu


def test_captured_graphs_share_none():
    """Neither a graph whose clearing is only captured, nor two graphs, may
    leave theirs to another call."""
    a, b = (nv.nvfp4_quantize(torch.randn((n, 128), device="cuda")) for n in (300, 200))
    want = nv.nvfp4_gemm_ws(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = {k: v.data_ptr() for k, v in nv._workspaces.items()}
    held, graphs, outs = [], [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held.append(nv.gemm_workspace())
            outs.append(nv.nvfp4_gemm_ws(a, b))
        graphs.append(graph)
    assert {k: v.data_ptr() for k, v in nv._workspaces.items()} == before
    assert len({t.data_ptr() for t in held} | set(before.values())) == 2 + len(set(before.values()))
    for _ in range(3):
        for graph, out in zip(graphs[::-1], outs[::-1]):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(nv.nvfp4_gemm_ws(a, b), want)
    for t in held:
        assert torch.all(t[:1 << 16] == 0)


def test_one_for_each_stream():
    side = torch.cuda.Stream()
    a, b = nv.gemm_workspace(), nv.gemm_workspace(stream=side)
    assert a.data_ptr() != b.data_ptr()
    for device in (None, 0, "cuda", "cuda:0", torch.device("cuda")):
        assert nv.gemm_workspace(device) is a and nv.gemm_workspace(device, side) is b
    with torch.cuda.stream(side):
        assert nv.gemm_workspace() is b


def test_cleared_in_its_streams_order():
    """The current stream is busy, and its allocator holds a block of ones."""
    size = int(nv.lib().nvfp4_gemm_workspace_bytes())
    torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    ws = nv.gemm_workspace(stream=side)
    with torch.cuda.stream(side):
        flags = ws[:1 << 16].clone()
    side.synchronize()
    assert torch.all(flags == 0)
    torch.cuda.synchronize()
