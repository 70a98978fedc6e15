"""The workspace that nvfp4_gemm_ws takes by itself: one for each stream, cleared
in that stream's order."""
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu


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
