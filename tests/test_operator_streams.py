"""The stream that a call is given has to be one of its tensors' device."""
from types import SimpleNamespace

import pytest
import torch

import gemm_amax_reduce_amd as nv


def test_stream_of_another_device():
    # (the check comes before anything that needs a GPU; a stream is known by its device)
    with pytest.raises(nv.NVFP4Error, match="stream"):
        nv._on(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.gpu
def test_own_stream():
    side = torch.cuda.Stream()
    x = torch.randn((3, 64), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    y = nv.nvfp4_layer_norm(x, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, nv.nvfp4_layer_norm(x)[0])
