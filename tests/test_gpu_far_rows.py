"""Rows that lie so far apart that a tile's own offsets pass 32 bits: the
operators on such matrices give what they give on compact copies of them."""
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

ROWS, COLS, LD = 40, 96, (1 << 25) + 4          # float32: 134 MB from row to row


@pytest.fixture(scope="module")
def far():
    """[ROWS, COLS] views of two buffers of 5.4 GB, with their values elsewhere."""
    if torch.cuda.mem_get_info()[0] < (24 << 30):
        pytest.skip("needs 24 GB")
    torch.manual_seed(1)
    out = []
    for dtype, ld in ((torch.float32, LD), (torch.bfloat16, 2 * LD)):
        view = torch.empty(ROWS * ld, dtype=dtype, device="cuda").view(ROWS, ld)[:, :COLS]
        view.copy_(torch.randn((ROWS, COLS), device="cuda"))
        out.append(view)
    yield out
    out.clear()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("which", [0, 1])
def test_norm(far, which):
    x = far[which]
    near = x.contiguous()
    for got, want in zip(nv.nvfp4_rms_norm(x, None, x), nv.nvfp4_rms_norm(near, None, near)):
        assert torch.equal(got, want)
    rstd = torch.rand(ROWS, device="cuda")
    for got, want in zip(nv.nvfp4_rms_norm_backward(x, x, rstd, dh=x), nv.nvfp4_rms_norm_backward(near, near, rstd, dh=near)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("ends", [[0, 40], [0, 2, 5, 40]])
def test_grouped(far, which, ends):
    x = far[which]
    near = x.contiguous()
    experts = len(ends) - 1
    offsets = torch.tensor(ends, device="cuda")
    w = nv.nvfp4_quantize(torch.randn((experts * 160, COLS), device="cuda"))
    assert torch.equal(nv.nvfp4_grouped_matmul(w, x, offsets), nv.nvfp4_grouped_matmul(w, near, offsets))
    assert torch.equal(nv.nvfp4_grouped_wgrad(x, x, offsets), nv.nvfp4_grouped_wgrad(near, near, offsets))


@pytest.mark.parametrize("which", [0, 1])
def test_adapters(far, which):
    x = far[which]
    near = x.contiguous()
    offsets, index = torch.tensor([0, 1, 40], device="cuda"), torch.tensor([1, 0], device="cuda")
    a = torch.randn((2, 8, COLS), device="cuda", dtype=x.dtype)
    b = torch.randn((2, COLS, 8), device="cuda", dtype=x.dtype)
    y, u = nv.nvfp4_adapters(x, a, b, offsets, index, base=x)
    want_y, want_u = nv.nvfp4_adapters(near, a, b, offsets, index, base=near)
    assert torch.equal(y, want_y) and torch.equal(u, want_u)
    for got, want in zip(nv.nvfp4_adapters_backward(x, x, u, a, b, offsets, index, base=x),
                         nv.nvfp4_adapters_backward(near, near, u, a, b, offsets, index, base=near)):
        assert torch.equal(got, want)
