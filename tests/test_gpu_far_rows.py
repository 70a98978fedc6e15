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


def _stack(outer, k):
    """Random codes with scales of one: weights are multiples of 1/2 up to 6."""
    codes = torch.randint(0, 256, (outer, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.ones((outer, k // 16), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    return nv.NVFP4Tensor(codes, scales, torch.tensor([2688.0, 1.0], device="cuda"), outer, k)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [3, 300])
def test_stack_past_4_gb(transposed, rows):
    """The last expert of a stack of 4.4 GB of codes, by whole numbers, whose
    sums (below 16384 * 6 * 3) have no rounding."""
    if torch.cuda.mem_get_info()[0] < (24 << 30):
        pytest.skip("needs 24 GB")
    torch.manual_seed(2)
    experts, n, k = (8192, 64, 16384) if transposed else (66, 8192, 16384)
    w = _stack(n, experts * k) if transposed else _stack(experts * n, k)
    if transposed:
        last = nv.NVFP4Tensor(w.codes[:, -k // 2:].contiguous(), w.scales[:, -k // 16:].contiguous(), w.meta, n, k)
    else:
        last = nv.NVFP4Tensor(w.codes[-n:].contiguous(), w.scales[-n:].contiguous(), w.meta, n, k)
    x = torch.randint(-3, 4, (rows, k), device="cuda").bfloat16()
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[-1] = rows
    got = nv.nvfp4_grouped_matmul(w, x, offsets, torch.float32, transposed=transposed)
    want = x.double() @ nv.nvfp4_dequantize(last).double().t()
    assert torch.equal(got.double(), want)


def test_weight_gradient_past_32_bits():
    """A gradient of 2^32 elements and more, its last expert's by whole numbers."""
    if torch.cuda.mem_get_info()[0] < (24 << 30):
        pytest.skip("needs 24 GB")
    torch.manual_seed(3)
    experts, n = 66, 8192
    dy, x = torch.randint(-3, 4, (2, 40, n), device="cuda").bfloat16()
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[-1] = 40
    dw = nv.nvfp4_grouped_wgrad(dy, x, offsets, torch.bfloat16, out=torch.full((experts, n, n), 5.0, device="cuda",
                                                                              dtype=torch.bfloat16))
    # (below 40 * 9 = 360: not every whole number above 256 is a bf16, so through float32)
    want = (dy.float().t() @ x.float()).bfloat16()
    assert torch.equal(dw[-1], want)
    for part in dw[:-1].split(11):
        assert part.abs().max() == 0
