"""GPU checks of the head module on inputs that do not lie as the kernels read
them: they give what their contiguous copies give."""
import pytest
import torch

import gemm_amax_reduce_amd.head as H

pytestmark = pytest.mark.gpu


def _layouts(rows, cols):
    """Name -> a [rows, cols] matrix of some layout."""
    g = torch.Generator(device="cuda").manual_seed(rows * cols)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)
    return {"transposed": r(cols, rows).t(), "one row for all": r(1, cols).expand(rows, cols),
            "windows": r(rows + cols).unfold(0, cols, 1)[:rows], "every other": r(rows, 2 * cols)[:, ::2],
            "padded": r(rows, cols + 3)[:, :cols], "one value": r(1, 1).expand(rows, cols)}


NAMES = ["transposed", "one row for all", "windows", "every other", "padded", "one value"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 64), (33, 48)])
def test_norm(rows, cols, name):
    norm = H.LayerNorm(cols, device="cuda", dtype=torch.float32)
    torch.nn.init.normal_(norm.weight)
    x = _layouts(rows, cols)[name]
    up = torch.randn((rows, cols), device="cuda")
    got = x.detach().requires_grad_(True)
    want = x.detach().contiguous().clone().requires_grad_(True)
    y, z = norm(got), norm(want)
    assert torch.equal(y, z)
    assert torch.equal(torch.autograd.grad(y, got, up)[0], torch.autograd.grad(z, want, up)[0])


@pytest.mark.parametrize("name", NAMES)
def test_loss(name):
    z = _layouts(6, 40)[name]
    idx = torch.randint(0, 40, (6, 3), device="cuda")
    t = torch.randn((6, 3), device="cuda")
    got = z.detach().requires_grad_(True)
    want = z.detach().contiguous().clone().requires_grad_(True)
    a, b = H.distill_topk_loss(got, idx, t), H.distill_topk_loss(want, idx, t)
    assert torch.equal(a, b)
    assert torch.equal(torch.autograd.grad(a, got)[0], torch.autograd.grad(b, want)[0])


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows", [1, 5, 16, 17, 48])
def test_answer(rows, name):
    torch.manual_seed(6)
    head = H.NVFP4Head(64, 80, device="cuda", dtype=torch.float32)
    packed = head.pack()
    x = _layouts(rows, 64)[name]
    assert torch.equal(head.answer(x, packed), head.answer(x.contiguous().clone(), packed))


def test_loss_of_shortened_lists():
    """The best of longer lists, as slices of them, and lists by columns."""
    z = torch.randn((6, 40), device="cuda", requires_grad=True)
    best = torch.topk(torch.randn((6, 40), device="cuda"), 8, 1)
    for idx, t in ((best.indices[:, :3], best.values[:, :3]),
                   (best.indices.t().contiguous().t(), best.values.t().contiguous().t())):
        a = H.distill_topk_loss(z, idx, t, temperature=2.0)
        b = H.distill_topk_loss(z, idx.contiguous(), t.contiguous(), temperature=2.0)
        assert torch.equal(a, b)
        assert torch.equal(torch.autograd.grad(a, z)[0], torch.autograd.grad(b, z)[0])
