"""GPU checks of the head module: autograd through norm and loss against
float64, the answer's two forms against the decoded weights, and the example,
which uses all of it together."""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv
import gemm_amax_reduce_amd.head as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _ref_norm(x, w, b, eps):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps) * w + b


def test_norm_module_gradients():
    """Float32 against float64 autograd; 256 u covers two row sums of 64
    roundings and the products around them, relative to each gradient's
    largest parts (all of order one times the upstream gradient here)."""
    torch.manual_seed(1)
    norm = H.LayerNorm(160, device="cuda", dtype=torch.float32)
    torch.nn.init.normal_(norm.weight, 1.0, 0.2)
    torch.nn.init.normal_(norm.bias, 0.0, 0.2)
    x = torch.randn((3, 11, 160), device="cuda", requires_grad=True)
    up = torch.randn((3, 11, 160), device="cuda")
    (norm(x) * up).sum().backward()
    xd = x.detach().double().requires_grad_(True)
    wd, bd = (p.detach().double().requires_grad_(True) for p in (norm.weight, norm.bias))
    (_ref_norm(xd, wd, bd, norm.eps) * up.double()).sum().backward()
    for got, want in ((x.grad, xd.grad), (norm.weight.grad, wd.grad), (norm.bias.grad, bd.grad)):
        assert (got.double() - want).abs().max() <= 256 * U * want.abs().max()


def test_norm_module_takes_strided_input_and_gradient():
    norm = H.LayerNorm(64, device="cuda", dtype=torch.float32)
    base = torch.randn((64, 30), device="cuda")
    x = base.t().requires_grad_(True)                       # columns are not contiguous
    y = norm(x)
    y.sum().backward()                                      # an expanded gradient
    assert torch.equal(y, norm(x.detach().contiguous()))
    # dy = 1 and weight 1: a - mean(a) = 0, so dx is 0 up to rounding of the sums
    assert x.grad.abs().max() <= 64 * U * 4


def test_loss_gradient_and_weights():
    torch.manual_seed(2)
    z = torch.randn((10, 300), device="cuda", requires_grad=True)
    t, idx = torch.topk(torch.randn((10, 300), device="cuda"), 7, 1)
    weight = torch.rand(10, device="cuda")
    for w in (weight, None):
        z.grad = None
        H.distill_topk_loss(z, idx, t, w, temperature=1.5).backward()
        zd = z.detach().double().requires_grad_(True)
        p = torch.softmax(t.double() / 1.5, 1)
        q = torch.log_softmax(zd / 1.5, 1).gather(1, idx)
        loss = 1.5 ** 2 * (p * (p.log() - q)).sum(1)
        (loss.mean() if w is None else (loss * w.double()).sum()).backward()
        # shares to within 4 u (64 + 70 + spans below 10)
        assert (z.grad.double() - zd.grad).abs().max() <= 4 * U * 144 * 1.5


def test_head_gradients_flow_through_the_whole():
    torch.manual_seed(3)
    head = H.NVFP4Head(64, 96, device="cuda", dtype=torch.float32)
    x = torch.randn((2, 16, 64), device="cuda", requires_grad=True)
    idx = torch.randint(0, 96, (32, 4), device="cuda")
    head.loss(x, idx, torch.randn((32, 4), device="cuda")).backward()
    for g in (x.grad, head.norm.weight.grad, head.norm.bias.grad, head.proj.weight.grad):
        assert g is not None and torch.isfinite(g).all() and g.abs().max() > 0


@pytest.mark.parametrize("tokens", [0, 1, 5, 16, 17, 48])
def test_answer(tokens):
    """A few tokens unquantized, more through the quantizer fed by the norm's
    maximum; both against the decoded operands in float64."""
    torch.manual_seed(4)
    head = H.NVFP4Head(128, 208, device="cuda", dtype=torch.bfloat16)
    packed = head.pack()
    x = torch.randn((1, tokens, 128), device="cuda", dtype=torch.bfloat16)
    y = head.answer(x, packed)
    assert y.shape == (1, tokens, 208) and y.dtype == torch.float32
    h = head.norm(x).detach().reshape(-1, 128)
    if tokens > H.MATVEC_TOKENS:
        h = nv.nvfp4_dequantize(nv.nvfp4_quantize(h))
    w = nv.nvfp4_dequantize(packed).double()
    want, mass = h.double() @ w.t(), h.double().abs() @ w.abs().t()
    err = (y[0].double() - want).abs()
    assert tokens == 0 or (err <= 1e-5 * mass).all()


def test_refusals():
    norm = H.LayerNorm(64, device="cuda")
    with pytest.raises(nv.NVFP4Error, match="features"):
        norm(torch.zeros((4, 32), device="cuda"))
    with pytest.raises(nv.NVFP4Error, match="GPU"):
        H.LayerNorm(64)(torch.zeros(4, 64))


def test_example():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("distill_head", os.path.join(root, "examples", "distill_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, before, after = m.train(steps=40, features=256, vocab=1024, tokens=512, top=16)
    assert last < 0.7 * first
    assert after > before + 0.2
