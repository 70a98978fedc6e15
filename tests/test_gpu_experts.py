"""GPU checks of the modules around grouped products, RMS norm and low-rank
adapters, alone and together as a model uses them, against float64 with the
decoded 4-bit weights.

Everything here is float32 unless said otherwise.  With u = 2^-24, a product of
K terms is off by 6 K u of its mass at most (six partial products of a float32
pair, each added with one rounding); masses are computed beside the values.
"""
import pytest
import torch

import gemm_amax_reduce_amd as nv
import gemm_amax_reduce_amd.experts as E
import gemm_amax_reduce_amd.head as H
from gemm_amax_reduce_amd.adapters import LowRankAdapters

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def ref_rms(h, w, eps):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w


def decoded(weight):
    """The experts' weights in float64 as the forward pass and as the data
    gradient have them."""
    stack = weight.detach().reshape(-1, weight.shape[2])
    q1, q0 = nv.nvfp4_quantize_dual(stack)
    return [t.double().reshape(weight.shape) for t in (nv.nvfp4_dequantize(q1), nv.nvfp4_dequantize(q0).t())]


class RefExperts(torch.autograd.Function):
    """The grouped layer in float64: W1 forward, W0 for dx, dW of the rows."""

    @staticmethod
    def forward(ctx, x, weight, w1, w0, offsets):
        ctx.save_for_backward(x, w0)
        ctx.offsets = offsets
        y = x.new_zeros(x.shape[0], w1.shape[1])
        for e, (b, end) in enumerate(zip(offsets, offsets[1:])):
            y[b:end] = x[b:end] @ w1[e].t()
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w0 = ctx.saved_tensors
        dx, dw = torch.zeros_like(x), torch.zeros_like(w0)
        for e, (b, end) in enumerate(zip(ctx.offsets, ctx.offsets[1:])):
            dx[b:end] = dy[b:end] @ w0[e]
            dw[e] = dy[b:end].t() @ x[b:end]
        return dx, dw, None, None, None


@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_module(residual):
    """Gradients within 256 u of their largest entries: two row sums and a
    column sum of at most 160 roundings, parts of order one times upstream."""
    torch.manual_seed(1)
    norm = H.RMSNorm(160, device="cuda", dtype=torch.float32)
    torch.nn.init.normal_(norm.weight, 1.0, 0.2)
    x = torch.randn((160, 3, 11), device="cuda").permute(1, 2, 0).requires_grad_(True)       # strided
    r = torch.randn((3, 11, 160), device="cuda", requires_grad=True) if residual else None
    up, up_h = torch.randn((2, 3, 11, 160), device="cuda")
    xd, wd = (t.detach().double().requires_grad_(True) for t in (x, norm.weight))
    rd = r.detach().double().requires_grad_(True) if residual else None
    if residual:
        y, h = norm(x, r)
        ((y * up).sum() + (h * up_h).sum()).backward()
        hd = xd + rd
        yd = ref_rms(hd, wd, norm.eps)
        ((yd * up.double()).sum() + (hd * up_h.double()).sum()).backward()
        assert (h.double() - hd).abs().max() <= U * hd.abs().max()
    else:
        y = norm(x)
        (y * up).sum().backward()
        yd = ref_rms(xd, wd, norm.eps)
        (yd * up.double()).sum().backward()
    assert y.shape == x.shape and (y.double() - yd).abs().max() <= 256 * U * yd.abs().max()
    pairs = [(x.grad, xd.grad), (norm.weight.grad, wd.grad)] + ([(r.grad, rd.grad)] if residual else [])
    for got, want in pairs:
        assert (got.double() - want).abs().max() <= 256 * U * want.abs().max()


def test_rms_norm_module_types():
    """A residual stream in float32 beside bf16 activations; one output unused."""
    norm = H.RMSNorm(64, device="cuda")
    x = torch.randn((5, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    r = torch.randn((5, 64), device="cuda", requires_grad=True)
    y, h = norm(x, r)
    assert y.dtype == torch.bfloat16 and h.dtype == torch.float32
    h.sum().backward()
    assert x.grad.dtype == torch.bfloat16 and torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, torch.ones_like(r))
    assert torch.equal(norm.weight.grad, torch.zeros_like(norm.weight))


@pytest.mark.parametrize("cols", [64, 203])
def test_rms_norm_module_keeps_a_float32_gradient(cols):
    """float32 activations beside a bf16 residual: x's gradient carries float32
    roundings alone (as in test_rms_norm_module, from the sum as it is stored),
    the residual's that and half a bf16 step."""
    torch.manual_seed(13)
    norm = H.RMSNorm(cols, device="cuda", dtype=torch.float32)
    torch.nn.init.normal_(norm.weight, 1.0, 0.2)
    x = torch.randn((33, cols), device="cuda", requires_grad=True)
    r = torch.randn((33, cols), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    up = torch.randn((33, cols), device="cuda")
    up_h = torch.randn((33, cols), device="cuda", dtype=torch.bfloat16)
    y, h = norm(x, r)
    assert y.dtype == torch.float32 and h.dtype == torch.bfloat16
    torch.autograd.backward([y, h], [up, up_h])
    hd, wd = (t.detach().double().requires_grad_(True) for t in (h, norm.weight))
    ((ref_rms(hd, wd, norm.eps) * up.double()).sum() + (hd * up_h.double()).sum()).backward()
    assert x.grad.dtype == torch.float32 and r.grad.dtype == torch.bfloat16
    top = hd.grad.abs().max()
    assert (x.grad.double() - hd.grad).abs().max() <= 256 * U * top
    assert ((r.grad.double() - hd.grad).abs() <= 256 * U * top + 2.0 ** -8 * hd.grad.abs()).all()
    assert (norm.weight.grad.double() - wd.grad).abs().max() <= 256 * U * wd.grad.abs().max()


@pytest.mark.parametrize("sizes", [[3, 0, 1, 9], [200, 0, 31, 90], [0, 0, 0, 0]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_module(sizes, dtype):
    """Each of the three products by its own mass; half a bf16 step (2^-8)
    where the result is bf16."""
    torch.manual_seed(2)
    layer = E.NVFP4Experts(4, 64, 96, device="cuda", dtype=dtype)
    rows = sum(sizes) + 2                                      # two of no group
    x = torch.randn((rows, 64), device="cuda").to(dtype).requires_grad_(True)
    up = torch.randn((rows, 96), device="cuda").to(dtype)
    ends = [0]
    for s in sizes:
        ends.append(ends[-1] + s)
    offsets = torch.tensor(ends, device="cuda")
    y = layer(x, offsets)
    y.backward(up)
    w1, w0 = decoded(layer.weight)
    xd = x.detach().double()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0

    def close(got, want, mass, terms):
        assert got.dtype == dtype
        assert ((got.double() - want).abs() <= (6 * terms + 8) * U * mass * 1.02 + half * want.abs() * 1.02).all()

    for e, (b, end) in enumerate(zip(ends, ends[1:])):
        close(y[b:end], xd[b:end] @ w1[e].t(), xd[b:end].abs() @ w1[e].abs().t(), 64)
        close(x.grad[b:end], up[b:end].double() @ w0[e], up[b:end].double().abs() @ w0[e].abs(), 96)
        close(layer.weight.grad[e], up[b:end].double().t() @ xd[b:end], up[b:end].double().abs().t() @ xd[b:end].abs(),
              max(sizes[e], 1))
    assert torch.all(y[ends[-1]:] == 0) and torch.all(x.grad[ends[-1]:] == 0)
    assert torch.equal(layer(x, offsets, layer.pack()), y.detach())


@pytest.mark.parametrize("sizes", [[3, 0, 1, 9], [200, 0, 31, 90], [0, 0, 0, 0]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed_experts_pass_the_gradient_on(sizes, dtype):
    """dx against the packed weights in the data gradient's layout (their decoded
    values quantized along N), the weights themselves left alone; rows of no
    group get zeros.  Bounds as of the module that is trained."""
    torch.manual_seed(11)
    layer = E.NVFP4Experts(4, 64, 96, device="cuda", dtype=dtype)
    packed = layer.pack()
    with torch.no_grad():
        layer.weight.normal_()                                     # what is packed counts
    rows = sum(sizes) + 2
    x = torch.randn((rows, 64), device="cuda").to(dtype).requires_grad_(True)
    up = torch.randn((rows, 96), device="cuda").to(dtype)
    ends = [0]
    for s in sizes:
        ends.append(ends[-1] + s)
    offsets = torch.tensor(ends, device="cuda")
    y = layer(x * 1, offsets, packed)
    assert torch.equal(y, layer(x.detach(), offsets, packed))
    first, = torch.autograd.grad(y, [x], up, retain_graph=True)
    y.backward(up)
    assert torch.equal(first, x.grad) and x.grad.dtype == dtype and layer.weight.grad is None
    w1 = nv.nvfp4_dequantize(packed)
    w0 = nv.nvfp4_dequantize(nv.nvfp4_quantize(w1, axis=0)).t().double().reshape(4, 96, 64)
    w1 = w1.double().reshape(4, 96, 64)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for e, (b, end) in enumerate(zip(ends, ends[1:])):
        want, mass = up[b:end].double() @ w0[e], up[b:end].double().abs() @ w0[e].abs()
        bound = (6 * 96 + 8) * U * mass * 1.02 + half * want.abs() * 1.02
        assert ((x.grad[b:end].double() - want).abs() <= bound).all()
        # and the formula's own gradient, as near as the two layouts' weights are
        off = (x.grad[b:end].double() - up[b:end].double() @ w1[e]).abs()
        assert (off <= bound + up[b:end].double().abs() @ (w0[e] - w1[e]).abs()).all()
    assert torch.all(x.grad[ends[-1]:] == 0)
    assert (w0 - w1).norm() <= 0.2 * w1.norm()


def test_a_packed_block_passes_the_gradient_on():
    """Frozen experts between trained parts: what lies before them gets the
    gradient that the trained form gives it, to the rounding of the 4-bit
    layouts: a quantization is off by some 0.1 of the weights' norm, and three of
    them lie between the two forms' data gradients of each of two products,
    2 * sqrt(3) * 0.1 < 0.5."""
    torch.manual_seed(12)
    block = E.NVFP4ExpertBlock(4, 2, 64, 96, device="cuda", dtype=torch.float32)
    for p, std in ((block.up.weight, 0.125), (block.down.weight, 0.1), (block.router, 0.125)):
        torch.nn.init.normal_(p, std=std)
    x, r, up = torch.randn((3, 40, 64), device="cuda")
    x.requires_grad_(True)
    leaves = [x, block.norm.weight, block.router]
    want = torch.autograd.grad(block(x, r)[0], leaves, up)
    got = torch.autograd.grad(block(x, r, block.pack())[0], leaves, up)
    for p, q in zip(got, want):
        assert (p - q).norm() <= 0.5 * q.norm()


def test_experts_backward_twice():
    layer = E.NVFP4Experts(2, 32, 32, device="cuda")
    x = torch.randn((9, 32), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = layer(x, torch.tensor([0, 4, 9], device="cuda")).sum()
    first = torch.autograd.grad(y, [x, layer.weight], retain_graph=True)
    again = torch.autograd.grad(y, [x, layer.weight])
    assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_group_by_expert():
    choice = torch.tensor([[2, 0], [1, 2], [-1, 2], [0, 7]], device="cuda")
    order, offsets = E.group_by_expert(choice, 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert choice.reshape(-1)[order].tolist()[:6] == [0, 0, 1, 2, 2, 2]
    assert order.tolist() == [1, 6, 2, 0, 3, 5, 4, 7]
    order, offsets = E.group_by_expert(torch.empty((0, 2), dtype=torch.int64, device="cuda"), 3)
    assert order.numel() == 0 and offsets.tolist() == [0, 0, 0, 0]


def ref_adapters(x, a, b, scale, base, offsets, index):
    y = base.clone() if base is not None else x.new_zeros(x.shape[0], b.shape[1])
    for i, (s, e) in enumerate(zip(offsets, offsets[1:])):
        if index[i] >= 0:
            y[s:e] = y[s:e] + scale[index[i]] * (x[s:e] @ a[index[i]].t()) @ b[index[i]].t()
    return y


@pytest.mark.parametrize("with_base", [False, True])
def test_adapters_module(with_base):
    """Relative to the largest entry of each result: sums of at most 6 (96 + 8)
    roundings forward, and as many again behind them in the gradients, with
    masses below 16 times the largest entry."""
    torch.manual_seed(3)
    low = LowRankAdapters(3, 96, 80, 8, scale=0.7, device="cuda", dtype=torch.float32)
    torch.nn.init.normal_(low.b)
    x = torch.randn((2, 20, 96), device="cuda", requires_grad=True)
    base = torch.randn((2, 20, 80), device="cuda", requires_grad=True) if with_base else None
    at, which = [0, 7, 7, 30, 38], [2, 0, -1, 2]
    offsets, index = torch.tensor(at, device="cuda"), torch.tensor(which, device="cuda")
    up = torch.randn((2, 20, 80), device="cuda")
    y = low(x, base, offsets, index)
    y.backward(up)
    leaves = [x, low.a, low.b] + ([base] if with_base else [])
    dd = [t.detach().double().requires_grad_(True) for t in leaves]
    yd = ref_adapters(dd[0].reshape(-1, 96), dd[1], dd[2], low.scale.double(),
                      dd[3].reshape(-1, 80) if with_base else None, at, which).reshape(2, 20, 80)
    yd.backward(up.double())
    tolerance = 2 * 6 * 104 * U * 16
    for got, want in [(y, yd)] + [(p.grad, q.grad) for p, q in zip(leaves, dd)]:
        assert (got.double() - want).abs().max() <= tolerance * want.abs().max()
    assert torch.all(low.a.grad[1] == 0) and torch.all(low.b.grad[1] == 0)
    with torch.no_grad():
        assert torch.equal(LowRankAdapters(3, 96, 80, 8, device="cuda", dtype=torch.float32)(x, base, offsets, index),
                           base if with_base else torch.zeros_like(y))


def test_adapters_converted_to_another_type():
    """A module made in float32 and brought to bf16 (beside a head that is, too)
    is the one made in bf16: forward, gradients, and the part added in place."""
    torch.manual_seed(10)
    low = LowRankAdapters(2, 64, 96, 8, scale=0.3)                 # on the CPU
    torch.nn.init.normal_(low.b)
    same = LowRankAdapters(2, 64, 96, 8, scale=0.3, device="cuda")
    with torch.no_grad():
        same.a.copy_(low.a), same.b.copy_(low.b)
    low.cuda().to(torch.bfloat16)
    offsets, index = torch.tensor([0, 5, 20], device="cuda"), torch.tensor([1, 0], device="cuda")
    x = torch.randn((20, 64), device="cuda", dtype=torch.bfloat16)
    base = torch.randn((20, 96), device="cuda", dtype=torch.bfloat16)
    ys = []
    for m in (low, same):
        y = m(x, base, offsets, index)
        y.sum().backward()
        ys.append(y)
        assert torch.equal(m.add(x, base.clone(), offsets, index), y)
    assert torch.equal(*ys) and torch.equal(low.a.grad, same.a.grad) and torch.equal(low.b.grad, same.b.grad)


@pytest.mark.parametrize("tokens", [0, 1, 16, 17, 48])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_answers_with_adapters(tokens, norm):
    """A batch of requests on one packed head, each token with its request's
    adapter, against float64 from the same normed activations."""
    torch.manual_seed(4)
    head = H.NVFP4Head(128, 208, device="cuda", norm=norm)
    low = LowRankAdapters(3, 128, 208, 16, device="cuda")
    torch.nn.init.normal_(low.b)
    packed = head.pack()
    x = torch.randn((tokens, 128), device="cuda", dtype=torch.bfloat16)
    at = [0, tokens // 3, tokens // 3, tokens - tokens // 4]
    which = [1, 0, 2]
    offsets, index = (torch.tensor(t, device="cuda", dtype=torch.int32) for t in (at, which))
    plain = head.answer(x, packed)
    y = head.answer(x, packed, adapters=low, offsets=offsets, index=index)
    h = head.norm(x).detach().double()
    a, b = low.a.detach().double(), low.b.detach().double()
    want = ref_adapters(h, a, b, low.scale, plain.double(), at, which)
    mass = ref_adapters(h.abs(), a.abs(), b.abs(), low.scale, plain.double().abs(), at, which)
    assert y.dtype == torch.float32 and y.shape == (tokens, 208)
    # u of 128 exact products, then 3 partial products for each of 16 ranks
    assert ((y.double() - want).abs() <= (128 + 3 * 16 + 8) * U * mass).all()


def ref_block(block, x, residual, w_norm, router, ups, downs):
    """The expert block in float64; ups, downs: (weight leaf, W1, W0)."""
    h = x + residual
    n = ref_rms(h, w_norm, block.norm.eps)
    rows = n.reshape(-1, n.shape[-1])
    best, choice = torch.topk(rows @ router.t(), block.top, dim=1)
    order, offsets = E.group_by_expert(choice, router.shape[0])
    at = offsets.tolist()
    both = RefExperts.apply(rows[order // block.top], *ups, at)
    gate, up = both.chunk(2, 1)
    out = RefExperts.apply(torch.nn.functional.silu(gate) * up, *downs, at)
    y = torch.zeros_like(rows).index_add(0, order // block.top, out * torch.softmax(best, 1).reshape(-1)[order][:, None])
    return y.reshape(x.shape), h


@pytest.mark.parametrize("tokens,experts,top", [(1, 4, 2), (33, 4, 2), (40, 16, 1), (300, 3, 3)])
def test_block(tokens, experts, top):
    """Norm, grouped products both ways and their gradients as one block.  Each
    of its ten stages is off by at most 6 * 256 u times the ratio of its mass
    to its largest entry, below 8 here: 10 * 6 * 256 * 8 u < 2^-7 of the largest
    entry of each result."""
    torch.manual_seed(5)
    block = E.NVFP4ExpertBlock(experts, top, 64, 96, device="cuda", dtype=torch.float32)
    for p, std in ((block.up.weight, 0.125), (block.down.weight, 0.1), (block.router, 0.125)):
        torch.nn.init.normal_(p, std=std)
    x, r, up_y, up_h = torch.randn((4, tokens, 64), device="cuda")
    x.requires_grad_(True), r.requires_grad_(True)
    y, h = block(x, r)
    ((y * up_y).sum() + (h * up_h).sum()).backward()
    leaves = [x, r, block.norm.weight, block.router, block.up.weight, block.down.weight]
    d = [t.detach().double().requires_grad_(True) for t in leaves]
    yd, hd = ref_block(block, *d[:4], (d[4], *decoded(block.up.weight)), (d[5], *decoded(block.down.weight)))
    ((yd * up_y.double()).sum() + (hd * up_h.double()).sum()).backward()
    for got, want in [(y, yd), (h, hd)] + [(p.grad, q.grad) for p, q in zip(leaves, d)]:
        assert (got.double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
    with torch.no_grad():
        answer, _ = block(x, r, block.pack())
    assert torch.equal(answer, y)                             # the same weights, packed once


def test_a_model_of_them():
    """Two blocks and a head with adapters, trained for a step and answering:
    every parameter has a finite gradient, and the packed weights answer."""
    torch.manual_seed(6)
    blocks = [E.NVFP4ExpertBlock(4, 2, 64, 64, device="cuda") for _ in range(2)]
    head = H.NVFP4Head(64, 96, device="cuda", norm="rms")
    low = LowRankAdapters(2, 64, 96, 4, device="cuda")
    torch.nn.init.normal_(low.b, std=0.1)
    offsets, index = torch.tensor([0, 10, 32], device="cuda"), torch.tensor([1, 0], device="cuda")
    x = torch.randn((32, 64), device="cuda", dtype=torch.bfloat16)

    def through(x, packed):
        residual = torch.zeros_like(x)
        for block, p in zip(blocks, packed):
            x, residual = block(x, residual, p)
        return x + residual

    h = through(x, [None, None])
    n = head.norm(h)
    logits = low(n, head.proj(n), offsets, index)
    choice = torch.randint(0, 96, (32, 4), device="cuda")
    H.distill_topk_loss(logits, choice, torch.randn((32, 4), device="cuda")).backward()
    for module in (*blocks, head, low):
        for name, p in module.named_parameters():
            assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
    with torch.no_grad():
        packed = [b.pack() for b in blocks]
        one = through(x[:1], packed)
        y = head.answer(one, head.pack(), adapters=low, offsets=torch.tensor([0, 1], device="cuda"),
                        index=torch.tensor([1], device="cuda"))
    assert y.shape == (1, 96) and torch.isfinite(y).all()


def _chain():
    torch.manual_seed(7)
    norm = H.RMSNorm(64, device="cuda")
    layer = E.NVFP4Experts(3, 64, 96, device="cuda")
    low = LowRankAdapters(2, 96, 64, 8, device="cuda")
    torch.nn.init.normal_(low.b)
    x = torch.randn((90, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    r = torch.randn((90, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    offsets, index = torch.tensor([0, 20, 61, 80], device="cuda"), torch.tensor([1, -1, 0], device="cuda")
    leaves = [x, r, norm.weight, layer.weight, low.a, low.b]

    def step():
        n, h = norm(x, r)
        y = low(layer(n, offsets), h, offsets, index)
        return [y.detach(), *torch.autograd.grad(y, leaves, torch.ones_like(y))]

    return step, x, r, offsets, index


def test_captured_and_replayed():
    step, x, r, offsets, index = _chain()
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        with torch.no_grad():
            x.copy_(torch.randn_like(x)), r.copy_(torch.randn_like(r))
        offsets[1:-1] //= 2
        index.copy_(index.roll(1))
        want = step()


def test_tensors_stay_plain():
    """Nothing is left on parameters or inputs that would be saved with them."""
    step, x, r, _, _ = _chain()
    step()
    assert not vars(x) and not vars(r)


def test_capture_beside_an_eager_graph_is_refused():
    layer = E.NVFP4Experts(2, 32, 32, device="cuda")
    x = torch.randn((8, 32), device="cuda", dtype=torch.bfloat16)
    offsets = torch.tensor([0, 3, 8], device="cuda")
    alive = layer(x, offsets)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        with torch.cuda.graph(graph):
            layer(x, offsets)
    del alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, offsets)
        grad, = torch.autograd.grad(y, [layer.weight], torch.ones_like(y))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, nv.nvfp4_grouped_wgrad(torch.ones_like(y), x, offsets, torch.bfloat16))


def test_answers_are_captured_beside_an_eager_graph():
    """Without gradients no node is recorded, and a training output may live on."""
    torch.manual_seed(8)
    block = E.NVFP4ExpertBlock(4, 2, 64, 64, device="cuda")
    low = LowRankAdapters(2, 64, 64, 4, device="cuda")
    torch.nn.init.normal_(low.b)
    x, r = (torch.randn((24, 64), device="cuda", dtype=torch.bfloat16).requires_grad_(True) for _ in range(2))
    offsets, index = torch.tensor([0, 10, 24], device="cuda"), torch.tensor([1, 0], device="cuda")
    at = torch.tensor([0, 5, 9, 20, 24], device="cuda")

    def run(packed=None):
        n, h = block.norm(x, r)
        return [low(n, h, offsets, index), block.up(n, at, packed)]

    alive = run()                                                  # an eager graph of every parameter
    packed = block.pack()
    with torch.no_grad():
        want = run(packed[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(packed[0])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(packed[0])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
            want = run(packed[0])
    assert all(t.grad_fn is not None for t in alive)


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_a_head_captured_beside_an_eager_graph(norm):
    """Norm, 4-bit projection and loss: the forward pass is captured beside a
    live eager graph (without the gradient of an RMS norm, which is refused at
    once), the backward pass is refused until that is gone."""
    torch.manual_seed(9)
    head = H.NVFP4Head(64, 96, device="cuda", norm=norm)
    head.proj.requires_grad_(False)                                # (its rounding draws anew in every call)
    x = torch.randn((32, 64), device="cuda", dtype=torch.bfloat16, requires_grad=norm == "layer")
    at, teacher = torch.randint(0, 96, (32, 4), device="cuda"), torch.randn((32, 4), device="cuda")
    leaves = [head.norm.weight] + ([x] if norm == "layer" else [])

    def forward():
        return H.distill_topk_loss(head.proj(head.norm(x)), at, teacher)

    alive = forward()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        with torch.cuda.graph(graph):
            loss = forward()
            assert norm == "layer"
            torch.autograd.grad(loss, leaves)
    if norm == "layer":
        del loss
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss = forward()
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss, alive)
        del loss, graph
    del alive
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(forward(), leaves)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.isfinite(g).all() and g.abs().max() > 0 for g in got)


def test_a_layer_captured_beside_the_graph_of_another():
    """The eager graph is a layer norm's, the captured function an RMS norm of
    the same x."""
    x = torch.randn((8, 64), device="cuda", requires_grad=True)
    layer, rms = H.LayerNorm(64, device="cuda", dtype=torch.float32), H.RMSNorm(64, device="cuda", dtype=torch.float32)
    alive = layer(x)
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            rms(x)
    assert alive.grad_fn is not None


def test_packed_experts_captured():
    """Beside a live eager graph of x forward alone, its backward pass once that
    is gone; every replay with the eager result."""
    layer = E.NVFP4Experts(2, 32, 48, device="cuda")
    packed, offsets = layer.pack(), torch.tensor([0, 3, 8], device="cuda")
    x = torch.randn((8, 32), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    up = torch.randn((8, 48), device="cuda", dtype=torch.bfloat16)
    alive = layer(x, offsets, packed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, offsets, packed)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, alive)
    with pytest.raises(nv.NVFP4Error, match="still lives"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(layer(x, offsets, packed), [x], up)
    del alive, y, graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(layer(x, offsets, packed), [x], up)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        q = nv.nvfp4_quantize(nv.nvfp4_dequantize(packed), axis=0)
        assert torch.equal(got, nv.nvfp4_grouped_matmul(q, up, offsets, transposed=True))
        up.copy_(torch.randn_like(up))


@pytest.mark.parametrize("part", ["linear", "layer norm", "rms norm", "experts", "adapters", "packed experts"])
def test_captured_beside_the_graph_of_a_warm_up(part):
    """The usual way to a captured training step: a warm-up on a side stream, whose
    outputs stay in scope, then the capture."""
    torch.manual_seed(14)
    x = torch.randn((32, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    offsets, index = torch.tensor([0, 10, 32], device="cuda"), torch.tensor([1, 0], device="cuda")
    experts, low = E.NVFP4Experts(2, 64, 64, device="cuda"), LowRankAdapters(2, 64, 64, 4, device="cuda")
    torch.nn.init.normal_(low.b)
    packed, linear = experts.pack(), H.NVFP4Linear(64, 64, device="cuda")
    linear.weight.requires_grad_(part == "linear")
    norm = (H.LayerNorm if part == "layer norm" else H.RMSNorm)(64, device="cuda")
    call, leaves = {"linear": (lambda: linear(x), [x, linear.weight]), "layer norm": (lambda: norm(x), [x, norm.weight]),
                    "rms norm": (lambda: norm(x), [x, norm.weight]),
                    "experts": (lambda: experts(x, offsets), [x, experts.weight]),
                    "adapters": (lambda: low(x, None, offsets, index), [x, low.a, low.b]),
                    "packed experts": (lambda: experts(x, offsets, packed), [x])}[part]
    up = torch.randn((32, 64), device="cuda", dtype=torch.bfloat16)

    def step():
        y = call()
        y.backward(up)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            alive = step()
    torch.cuda.current_stream().wait_stream(side)
    for leaf in leaves:
        leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    grads = [leaf.grad for leaf in leaves]
    for _ in range(3):
        for g in grads:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, alive)
        assert all(torch.isfinite(g).all() and g.abs().max() > 0 for g in grads)
