"""GPU checks of layer norm, forward and backward, against the definition in
float64, element by element, within error bounds derived from binary32
arithmetic (u = 2^-24).

Forward: the mean is a sum in at most 64 roundings after each other, and so is
the variance, whose relative error halves in rstd; with the subtraction, two
products and the bias one output is off by at most
    64 u (|w| (r (mean|x| + |x|) + |h|) + |b|),    h = (x - m) r,
and half a bf16 step (2^-8 of the value) where it is stored in bf16.
Backward: with a = dy w, two sums in at most 64 roundings each,
    64 u r (|a| + mean|a| + 2 |h| mean|a h|)
and the sums over rows in whatever order (rows + 2) u sum|.|.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _matrix(values, dtype, pad=0, shift=0):
    """values on the GPU as a view with `pad` spare elements per row, `shift`
    elements off the allocation's start."""
    rows, cols = values.shape
    flat = torch.full((shift + rows * (cols + pad),), 7.0, dtype=dtype, device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(values.to(dtype))
    return view


def _inputs(rows, cols, dtype, wdtype, seed, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * 2 + torch.randn((1, cols), generator=g)
    x *= 1 + 30 * (torch.rand((1, cols), generator=g) < 0.02)
    dy = torch.randn((rows, cols), generator=g) * 1e-3
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(wdtype).cuda()
    b = (0.2 * torch.randn(cols, generator=g)).to(wdtype).cuda()
    return _matrix(x, dtype, pad, shift), _matrix(dy, dtype, pad, shift), w, b


def _ref_forward(x, w, b, eps):
    x = x.double().cpu().numpy()
    w = np.ones(x.shape[1]) if w is None else w.double().cpu().numpy()
    b = np.zeros(x.shape[1]) if b is None else b.double().cpu().numpy()
    m = x.mean(1, keepdims=True)
    v = ((x - m) ** 2).mean(1, keepdims=True)
    r = 1 / np.sqrt(v + eps)
    h = (x - m) * r
    bound = 64 * U * (np.abs(w) * (r * (np.abs(x).mean(1, keepdims=True) + np.abs(x)) + np.abs(h)) + np.abs(b))
    return h * w + b, m[:, 0], r[:, 0], bound


def _check(got, want, bound, dtype, label):
    got = got.double().cpu().numpy()
    if dtype == torch.bfloat16:
        bound = bound + HALF_BF16 * (np.abs(want) + bound)
    worst = np.max(np.abs(got - want) / (bound + 1e-40)) if got.size else 0.0
    print(f"[layer norm] {label}: worst error / bound {worst:.3f}", flush=True)
    assert np.all(np.abs(got - want) <= bound + 1e-40), label


SIZES = [(1, 1), (3, 1), (2, 7), (5, 8), (4, 9), (7, 63), (3, 64), (6, 65), (33, 513), (9, 1000), (17, 2056),
         (5, 5003), (4, 5120), (3, 8192), (2, 16384), (3, 16391), (2, 20480), (2, 33001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_and_backward(rows, cols, dt):
    dtype, eps = DT[dt], 1e-5
    wdtype = torch.float32 if cols % 2 else dtype
    x, dy, w, b = _inputs(rows, cols, dtype, wdtype, rows * 100003 + cols)
    print(f"[layer norm] {rows}x{cols} {dt}", flush=True)
    y, mean, rstd, amax = nv.nvfp4_layer_norm(x, w, b, eps=eps, amax=True)
    want, m, r, bound = _ref_forward(x, w, b, eps)
    _check(y, want, bound, dtype, "y")
    absx = x.double().abs().mean(1).cpu().numpy()
    assert np.all(np.abs(mean.double().cpu().numpy() - m) <= 64 * U * absx + 1e-40)
    assert np.all(np.abs(rstd.double().cpu().numpy() - r) <= 64 * U * r * (1 + (r * absx) ** 2 * 64 * U))
    assert amax.item() == y.float().abs().max().item()
    _check_backward(x, dy, mean, rstd, w)


def _check_backward(x, dy, mean, rstd, w, grad_dtype=torch.float32, **kw):
    dx, dw, db = nv.nvfp4_layer_norm_backward(dy, x, mean, rstd, w, grad_dtype=grad_dtype, **kw)
    rows = x.shape[0]
    xd, d = x.double().cpu().numpy(), dy.double().cpu().numpy()
    m, r = mean.double().cpu().numpy()[:, None], rstd.double().cpu().numpy()[:, None]
    wd = np.ones(x.shape[1]) if w is None else w.double().cpu().numpy()
    h, a = (xd - m) * r, d * wd
    s1, s2 = a.mean(1, keepdims=True), (a * h).mean(1, keepdims=True)
    want = r * (a - s1 - h * s2)
    bound = 64 * U * r * (np.abs(a) + np.abs(a).mean(1, keepdims=True)
                          + 2 * np.abs(h) * np.abs(a * h).mean(1, keepdims=True))
    assert dx.dtype == x.dtype and dw.dtype == grad_dtype and db.dtype == grad_dtype
    _check(dx, want, bound, x.dtype, "dx")
    # h itself is off by 2 roundings
    _check(dw, (d * h).sum(0), (rows + 4) * U * np.abs(d * h).sum(0), grad_dtype, "dweight")
    _check(db, d.sum(0), (rows + 2) * U * np.abs(d).sum(0), grad_dtype, "dbias")
    return dx, dw, db


@pytest.mark.parametrize("xd,yd,wd", [("bf16", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "bf16", "f32"),
                                      ("f32", "f32", "bf16")])
@pytest.mark.parametrize("cols", [264, 20488])
def test_mixed_types(xd, yd, wd, cols):
    rows = 11
    x, _, w, b = _inputs(rows, cols, DT[xd], DT[wd], 5)
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b, out_dtype=DT[yd])
    want, _, _, bound = _ref_forward(x, w, b, 1e-5)
    assert y.dtype == DT[yd]
    _check(y, want, bound, DT[yd], f"{xd} -> {yd}")
    dy = _matrix(torch.randn((rows, cols), generator=torch.Generator().manual_seed(6)), DT[yd])
    _check_backward(x, dy, mean, rstd, w, grad_dtype=DT[wd])


@pytest.mark.parametrize("xd,yd", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", [(3, 8), (5, 9), (4, 77), (40, 515), (7, 2051), (9, 5003)])
def test_mixed_types_odd_widths(xd, yd, rows, cols):
    """Rows of both types that start and end anywhere."""
    x, _, w, b = _inputs(rows, cols, DT[xd], DT[yd], rows + cols, pad=1, shift=1)
    y, mean, rstd, amax = nv.nvfp4_layer_norm(x, w, b, out_dtype=DT[yd], amax=True)
    want, _, _, bound = _ref_forward(x, w, b, 1e-5)
    _check(y, want, bound, DT[yd], f"{xd} -> {yd} {rows}x{cols}")
    assert amax.item() == y.float().abs().max().item()
    dy = _matrix(torch.randn((rows, cols), generator=torch.Generator().manual_seed(8)), DT[yd], 3, 1)
    _check_backward(x, dy, mean, rstd, w, grad_dtype=DT[xd])
    _check_backward(x, dy, mean, rstd, None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(5, 40, 3, 1), (6, 1001, 5, 3), (3, 8191, 1, 0), (2, 17000, 7, 5)])
def test_strides_and_alignment(dt, rows, cols, pad, shift):
    x, dy, w, b = _inputs(rows, cols, DT[dt], torch.float32, 17, pad, shift)
    out = _matrix(torch.zeros(rows, cols), DT[dt], 2, 1)
    base = out._base.clone()
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b, out=out)
    want, _, _, bound = _ref_forward(x, w, b, 1e-5)
    _check(y, want, bound, DT[dt], "y strided")
    # nothing outside the view was written
    mask = torch.ones_like(base, dtype=torch.bool)
    mask[1:].view(rows, cols + 2)[:, :cols] = False
    assert torch.equal(out._base[mask], base[mask])
    _check_backward(x, dy, mean, rstd, w)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_absent_parameters(weight, bias):
    x, dy, w, b = _inputs(9, 777, torch.float32, torch.float32, 23)
    w, b = (w if weight else None), (b if bias else None)
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b)
    want, _, _, bound = _ref_forward(x, w, b, 1e-5)
    _check(y, want, bound, torch.float32, "y")
    _check_backward(x, dy, mean, rstd, w)


def test_many_rows():
    """More rows than workgroups, so each walks several and the partial sums
    of the weight gradient join."""
    x, dy, w, b = _inputs(9001, 136, torch.float32, torch.float32, 29)
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b)
    want, _, _, bound = _ref_forward(x, w, b, 1e-5)
    _check(y, want, bound, torch.float32, "y")
    first = _check_backward(x, dy, mean, rstd, w)
    again = nv.nvfp4_layer_norm_backward(dy, x, mean, rstd, w)
    for p, q in zip(first, again):
        assert torch.equal(p, q)          # the sums' order is fixed


@pytest.mark.parametrize("cols", [511, 2041, 4099, 12293])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_calls(dt, cols):
    """More than the last cache holds: rows do not know of each other, so some
    of them come out bit for bit as in a small call; the sums over all rows
    are checked against float64."""
    rows = 272_000_000 // (4 if dt == "bf16" else 8) // cols
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn((rows, cols), generator=g, device="cuda") * 2 + 0.5).to(DT[dt])
    dy = torch.randn((rows, cols), generator=g, device="cuda").to(DT[dt])
    w, b = torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    print(f"[layer norm] {rows}x{cols} {dt}", flush=True)
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b)
    dx, dw, db = nv.nvfp4_layer_norm_backward(dy, x, mean, rstd, w, grad_dtype=torch.float32)
    for at in (slice(0, 3), slice(rows // 2, rows // 2 + 5), slice(rows - 4, rows)):
        ys, ms, rs = nv.nvfp4_layer_norm(x[at], w, b)
        assert torch.equal(ys, y[at]) and torch.equal(ms, mean[at]) and torch.equal(rs, rstd[at])
        assert torch.equal(nv.nvfp4_layer_norm_backward(dy[at], x[at], ms, rs, w)[0], dx[at])
    sums = torch.zeros((4, cols), dtype=torch.float64, device="cuda")
    for at in range(0, rows, 4096):
        d = dy[at:at + 4096].double()
        h = (x[at:at + 4096].double() - mean[at:at + 4096, None].double()) * rstd[at:at + 4096, None].double()
        sums += torch.stack([(d * h).sum(0), (d * h).abs().sum(0), d.sum(0), d.abs().sum(0)])
    assert torch.all((dw.double() - sums[0]).abs() <= (rows + 4) * U * sums[1])
    assert torch.all((db.double() - sums[2]).abs() <= (rows + 2) * U * sums[3])


def test_large_mean_keeps_the_variance():
    """x = 4096 + noise: the variance is taken about the mean, so its digits
    do not cancel (the bound grows only with the rounding of the mean)."""
    x, _, w, b = _inputs(4, 5120, torch.float32, torch.float32, 31)
    x = (x * 0.1 + 4096).contiguous()
    y, _, rstd = nv.nvfp4_layer_norm(x, w, b)
    want, _, r, bound = _ref_forward(x, w, b, 1e-5)
    _check(y, want, bound, torch.float32, "offset rows")
    # the mean's error e <= 64 u 4096 enters the variance as e^2
    assert np.all(np.abs(rstd.double().cpu().numpy() / r - 1) <= 64 * U + (64 * U * 4096 * r) ** 2)


def test_constant_rows_and_eps():
    x = torch.full((3, 100), 2.5, device="cuda")
    w, b = torch.full((100,), 3.0, device="cuda"), torch.full((100,), -1.0, device="cuda")
    y, mean, rstd = nv.nvfp4_layer_norm(x, w, b, eps=0.25)
    assert torch.all(y == -1.0) and torch.all(mean == 2.5) and torch.all(rstd == 2.0)


@pytest.mark.parametrize("cols", [100, 20000])
def test_non_finite_rows_stay_alone(cols):
    x, dy, w, b = _inputs(6, cols, torch.float32, torch.float32, 37)
    clean, mean, rstd = nv.nvfp4_layer_norm(x, w, b)
    bad = x.clone()
    bad[1, 3], bad[4, cols - 1] = float("nan"), float("inf")
    y, m2, r2, amax = nv.nvfp4_layer_norm(bad, w, b, amax=True)
    assert torch.isnan(y[1]).all() and torch.isnan(y[4]).any() and torch.isnan(amax).all()
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(m2[keep], mean[keep]) and torch.equal(r2[keep], rstd[keep])
    dx0, _, _ = nv.nvfp4_layer_norm_backward(dy, x, mean, rstd, w)
    dx, _, _ = nv.nvfp4_layer_norm_backward(dy, bad, m2, r2, w)
    assert torch.equal(dx[keep], dx0[keep])


def test_no_rows():
    x = torch.empty((0, 48), device="cuda")
    y, mean, rstd, amax = nv.nvfp4_layer_norm(x, amax=True)
    assert y.shape == (0, 48) and mean.numel() == 0 and amax.item() == 0.0
    dx, dw, db = nv.nvfp4_layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 48) and torch.all(dw == 0) and torch.all(db == 0)


def test_maximum_feeds_the_quantizer():
    """quantize_amax with the norm's maximum equals the two-pass quantization
    bit for bit."""
    for dtype in (torch.bfloat16, torch.float32):
        x, _, w, b = _inputs(96, 320, dtype, torch.float32, 41)
        y, _, _, amax = nv.nvfp4_layer_norm(x, w, b, amax=True)
        p, q = nv.nvfp4_quantize_amax(y, amax), nv.nvfp4_quantize(y)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales) and torch.equal(p.meta, q.meta)


@pytest.mark.parametrize("rows,cols", [(9001, 24), (4100, 700), (700, 5003), (600, 16500)])
def test_maximum_over_many_workgroups(rows, cols):
    x, _, w, b = _inputs(rows, cols, torch.bfloat16, torch.float32, 41)
    y, _, _, amax = nv.nvfp4_layer_norm(x, w, b, amax=True)
    assert amax.item() == y.float().abs().max().item()
    for value in (float("inf"), float("nan")):
        x[rows - 1, cols - 1] = value            # the row's mean is not finite then
        assert np.isnan(nv.nvfp4_layer_norm(x, w, b, amax=True)[3].item())
        x[rows - 1, cols - 1] = 0.0
    b[cols // 2] = float("-inf")                 # an infinite output, no NaN
    assert nv.nvfp4_layer_norm(x, w, b, amax=True)[3].item() == float("inf")


def test_gradient_against_differences():
    """The directional derivative of sum(dy * y) from central differences of
    the float64 formula; the kernel's share of the error is its bound, the
    differences' is their step squared."""
    rows, cols, eps = 7, 203, 1e-5
    x, dy, w, b = _inputs(rows, cols, torch.float32, torch.float32, 43)
    _, mean, rstd = nv.nvfp4_layer_norm(x, w, b, eps=eps)
    dx, dw, db = (t.double().cpu().numpy() for t in nv.nvfp4_layer_norm_backward(dy, x, mean, rstd, w))
    xd, wd, bd, d = (t.double().cpu().numpy() for t in (x, w, b, dy))

    def loss(x, w, b):
        m = x.mean(1, keepdims=True)
        return (d * ((x - m) / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps) * w + b)).sum()

    rng = np.random.default_rng(3)
    step = 1e-4
    for which, grad in ((0, dx), (1, dw), (2, db)):
        args = [xd, wd, bd]
        v = rng.standard_normal(args[which].shape)
        lo, hi = list(args), list(args)
        lo[which], hi[which] = args[which] - step * v, args[which] + step * v
        numeric = (loss(*hi) - loss(*lo)) / (2 * step)
        scale = np.abs(grad * v).sum()
        # 1e-6: 64 u of each term's parts, which exceed the terms by less than 4 here; 1e-8 the step squared
        assert abs((grad * v).sum() - numeric) <= (4 * 64 * U + step ** 2) * scale


def test_other_stream():
    x, dy, w, b = _inputs(64, 520, torch.bfloat16, torch.bfloat16, 47)
    want = nv.nvfp4_layer_norm(x, w, b, amax=True)
    grads = nv.nvfp4_layer_norm_backward(dy, x, want[1], want[2], w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.nvfp4_layer_norm(x, w, b, amax=True, stream=side)
    back = nv.nvfp4_layer_norm_backward(dy, x, got[1], got[2], w, stream=side)
    side.synchronize()
    for p, q in zip(want + grads, got + back):
        assert torch.equal(p, q)


def test_graph_replays():
    x, dy, w, b = _inputs(40, 1032, torch.bfloat16, torch.bfloat16, 53)
    nv.nvfp4_layer_norm(x, w, b, amax=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.nvfp4_layer_norm(x, w, b, amax=True)
        back = nv.nvfp4_layer_norm_backward(dy, x, got[1], got[2], w)
    for turn in range(4):
        x.copy_(torch.randn(40, 1032, generator=torch.Generator().manual_seed(turn)).to(torch.bfloat16) * (turn + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = nv.nvfp4_layer_norm(x, w, b, amax=True)
        grads = nv.nvfp4_layer_norm_backward(dy, x, want[1], want[2], w)
        for p, q in zip(want + grads, tuple(got) + tuple(back)):
            assert torch.equal(p, q)


def test_offsets_past_32_bits():
    """2.2e9 elements: sampled rows of both directions."""
    rows, cols = 262600, 8200
    assert rows * cols > 2 ** 31
    block = torch.randn((1313, cols), generator=torch.Generator().manual_seed(59)).to(torch.bfloat16).cuda()
    x = block.repeat(200, 1)
    w = torch.linspace(0.5, 1.5, cols, device="cuda")
    y, mean, rstd, amax = nv.nvfp4_layer_norm(x, w, amax=True)
    dx, _, db = nv.nvfp4_layer_norm_backward(x, x, mean, rstd, w)
    yb, mb, rb, ab = nv.nvfp4_layer_norm(block, w, amax=True)
    dxb, _, _ = nv.nvfp4_layer_norm_backward(block, block, mb, rb, w)
    assert torch.equal(amax, ab)
    for rep in (0, 100, 199):
        s = slice(rep * 1313, (rep + 1) * 1313)
        assert torch.equal(y[s], yb) and torch.equal(dx[s], dxb)
    want = 200 * block.double().sum(0)
    tol = 200 * (rows + 2) * U * block.double().abs().sum(0)
    assert torch.all((db.double() - want).abs() <= tol)
