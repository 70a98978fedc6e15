"""GPU checks of the RMS norm with the residual's addition, forward (f32, bf16,
MXFP8) and backward, against the definition in float64, element by element,
within error bounds derived from binary32 arithmetic (u = 2^-24).

Forward: h is the binary32 sum rounded once more to its type, compared bit for
bit.  The sum of squares goes through at most 60 roundings after each other,
which halve in rstd; with its root, its reciprocal and two products an output
is off by at most 64 u |y|, and half a bf16 step (2^-8 of the value) where it
is stored in bf16.  MXFP8 is compared bit for bit with the quantizer's result
for the binary32 products (h w) r.
Backward: with a = dy w and n = h r one sum in at most 60 roundings,
    64 u (r (|a| + 2 |n| mean|a n|) + |dh|)
and the sums over rows in whatever order (rows + 4) u sum|.|.
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


def _values(rows, cols, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * size
    return x * (1 + 30 * (torch.rand((1, cols), generator=g) < 0.02))


def _check(got, want, bound, dtype, label):
    got = got.double().cpu().numpy()
    if dtype == torch.bfloat16:
        bound = bound + HALF_BF16 * (np.abs(want) + bound)
    worst = np.max(np.abs(got - want) / (bound + 1e-40)) if got.size else 0.0
    print(f"[rms norm] {label}: worst error / bound {worst:.3f}", flush=True)
    assert np.all(np.abs(got - want) <= bound + 1e-40), label


def _check_forward(x, w, res, eps, out):
    """One call against the definition; out: a dtype, or "mxfp8"."""
    rows, cols = x.shape
    before = None if res is None else res.clone()
    if out == "mxfp8":
        y, rstd, *rest = nv.mxfp8_rms_norm(x, w, res, eps=eps)
    else:
        y, rstd, *rest = nv.nvfp4_rms_norm(x, w, res, eps=eps, out_dtype=out)
    h = x
    if res is not None:
        h, = rest
        assert torch.equal(res, before)
        assert h.dtype == res.dtype and torch.equal(h, (x.float() + res.float()).to(res.dtype))
    hd = h.double().cpu().numpy()
    r = 1 / np.sqrt((hd * hd).mean(1) + eps)
    assert np.all(np.abs(rstd.double().cpu().numpy() - r) <= 64 * U * r)
    if out == "mxfp8":
        wf = torch.ones(cols, device="cuda") if w is None else w.float()
        want = nv.mxfp8_quantize(((h.float() * wf) * rstd[:, None]).contiguous())
        assert torch.equal(y.codes, want.codes) and torch.equal(y.scales, want.scales)
        return
    wd = np.ones(cols) if w is None else w.double().cpu().numpy()
    want = hd * wd * r[:, None]
    assert y.dtype == out
    _check(y, want, 64 * U * np.abs(want), out, "y")


SIZES = [(1, 1), (3, 1), (2, 7), (5, 8), (4, 9), (7, 63), (3, 64), (6, 65), (33, 513), (9, 1000), (17, 2056),
         (5, 5003), (4, 5120), (3, 8192), (2, 16384), (3, 16391), (2, 20480), (2, 24577), (2, 33001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward(rows, cols, dt):
    print(f"[rms norm] {rows}x{cols} {dt}", flush=True)
    x = _matrix(_values(rows, cols, cols), DT[dt])
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(1))).to(DT[dt]).cuda()
    for res in (None, "bf16", "f32"):
        r = None if res is None else _matrix(_values(rows, cols, cols + 1, 3.0), DT[res])
        for out in (torch.bfloat16, torch.float32):
            _check_forward(x, w, r, 1e-6, out)


MX_SIZES = [(1, 32), (3, 64), (5, 96), (2, 544), (33, 2048), (7, 2080), (4, 5120), (2, 16416), (3, 20480), (2, 24608),
            (2, 32800)]


@pytest.mark.parametrize("rows,cols", MX_SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_mxfp8(rows, cols, dt):
    print(f"[rms norm] mxfp8 {rows}x{cols} {dt}", flush=True)
    v = _values(rows, cols, cols)
    v[0, :32] = 0                                    # a block of zeros, one of -0.0, one of tiny values
    if cols > 64:
        v[0, 32:64] = -0.0
        v[0, 64:96] *= 1e-12
    x = _matrix(v, DT[dt], pad=3)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(1))).cuda()
    for res in (None, "bf16", "f32"):
        r = None if res is None else _matrix(_values(rows, cols, cols + 1, 3.0), DT[res], pad=1)
        _check_forward(x, w, r, 1e-6, "mxfp8")


@pytest.mark.parametrize("cols", [264, 5120, 20480, 33024])
@pytest.mark.parametrize("wd", [None, "bf16", "f32"])
def test_strides_shifts_and_weights(cols, wd):
    w = None if wd is None else (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(2))).to(
        DT[wd]).cuda()
    for dt, pad, shift in (("bf16", 5, 1), ("f32", 3, 1), ("bf16", 8, 8)):
        x = _matrix(_values(4, cols, 3), DT[dt], pad, shift)
        res = _matrix(_values(4, cols, 4), DT["f32" if pad == 5 else "bf16"], pad + 2, shift)
        _check_forward(x, w, res, 1e-5, torch.bfloat16)
        _check_forward(x, w, None, 0.0, torch.float32)
        if cols % 32 == 0:
            _check_forward(x, w, res, 1e-5, "mxfp8")


@pytest.mark.parametrize("rows,cols", [(1, 5120), (700, 264), (300, 5003), (5, 20480), (3, 33001), (9, 3)])
@pytest.mark.parametrize("rd", ["bf16", "f32"])
def test_residual_in_place_and_given_outputs(rows, cols, rd):
    """h in the residual's place and y in a window of a wider buffer: the same
    bits, and nothing beside them is touched."""
    x = _matrix(_values(rows, cols, 5), torch.bfloat16)
    res = _matrix(_values(rows, cols, 6), DT[rd], pad=4)
    w = torch.rand(cols, generator=torch.Generator().manual_seed(7)).cuda()
    y, rstd, h = nv.nvfp4_rms_norm(x, w, res)
    wide = torch.full((rows, cols + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 4:4 + cols]
    stream = res._base
    y2, rstd2, h2 = nv.nvfp4_rms_norm(x, w, res, out=out, residual_out=res)
    assert y2 is out and h2 is res
    assert torch.equal(out, y) and torch.equal(rstd2, rstd) and torch.equal(res, h)
    assert torch.all(wide[:, :4] == 5) and torch.all(wide[:, 4 + cols:] == 5)
    assert torch.all(stream.view(rows, cols + 4)[:, cols:] == 7)


def test_no_rows_and_non_finite_rows():
    w = torch.ones(96, device="cuda")
    y, rstd = nv.nvfp4_rms_norm(torch.empty((0, 96), device="cuda"), w)
    assert y.shape == (0, 96) and rstd.shape == (0,)
    q, rstd = nv.mxfp8_rms_norm(torch.empty((0, 96), device="cuda"), w)
    assert q.codes.shape == (0, 96)
    dx, dw = nv.nvfp4_rms_norm_backward(torch.empty((0, 96), device="cuda"), torch.empty((0, 96), device="cuda"),
                                        torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 96) and torch.all(dw == 0)
    x = torch.randn((5, 96), generator=torch.Generator().manual_seed(8)).cuda()
    want, _ = nv.nvfp4_rms_norm(x, w)
    x[1, 3], x[3, 95] = float("nan"), float("inf")
    y, rstd = nv.nvfp4_rms_norm(x, w)
    assert torch.equal(y[[0, 2, 4]], want[[0, 2, 4]])
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 95]) and torch.all(y[3, :95] == 0)
    q, _ = nv.mxfp8_rms_norm(x, w)
    fine, _ = nv.mxfp8_rms_norm(x[[0, 2, 4]].contiguous(), w)
    assert torch.equal(q.codes[[0, 2, 4]], fine.codes)


def _check_backward(dy, h, rstd, w, dh, grad_dtype=torch.float32, **kw):
    rows, cols = h.shape
    dx, dw = nv.nvfp4_rms_norm_backward(dy, h, rstd, w, dh=dh, grad_dtype=grad_dtype, **kw)
    hd, d = h.double().cpu().numpy(), dy.double().cpu().numpy()
    r = rstd.double().cpu().numpy()[:, None]
    wd = np.ones(cols) if w is None else w.double().cpu().numpy()
    e = 0.0 if dh is None else dh.double().cpu().numpy()
    n, a = hd * r, d * wd
    want = r * (a - n * (a * n).mean(1, keepdims=True)) + e
    bound = 64 * U * (r * (np.abs(a) + 2 * np.abs(n) * np.abs(a * n).mean(1, keepdims=True)) + np.abs(e))
    assert dx.dtype == h.dtype and dw.dtype == grad_dtype
    _check(dx, want, bound, h.dtype, "dx")
    _check(dw, (d * n).sum(0), (rows + 4) * U * np.abs(d * n).sum(0), grad_dtype, "dweight")


BACK_SIZES = SIZES + [(40, 5120), (600, 264), (300, 5120), (1537, 515), (40, 20480), (6, 5120)]


@pytest.mark.parametrize("rows,cols", BACK_SIZES)
@pytest.mark.parametrize("hd,dd", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward(rows, cols, hd, dd):
    print(f"[rms norm] backward {rows}x{cols} {hd} {dd}", flush=True)
    h = _matrix(_values(rows, cols, cols), DT[hd], pad=cols % 3)
    dy = _matrix(1e-3 * _values(rows, cols, cols + 2), DT[dd], pad=1)
    dh = _matrix(1e-3 * _values(rows, cols, cols + 3), DT[hd], pad=2)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(9))).to(DT[dd]).cuda()
    rstd = torch.rsqrt((h.float() ** 2).mean(1) + 1e-6)
    _check_backward(dy, h, rstd, w, dh)
    _check_backward(dy, h, rstd, w if cols % 2 else None, None, grad_dtype=DT[dd])


def test_gradients_are_those_of_the_forward_pass():
    """Differences of the float64 definition of sum(y dy) + sum(h dh) along
    random directions: two-sided differences of step t are off by t^2 times a
    third derivative (here below 1e-6 of the value)."""
    rows, cols, eps = 7, 96, 1e-3
    g = torch.Generator().manual_seed(10)
    x, res, dy, dh = (torch.randn((rows, cols), generator=g).double() for _ in range(4))
    w = 1 + 0.3 * torch.randn(cols, generator=g).double()
    f = [t.float().cuda() for t in (x, res, w, dy, dh)]
    x, res, w, dy, dh = (t.double().cpu() for t in f)

    def loss(x, res, w):
        h = x + res
        return float((h * w / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * dy).sum() + (h * dh).sum())

    _, rstd, h = nv.nvfp4_rms_norm(f[0], f[2], f[1], eps=eps)
    dx, dw = nv.nvfp4_rms_norm_backward(f[3], h, rstd, f[2], dh=f[4])
    t = 1e-4
    for grad, at in ((dx, 0), (dx, 1), (dw, 2)):
        args = [x, res, w]
        u = torch.randn(args[at].shape, generator=g).double()
        plus, minus = list(args), list(args)
        plus[at], minus[at] = args[at] + t * u, args[at] - t * u
        want = (loss(*plus) - loss(*minus)) / (2 * t)
        got = float((grad.double().cpu() * u).sum())
        scale = float((grad.double().cpu() * u).abs().sum())
        assert abs(got - want) <= 2e-6 * scale


def test_another_stream_and_a_graph():
    x = _matrix(_values(64, 5120, 11), torch.bfloat16)
    res = _matrix(_values(64, 5120, 12), torch.float32)
    dy = _matrix(_values(64, 5120, 13), torch.bfloat16).float()
    w = torch.rand(5120, device="cuda")
    want = nv.nvfp4_rms_norm(x, w, res)
    want8 = nv.mxfp8_rms_norm(x, w, res)
    wantb = nv.nvfp4_rms_norm_backward(dy, want[2], want[1], w, dh=want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.nvfp4_rms_norm(x, w, res, stream=side)
    got8 = nv.mxfp8_rms_norm(x, w, res, stream=side)
    gotb = nv.nvfp4_rms_norm_backward(dy, want[2], want[1], w, dh=want[2], stream=side)
    side.synchronize()

    def same(got, got8, gotb):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(got8[0].codes, want8[0].codes) and torch.equal(got8[0].scales, want8[0].scales)
        assert all(torch.equal(a, b) for a, b in zip(gotb, wantb))

    same(got, got8, gotb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.nvfp4_rms_norm(x, w, res)
        got8 = nv.mxfp8_rms_norm(x, w, res)
        gotb = nv.nvfp4_rms_norm_backward(dy, want[2], want[1], w, dh=want[2])
    for _ in range(3):
        for t in (*got, got8[0].codes, got8[0].scales, *gotb):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(got, got8, gotb)
        nv.nvfp4_rms_norm(x, w, res)
