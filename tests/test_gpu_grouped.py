"""GPU checks of the matrix products grouped by expert, forward, data gradient
(transposed stacks) and weight gradient, against float64.

Products of bf16 values with decoded weights are exact, so an output is off by
the binary32 additions alone, in whatever order: K u sum|x w| with u = 2^-24
(3 K terms where a float32 x goes as three parts), two roundings for the
tensor scale, and half a bf16 step (2^-8 of the value) where it is stored in
bf16.  Small whole numbers (weights times powers of two) have no rounding at
all, and are compared for equality at the larger sizes.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def stack(fmt, outer, k, seed, whole=False):
    """A 4-bit tensor with random codes and scales: (handle, its float64 values)."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (outer, k // 2), generator=g, dtype=torch.uint8)
    if fmt == "nvfp4":
        if whole:
            s8 = torch.tensor([0.5, 1.0, 2.0])[torch.randint(0, 3, (outer, k // 16), generator=g)]
        else:
            s8 = (torch.exp(torch.randn((outer, k // 16), generator=g)) * 20).clamp(max=448)      # (never NaN)
        s8 = s8.to(torch.float8_e4m3fn)
        meta = torch.tensor([2688.0, 1.0]) if whole else torch.tensor([0.37 * 2688, 0.37])
        w = nv.NVFP4Tensor(codes.cuda(), s8.view(torch.uint8).cuda(), meta.cuda(), outer, k)
        s = s8.double() * float(meta[1])
    else:
        e = torch.randint(126, 129, (outer, k // 32), generator=g) if whole else \
            torch.randint(110, 130, (outer, k // 32), generator=g)
        w = nv.MXFP4Tensor(codes.cuda(), e.to(torch.uint8).cuda(), outer, k)
        s = torch.exp2(e.double() - 127)
    q = torch.stack([GRID[(codes & 15).long()], GRID[(codes >> 4).long()]], 2).view(outer, s.shape[1], -1)
    return w, (q * s[..., None]).view(outer, k)


def experts_of(values, experts, transposed):
    """[experts, N, K] of a stack's values."""
    if transposed:
        return values.view(values.shape[0], experts, -1).transpose(0, 1)
    return values.view(experts, -1, values.shape[1])


def offsets_of(sizes, dtype=torch.int32, first=0):
    return torch.tensor([first] + list(first + np.cumsum(sizes)), dtype=dtype, device="cuda")


def product(fmt, w, x, offsets, **kw):
    f = nv.nvfp4_grouped_matmul if fmt == "nvfp4" else nv.mxfp4_grouped_matmul
    return f(w, x, offsets, **kw)


def matrix(values, dtype, pad=0, shift=0):
    rows, cols = values.shape
    flat = torch.full((shift + rows * (cols + pad),), 7.0, dtype=dtype, device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(values.to(dtype))
    return view


def check(y, x, values, sizes, first, out, label):
    """y against float64, group by group, and zeros elsewhere."""
    xd, y = x.double().cpu(), y.double().cpu()
    at, k = first, x.shape[1]
    terms = k if x.dtype == torch.bfloat16 else 3 * k
    worst = 0.0
    assert torch.all(y[:first] == 0) and torch.all(y[first + sum(sizes):] == 0), label
    for e, size in enumerate(sizes):
        rows = xd[at:at + size]
        want, mass = rows @ values[e].t(), rows.abs() @ values[e].abs().t()
        bound = (terms + 3) * U * 1.01 * mass
        if out == torch.bfloat16:
            bound = bound + HALF_BF16 * (want.abs() + bound)
        off = (y[at:at + size] - want).abs()
        worst = max(worst, float((off / (bound + 1e-40)).max()) if off.numel() else 0.0)
        assert torch.all(off <= bound + 1e-40), (label, e)
        at += size
    print(f"[grouped] {label}: worst error / bound {worst:.3f}", flush=True)


# group sizes: none, one row, a few, more than one tile, one group alone
SIZES = [([1], 0, 0), ([0, 1, 0, 3], 0, 2), ([5, 0, 17, 2, 1], 3, 4), ([33, 64, 31], 0, 0), ([200], 0, 0),
         ([0, 0, 150, 1], 1, 1), ([300, 7, 140], 0, 0), ([1] * 70 + [0] * 9 + [2] * 60, 0, 5), ([513, 130], 2, 0)]


@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("transposed", [False, True])
def test_groups(case, fmt, dt, out, transposed):
    sizes, first, rest = SIZES[case]
    experts = len(sizes)
    n, k = (96, 160) if transposed or case % 2 else (83, 288)
    rows = first + sum(sizes) + rest
    print(f"[grouped] {fmt} {sizes[:6]} {n}x{k} {dt} {out} {transposed}", flush=True)
    shape = (n, experts * k) if transposed else (experts * n, k)
    w, values = stack(fmt, *shape, seed=case)
    g = torch.Generator().manual_seed(case)
    x = matrix(torch.randn((rows, k), generator=g), DT[dt], pad=case % 3, shift=case % 2)
    y = product(fmt, w, x, offsets_of(sizes, first=first), out_dtype=DT[out], transposed=transposed)
    assert y.dtype == DT[out] and y.shape == (rows, n)
    check(y, x, experts_of(values, experts, transposed), sizes, first, DT[out], "y")


@pytest.mark.parametrize("fmt,k", [("nvfp4", 16), ("nvfp4", 48), ("nvfp4", 112), ("nvfp4", 128), ("nvfp4", 144),
                                   ("nvfp4", 272), ("nvfp4", 1040), ("mxfp4", 32), ("mxfp4", 96), ("mxfp4", 160),
                                   ("mxfp4", 2080)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[3, 0, 9], [50, 90], [260, 170]])
def test_reductions(fmt, k, dt, sizes):
    """K of every remainder, N of one and of odd counts."""
    for n in (1, 37, 130):
        w, values = stack(fmt, len(sizes) * n, k, seed=k + n)
        x = matrix(torch.randn((sum(sizes), k), generator=torch.Generator().manual_seed(k)), DT[dt], pad=1)
        y = product(fmt, w, x, offsets_of(sizes, torch.int64), out_dtype=torch.float32)
        check(y, x, experts_of(values, len(sizes), False), sizes, 0, torch.float32, f"{fmt} {n}x{k} {dt} {sizes}")


def whole_numbers(rows, cols, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, (rows, cols), generator=g, device="cuda").to(dtype)


LARGE = [("nvfp4", 1000, 5120, [700, 0, 1, 300, 129]), ("mxfp4", 2050, 2080, [1, 2, 0, 16, 17, 15]),
         ("nvfp4", 520, 1296, [2000, 30]), ("mxfp4", 768, 4096, [90, 100, 60]), ("nvfp4", 4100, 1024, [2, 1, 1, 0, 7]),
         ("nvfp4", 64, 24592, [1, 3, 20]), ("mxfp4", 16, 8192, [40, 1])]


@pytest.mark.parametrize("fmt,n,k,sizes", LARGE)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_whole_numbers(fmt, n, k, sizes, dt, transposed):
    """Multiples of 1/4 below 2^20: every product and sum is exact."""
    experts, rows = len(sizes), sum(sizes)
    print(f"[grouped] whole {fmt} {n}x{k} {sizes} {dt} {transposed}", flush=True)
    if transposed:
        n = (n + 31) // 32 * 32
    w, values = stack(fmt, *((n, experts * k) if transposed else (experts * n, k)), seed=n, whole=True)
    values = experts_of(values, experts, transposed).float().cuda()
    x = whole_numbers(rows, k, k, DT[dt])
    y = product(fmt, w, x, offsets_of(sizes), out_dtype=torch.float32, transposed=transposed)
    at = 0
    for e, size in enumerate(sizes):
        want = x[at:at + size].double() @ values[e].double().t()
        assert torch.equal(y[at:at + size].double(), want), (e, size)
        at += size


def test_rows_of_no_group_stay_in_a_given_output():
    sizes, first, rows, n, k = [3, 0, 40], 2, 51, 70, 128
    w, values = stack("nvfp4", 3 * n, k, 1)
    x = torch.randn((rows, k), device="cuda").bfloat16()
    x[:first], x[first + 43:] = float("nan"), float("inf")       # of no group: not read into any
    wide = torch.full((rows, n + 6), 5.0, device="cuda")
    out = wide[:, 2:2 + n]
    y = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes, first=first), out_dtype=torch.float32, out=out)
    assert y is out
    assert torch.all(wide[:first] == 5) and torch.all(wide[first + 43:] == 5)
    assert torch.all(wide[:, :2] == 5) and torch.all(wide[:, 2 + n:] == 5)
    fresh = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes, first=first), out_dtype=torch.float32)
    assert torch.equal(fresh[first:first + 43], out[first:first + 43])
    assert torch.all(fresh[:first] == 0) and torch.all(fresh[first + 43:] == 0)


def test_empty():
    w, _ = stack("nvfp4", 64, 32, 2)
    y = nv.nvfp4_grouped_matmul(w, torch.empty((0, 32), device="cuda"), offsets_of([0, 0]))
    assert y.shape == (0, 32)
    y = nv.nvfp4_grouped_matmul(w, torch.ones((5, 32), device="cuda"), offsets_of([0, 0]))
    assert torch.all(y == 0)
    w = nv.NVFP4Tensor.empty(64, 0)
    w.meta.fill_(float("nan"))
    out = torch.full((3, 32), 9.0, device="cuda")
    nv.nvfp4_grouped_matmul(w, torch.empty((3, 0), device="cuda"), offsets_of([1, 1]), out=out)
    assert torch.all(out[:2] == 0) and torch.all(out[2] == 9)
    dw = nv.nvfp4_grouped_wgrad(torch.empty((0, 40), device="cuda"), torch.empty((0, 24), device="cuda"),
                                offsets_of([0, 0, 0]))
    assert dw.shape == (3, 40, 24) and torch.all(dw == 0)


@pytest.mark.parametrize("sizes", [[2, 1], [200, 300]])
def test_offsets_outside_are_held_inside(sizes):
    """Offsets beyond the rows are taken as the nearest inside."""
    rows, n, k = sum(sizes), 48, 64
    w, _ = stack("nvfp4", 2 * n, k, 3)
    x = torch.randn((rows, k), device="cuda").bfloat16()
    want = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes))
    bad = torch.tensor([-5, sizes[0], rows + 1000], dtype=torch.int64, device="cuda")
    assert torch.equal(nv.nvfp4_grouped_matmul(w, x, bad), want)
    dy = torch.randn((rows, n), device="cuda").bfloat16()
    assert torch.equal(nv.nvfp4_grouped_wgrad(dy, x, bad), nv.nvfp4_grouped_wgrad(dy, x, offsets_of(sizes)))


@pytest.mark.parametrize("sizes", [[3, 2], [100, 60], [300, 170]])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_mxfp4_scales_at_both_ends(sizes, dt):
    """Scales of 2^-127 and 2^127, whose weights pass every 16-bit range, and
    the NaN code, in rows of their own."""
    n, k = 40, 64
    w, _ = stack("mxfp4", 2 * n, k, 4)
    w.scales[0], w.scales[1], w.scales[2], w.scales[3] = 0, 254, 255, 253
    w.scales[4] = 1
    w.scales[5, 0], w.scales[5, 1] = 2, 252
    w.codes[2, :4] = 0
    rows = sum(sizes)
    x = (1 + torch.rand((rows, k), device="cuda", generator=torch.Generator("cuda").manual_seed(5))) * 2.0 ** -20
    x = x.to(DT[dt])
    y = nv.mxfp4_grouped_matmul(w, x, offsets_of(sizes), out_dtype=torch.float32)[:sizes[0]].double().cpu()
    c = w.codes[:n].cpu()
    q = torch.stack([GRID[(c & 15).long()], GRID[(c >> 4).long()]], 2).view(n, 2, 32)
    values = (q * torch.exp2(w.scales[:n].double().cpu() - 127)[..., None]).view(n, k)
    xd = x[:sizes[0]].double().cpu()
    want, mass = xd @ values.t(), xd.abs() @ values.abs().t()
    assert torch.isnan(y[:, 2]).all()
    keep = [i for i in range(n) if i != 2]
    # (a product below 2^-126 is off by a binary32 denormal step at most, 2^-149)
    bound = 3 * (k + 3) * U * 1.01 * mass + 6 * k * 2.0 ** -149
    assert torch.all((y - want).abs()[:, keep] <= bound[:, keep])


def test_infinite_and_nan_activations_stay_in_their_rows():
    for sizes in ([4, 3], [70, 80], [300, 200]):
        for dt in ("bf16", "f32"):
            rows, n, k = sum(sizes), 40, 160
            w, _ = stack("nvfp4", 2 * n, k, 6)
            x = torch.randn((rows, k), device="cuda").to(DT[dt])
            want = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes))
            x[1, 5], x[sizes[0], k - 1] = float("nan"), float("inf")
            y = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes))
            bad = [1, sizes[0]]
            good = [i for i in range(rows) if i not in bad]
            assert torch.equal(y[good], want[good])
            assert torch.isnan(y[1]).all() and not torch.isfinite(y[sizes[0]]).all()


# ----------------------------------------------------------- weight gradient --

WGRAD = [([1], 1, 1, 0, 0), ([0, 5, 1], 33, 70, 2, 1), ([40, 0, 64, 31], 130, 65, 0, 3), ([129, 300], 257, 130, 1, 0),
         ([16] * 20, 64, 64, 0, 0)]


@pytest.mark.parametrize("sizes,n,k,first,rest", WGRAD)
@pytest.mark.parametrize("dd,xd", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wgrad(sizes, n, k, first, rest, dd, xd, out):
    """Sums of `rows` products (up to 6 partial ones each), a product off by
    2^-23 of its magnitude where an operand is float32."""
    rows = first + sum(sizes) + rest
    print(f"[grouped] wgrad {sizes[:5]} {n}x{k} {dd} {xd}", flush=True)
    g = torch.Generator().manual_seed(n)
    dy = matrix(torch.randn((rows, n), generator=g), DT[dd], pad=1)
    x = matrix(torch.randn((rows, k), generator=g), DT[xd], pad=2, shift=1)
    dw = nv.nvfp4_grouped_wgrad(dy, x, offsets_of(sizes, first=first), grad_dtype=DT[out])
    assert dw.dtype == DT[out] and dw.shape == (len(sizes), n, k)
    narrow = dd == xd == "bf16"
    at = first
    for e, size in enumerate(sizes):
        d, xx = dy[at:at + size].double().cpu(), x[at:at + size].double().cpu()
        want, mass = d.t() @ xx, d.abs().t() @ xx.abs()
        bound = ((size if narrow else 6 * size) * U + (0 if narrow else 2 * U)) * 1.01 * mass
        if out == "bf16":
            bound = bound + HALF_BF16 * (want.abs() + bound)
        assert torch.all((dw[e].double().cpu() - want).abs() <= bound + 1e-40), e
        at += size


@pytest.mark.parametrize("n,k,sizes", [(1283, 2050, [50, 0, 61, 700]), (512, 768, [2000, 1]), (256, 256, [64, 64, 63])])
@pytest.mark.parametrize("dd,xd", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_wgrad_whole_numbers(n, k, sizes, dd, xd):
    rows = sum(sizes)
    dy, x = whole_numbers(rows, n, n, DT[dd]), whole_numbers(rows, k, k, DT[xd])
    dw = nv.nvfp4_grouped_wgrad(dy, x, offsets_of(sizes))
    at = 0
    for e, size in enumerate(sizes):
        assert torch.equal(dw[e].double(), dy[at:at + size].double().t() @ x[at:at + size].double()), e
        at += size


def test_wgrad_extremes_of_float32():
    """Infinities, NaN, denormals and the largest values as operands.  An
    infinity meets the zero parts of the other operand, so that its products
    are infinite or NaN (inf * 0)."""
    big = 3.4e38
    dy = torch.tensor([[1.0, big, float("inf"), 2.0 ** -130]], device="cuda")
    x = torch.tensor([[1.0, -0.5, float("nan"), big, 2.0 ** -100]], device="cuda")
    dw = nv.nvfp4_grouped_wgrad(dy, x, offsets_of([1]))[0].double().cpu()
    want = dy[0].double().cpu()[:, None] * x[0].double().cpu()[None]
    assert torch.isnan(dw[:, 2]).all()
    assert not torch.isfinite(dw[2]).any() and torch.isinf(dw[1, 3])
    for i, j in ((0, 0), (0, 1), (0, 3), (0, 4), (1, 0), (1, 1), (1, 4)):
        assert abs(dw[i, j] - want[i, j]) <= 8 * U * abs(want[i, j])
    # a denormal operand keeps what binary32 has of it at most
    assert abs(dw[3, 0] - want[3, 0]) <= 2.0 ** -130


@pytest.mark.parametrize("sizes", [[3, 1, 0, 6], [150, 20, 90]])
def test_streams_and_graphs(sizes):
    rows, n, k = sum(sizes), 192, 256
    w, _ = stack("nvfp4", len(sizes) * n, k, 7)
    x = torch.randn((rows, k), device="cuda").bfloat16()
    dy = torch.randn((rows, n), device="cuda").bfloat16()
    offsets = offsets_of(sizes)
    want, wantw = nv.nvfp4_grouped_matmul(w, x, offsets), nv.nvfp4_grouped_wgrad(dy, x, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, dw = nv.nvfp4_grouped_matmul(w, x, offsets, stream=side), nv.nvfp4_grouped_wgrad(dy, x, offsets, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(dw, wantw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = nv.nvfp4_grouped_matmul(w, x, offsets), nv.nvfp4_grouped_wgrad(dy, x, offsets)
    for _ in range(3):                              # the same graph for groups of other sizes, too
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, nv.nvfp4_grouped_matmul(w, x, offsets))
        assert torch.equal(dw, nv.nvfp4_grouped_wgrad(dy, x, offsets))
        offsets[1:-1] = offsets[1:-1].flip(0).sort().values // 2


@pytest.mark.parametrize("n,k,sizes", [(128, 128, [2735]), (144, 4411, [1000, 524]), (2, 6, [5000, 0, 3]),
                                       (130, 258, [900, 33, 900])])
@pytest.mark.parametrize("dd,xd", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("pad", [0, 1])
def test_wgrad_of_few_tiles(n, k, sizes, dd, xd, pad):
    """Long groups of a small gradient, whose tokens are shared out."""
    rows = sum(sizes) + 4
    dy, x = matrix(whole_numbers(rows, n, n, DT[dd]), DT[dd], pad, pad), matrix(whole_numbers(rows, k, k, DT[xd]), DT[xd], pad)
    dy[:3], x[-1] = float("nan"), float("nan")
    dw = nv.nvfp4_grouped_wgrad(dy, x, offsets_of(sizes, first=3))
    at = 3
    for e, size in enumerate(sizes):
        assert torch.equal(dw[e].double(), dy[at:at + size].double().t() @ x[at:at + size].double()), e
        at += size
