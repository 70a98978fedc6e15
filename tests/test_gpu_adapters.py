"""GPU checks of the low-rank adapters of many requests, forward and backward,
against float64.

With u = 2^-24: u = A x is a sum of K products, each exact for bf16 operands
and off by 2 u of its magnitude where both are float32 (in 6 partial products
then, 3 with one float32 operand), added in binary32 in whatever order:
(P K + 2) u sum|a x|, P = 1, 3 or 6.  y adds the same of a sum over the rank
(always with the float32 u), the error of the u that it starts from (compared
with the u returned, so none), the scale and the base; stored in bf16 half a
step more, 2^-8 of the value.  Small whole numbers have no rounding at all.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def matrix(values, dtype, pad=0, shift=0):
    rows, cols = values.shape
    flat = torch.full((shift + rows * (cols + pad),), 7.0, dtype=dtype, device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(values.to(dtype))
    return view


def parts(*dtypes):
    wide = sum(d == torch.float32 for d in dtypes)
    return {0: 1, 1: 3, 2: 6}[wide]


def near(got, want, mass, terms, label):
    """Within `terms` binary32 roundings of the magnitudes, and half a step of
    a bf16 result."""
    bound = terms * U * 1.01 * mass
    if got.dtype == torch.bfloat16:
        bound = bound + HALF_BF16 * (want.abs() + bound)
    off = (got.double().cpu() - want).abs()
    worst = float((off / (bound + 1e-40)).max()) if off.numel() else 0.0
    print(f"[adapters] {label}: worst error / bound {worst:.3f}", flush=True)
    assert torch.all(off <= bound + 1e-40), label


def setup(sizes, index, first, rest, n, k, rank, adapters, dt, wdt, seed, index_type=torch.int32, pad=0):
    g = torch.Generator().manual_seed(seed)
    rows = first + sum(sizes) + rest
    x = matrix(torch.randn((rows, k), generator=g), DT[dt], pad, pad % 2)
    dy = matrix(torch.randn((rows, n), generator=g), DT[dt], pad)
    a = (torch.randn((adapters, rank, k), generator=g) / k ** 0.5).to(DT[wdt]).cuda()
    b = torch.randn((adapters, n, rank), generator=g).to(DT[wdt]).cuda()
    scale = (0.5 + torch.rand(adapters, generator=g)).cuda()
    offsets = torch.tensor([first] + list(first + np.cumsum(sizes)), dtype=index_type, device="cuda")
    return x, dy, a, b, scale, offsets, torch.tensor(index, dtype=index_type, device="cuda")


def rows_of(sizes, index, first, adapters):
    """[(begin, end, adapter or None)] of the segments."""
    ends = first + np.cumsum([0] + list(sizes))
    return [(int(s), int(e), i if 0 <= i < adapters else None) for s, e, i in zip(ends[:-1], ends[1:], index)]


def check_forward(x, a, b, scale, base, y, u, segments):
    rows, k = x.shape
    rank = a.shape[1]
    xd, ad, bd = x.double().cpu(), a.double().cpu(), b.double().cpu()
    sd = torch.ones(a.shape[0]).double() if scale is None else scale.double().cpu()
    ud, want_u, mass_u = u.double().cpu(), torch.zeros((rows, rank)).double(), torch.zeros((rows, rank)).double()
    want = torch.zeros(y.shape).double() if base is None else base.double().cpu()
    mass = want.abs()
    for s, e, i in segments:
        if i is None:
            continue
        want_u[s:e], mass_u[s:e] = xd[s:e] @ ad[i].t(), xd[s:e].abs() @ ad[i].abs().t()
        want[s:e] += sd[i] * (ud[s:e] @ bd[i].t())
        mass[s:e] += sd[i] * (ud[s:e].abs() @ bd[i].abs().t())
    near(u, want_u, mass_u, parts(x.dtype, a.dtype) * k + 4, "u")
    near(y, want, mass, parts(torch.float32, b.dtype) * rank + 6, "y")


def check_backward(dy, x, u, a, b, scale, base, dx, da, db, segments, count):
    rows, k = x.shape
    n, rank = b.shape[1], a.shape[1]
    xd, dyd, ud, ad, bd = (t.double().cpu() for t in (x, dy, u, a, b))
    sd = torch.ones(a.shape[0]).double() if scale is None else scale.double().cpu()
    want = torch.zeros(dx.shape).double() if base is None else base.double().cpu()
    mass = want.abs()
    wa, ma = torch.zeros(a.shape).double(), torch.zeros(a.shape).double()
    wb, mb = torch.zeros(b.shape).double(), torch.zeros(b.shape).double()
    for s, e, i in segments:
        if i is None:
            continue
        g, mg = sd[i] * (dyd[s:e] @ bd[i]), sd[i] * (dyd[s:e].abs() @ bd[i].abs())
        want[s:e] += g @ ad[i]
        mass[s:e] += mg @ ad[i].abs()
        wa[i] += g.t() @ xd[s:e]
        ma[i] += mg.t() @ xd[s:e].abs()
        wb[i] += sd[i] * dyd[s:e].t() @ ud[s:e]
        mb[i] += sd[i] * dyd[s:e].abs().t() @ ud[s:e].abs()
    # g's own error enters dx and da in full
    of_g = parts(dy.dtype, b.dtype) * n + 4
    near(dx, want, mass, of_g + parts(torch.float32, a.dtype) * rank + 6, "dx")
    near(da, wa, ma, of_g + parts(torch.float32, x.dtype) * count + 6, "da")
    near(db, wb, mb, parts(torch.float32, dy.dtype) * count + 6, "db")


# sizes, index (adapter or none), rows in front and behind, adapters
SEGMENTS = [([1], [0], 0, 0, 1), ([1, 1, 1], [2, 0, 1], 0, 0, 3), ([1, 0, 5, 2], [1, 0, -1, 7], 2, 3, 3),
            ([17, 16, 33], [0, 1, 0], 0, 1, 2), ([100, 1, 300], [3, 3, 0], 1, 0, 5), ([70, 200], [-1, 1], 0, 0, 2),
            ([1] * 130 + [3] * 5, list(range(130)) + [0, 1, 2, 0, -1], 0, 2, 140), ([600], [1], 5, 9, 2)]
# n, k, rank
SIZES = [(96, 128, 16), (83, 131, 8), (300, 257, 5), (64, 520, 33), (257, 64, 64), (40, 100, 128), (1, 1, 1),
         (130, 700, 24)]


@pytest.mark.parametrize("case", range(len(SEGMENTS)))
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_forward_and_backward(case, dt, wdt):
    sizes, index, first, rest, adapters = SEGMENTS[case]
    for j in range(3):
        n, k, rank = SIZES[(case + 3 * j) % len(SIZES)]
        print(f"[adapters] {sizes[:5]} {index[:5]} {n}x{k} rank {rank} {dt} {wdt}", flush=True)
        x, dy, a, b, scale, offsets, which = setup(sizes, index, first, rest, n, k, rank, adapters, dt, wdt, case,
                                                   torch.int64 if j == 1 else torch.int32, pad=j)
        segments = rows_of(sizes, index, first, adapters)
        rows = x.shape[0]
        g = torch.Generator().manual_seed(99)
        base = None if j == 2 else matrix(torch.randn((rows, n), generator=g), DT[dt if j else "f32"], 1)
        sc = None if j == 1 else scale
        y, u = nv.nvfp4_adapters(x, a, b, offsets, which, sc, base=base, out_dtype=DT["f32" if j == 0 else dt])
        assert y.shape == (rows, n) and u.shape == (rows, rank)
        check_forward(x, a, b, sc, base, y, u, segments)
        below = None if j == 0 else matrix(torch.randn((rows, k), generator=g), DT["f32" if j == 2 else dt], 2)
        grad = DT["bf16" if j == 1 else "f32"]
        dx, da, db = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, sc, base=below, grad_dtype=grad)
        assert dx.dtype == x.dtype and da.dtype == db.dtype == grad
        check_backward(dy, x, u, a, b, sc, below, dx, da, db, segments, rows)


@pytest.mark.parametrize("n,k,rank,sizes,adapters", [(5120, 5120, 16, [1] * 24, 32), (2050, 5003, 64, [40, 0, 300, 7], 3),
                                                     (20480, 1024, 32, [2500], 2), (512, 20480, 8, [1, 700, 64], 40)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_whole_numbers(n, k, rank, sizes, adapters, dt):
    """Sums below 2^24 of whole numbers are exact, whatever their order."""
    g = torch.Generator(device="cuda").manual_seed(n)

    def draw(*shape, most=1):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(DT[dt])

    rows = sum(sizes)
    print(f"[adapters] whole {n}x{k} rank {rank} {dt}", flush=True)
    x, dy, a, b = draw(rows, k), draw(rows, n), draw(adapters, rank, k), draw(adapters, n, rank)
    a *= (torch.rand(a.shape, device="cuda", generator=g) < 0.2)       # so that products of three stay below 2^24
    b *= (torch.rand(b.shape, device="cuda", generator=g) < 0.2)
    scale = torch.full((adapters,), 0.5, device="cuda")
    index = [(7 * i) % adapters for i in range(len(sizes))]
    offsets = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    which = torch.tensor(index, dtype=torch.int32, device="cuda")
    base, below = draw(rows, n), draw(rows, k)
    y, u = nv.nvfp4_adapters(x, a, b, offsets, which, scale, base=base, out_dtype=torch.float32)
    dx, da, db = nv.nvfp4_adapters_backward(dy.float(), x.float(), u, a, b, offsets, which, scale, base=below)
    wy, wdx = base.double(), below.double()
    wa, wb = torch.zeros(a.shape, device="cuda").double(), torch.zeros(b.shape, device="cuda").double()
    wu = torch.zeros(u.shape, device="cuda").double()
    for s, e, i in rows_of(sizes, index, 0, adapters):
        wu[s:e] = x[s:e].double() @ a[i].double().t()
        wy[s:e] += 0.5 * wu[s:e] @ b[i].double().t()
        gg = 0.5 * dy[s:e].double() @ b[i].double()
        wdx[s:e] += gg @ a[i].double()
        wa[i] += gg.t() @ x[s:e].double()
        wb[i] += 0.5 * dy[s:e].double().t() @ wu[s:e]
    for got, want in ((u, wu), (y, wy), (dx, wdx), (da, wa), (db, wb)):
        assert float(want.abs().max()) < 2 ** 22
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("sizes", [[1, 2, 1, 1], [90, 20, 200, 1]])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_the_place_of_the_base(sizes, dt):
    n, k, rank = 300, 200, 16
    x, dy, a, b, scale, offsets, which = setup(sizes, [1, -1, 0, 1], 2, 3, n, k, rank, 2, dt, dt, 1)
    rows = x.shape[0]
    wide = torch.randn((rows, n + 7), device="cuda").to(DT[dt])
    before, base = wide.clone(), wide[:, 3:3 + n]
    y, u = nv.nvfp4_adapters(x, a, b, offsets, which, scale, base=base)
    out, u2 = nv.nvfp4_adapters(x, a, b, offsets, which, scale, base=base, out=base)
    assert out is base and torch.equal(base, y) and torch.equal(u, u2)
    assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, 3 + n:], before[:, 3 + n:])
    none = slice(2 + sizes[0], 2 + sizes[0] + sizes[1])
    assert torch.equal(y[none], before[none, 3:3 + n]) and torch.equal(y[:2], before[:2, 3:3 + n])
    assert torch.all(u[none] == 0) and torch.all(u[:2] == 0) and torch.all(u[-3:] == 0)
    below = torch.randn((rows, k), device="cuda").to(DT[dt])
    want = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale, base=below)
    got = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale, base=below, out=below)
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and got[0] is below


def test_rows_without_an_adapter_may_hold_anything():
    """NaN and Inf in rows of no segment, or of one without an adapter, and in
    adapters that no segment has, reach nothing."""
    sizes, index = [3, 40, 5], [0, -1, 2]
    x, dy, a, b, scale, offsets, which = setup(sizes, index, 4, 6, 90, 70, 8, 4, "bf16", "bf16", 2)
    u = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[1]
    want = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[0], *nv.nvfp4_adapters_backward(
        dy, x, u, a, b, offsets, which, scale)
    for t in (x, dy):
        t[:4], t[7:47], t[-6:] = float("nan"), float("inf"), float("nan")
    for t in (a, b):
        t[1], t[3] = float("nan"), float("inf")
    u[7:47] = float("nan")
    got = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[0], *nv.nvfp4_adapters_backward(
        dy, x, u, a, b, offsets, which, scale)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.all(got[2][1] == 0) and torch.all(got[2][3] == 0) and torch.all(got[3][1] == 0)


@pytest.mark.parametrize("rows", [3, 600, 2000])
@pytest.mark.parametrize("rank", [8, 40, 100])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_scale_of_an_unused_adapter_reaches_nothing(rows, rank, dt):
    """Scales of NaN and Inf where no segment has the adapter, or an empty one
    has it: zeros, and the others' results unchanged.  Below 512 rows a sum
    over them is one share, above it is cut."""
    x, dy, a, b, scale, offsets, which = setup([rows, 0], [1, 3], 0, 1, 90, 70, rank, 5, dt, dt, 6)
    u = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[1]
    want = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[0], *nv.nvfp4_adapters_backward(
        dy, x, u, a, b, offsets, which, scale)
    scale[0], scale[2], scale[3], scale[4] = float("nan"), float("inf"), float("nan"), float("-inf")
    got = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[0], *nv.nvfp4_adapters_backward(
        dy, x, u, a, b, offsets, which, scale)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for unused in (0, 2, 3, 4):
        assert torch.all(got[2][unused] == 0) and torch.all(got[3][unused] == 0)


def test_an_infinite_scale_with_an_idle_share():
    """An adapter of one stage of rows beside one of many, whose sums are cut:
    the shares without rows of it add zeros to its infinite gradient."""
    x, dy, a, b, scale, offsets, which = setup([20, 700], [0, 1], 0, 0, 90, 70, 8, 2, "bf16", "bf16", 7)
    u = nv.nvfp4_adapters(x, a, b, offsets, which, scale)[1]
    want = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale)[2]
    scale[0] = float("inf")
    db = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale)[2]
    assert torch.equal(db[1], want[1]) and torch.isinf(db[0]).all() and torch.equal(db[0] > 0, want[0] > 0)


def test_empty():
    a, b = torch.ones((2, 4, 16), device="cuda"), torch.ones((2, 8, 4), device="cuda")
    offsets, index = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 16), device="cuda")
    y, u = nv.nvfp4_adapters(x, a, b, offsets, index)
    assert y.shape == (0, 8) and u.shape == (0, 4)
    dx, da, db = nv.nvfp4_adapters_backward(y, x, u, a, b, offsets, index)
    assert dx.shape == (0, 16) and torch.all(da == 0) and torch.all(db == 0)
    x = torch.ones((3, 16), device="cuda")                         # rows, but none in a segment
    y, u = nv.nvfp4_adapters(x, a, b, offsets, index)
    assert torch.all(y == 0) and torch.all(u == 0)
    dx, da, db = nv.nvfp4_adapters_backward(y + 1, x, u, a, b, offsets, index, base=x)
    assert torch.equal(dx, x) and torch.all(da == 0) and torch.all(db == 0)


def test_gradients_are_those_of_the_forward_pass():
    """Differences of the float64 definition of sum(y dy) along random
    directions; it is of degree 1 in each argument, so two-sided differences
    are exact up to their rounding."""
    sizes, index = [5, 9, 2], [1, 0, 1]
    x, dy, a, b, scale, offsets, which = setup(sizes, index, 1, 1, 40, 50, 6, 2, "f32", "f32", 3)
    _, u = nv.nvfp4_adapters(x, a, b, offsets, which, scale)
    grads = nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale)
    args = [t.double().cpu() for t in (x, a, b)]
    dyd, sd = dy.double().cpu(), scale.double().cpu()

    def loss(x, a, b):
        return sum(float(sd[i] * ((x[s:e] @ a[i].t()) @ b[i].t() * dyd[s:e]).sum()) for s, e, i in
                   rows_of(sizes, index, 1, 2))

    g = torch.Generator().manual_seed(4)
    for at, grad in enumerate(grads):
        v = torch.randn(args[at].shape, generator=g).double()
        plus, minus = list(args), list(args)
        plus[at], minus[at] = args[at] + v, args[at] - v
        got = float((grad.double().cpu() * v).sum())
        assert abs(got - (loss(*plus) - loss(*minus)) / 2) <= 1e-5 * float((grad.double().cpu() * v).abs().sum())


@pytest.mark.parametrize("sizes", [[1, 1, 0, 1], [200, 31, 90, 7]])
def test_streams_and_graphs(sizes):
    index = [1, 0, 1, -1]
    x, dy, a, b, scale, offsets, which = setup(sizes, index, 0, 2, 320, 260, 16, 2, "bf16", "bf16", 5)

    def both(**kw):
        y, u = nv.nvfp4_adapters(x, a, b, offsets, which, scale, **kw)
        return y, u, *nv.nvfp4_adapters_backward(dy, x, u, a, b, offsets, which, scale, **kw)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):                              # the same graph for other adapters and segments, too
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, both()))
        which.copy_(which.roll(1))
        offsets[1:-1] //= 2
