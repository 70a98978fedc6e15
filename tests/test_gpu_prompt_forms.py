"""GPU checks of the forms that only large calls take: grouped products by tiles
of 512 x 128, the adapters' A product by tiles of 32 rows, and RMS norms that
read past the caches' usual order.  Which sizes reach a form is restated from
the launch rules here, so that a test of a form that moved elsewhere fails.

Small whole numbers (weights times powers of two) have no rounding at all and
are compared for equality; other values as in the tests of the same calls:
binary32 additions in whatever order, K u sum|x w| with u = 2^-24, two roundings
for the tensor scale, half a bf16 step (2^-8) where a result is stored in bf16.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda"
                    if torch.cuda.is_available() else "cpu")


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---------------------------------------------------------- grouped products

def takes_large_tiles(n, k, sizes):
    """bf16 groups of more than 80 rows on average, with tiles for most CUs, whose
    weights the tiles for few rows would read for longer."""
    rows, experts = sum(sizes), len(sizes)
    groups = min(experts, rows)
    reads = (rows // 16 + groups) * n * k * 0.53 / 6.0e6
    rounds = max(1.0, (n + 255) // 256 * (rows // 64 + groups // 2) / (2 * cus()))
    few = k >= 128 and reads < rounds * 1.5 * ((k + 127) // 128)
    each = (rows + groups - 1) // groups
    return not few and each > 80 and 8 * ((n + 511) // 512 * (rows // 128 + groups // 2)) >= 5 * cus()


def stack(fmt, outer, k, seed, whole=False):
    """A 4-bit tensor with random codes and scales: (handle, its float64 values)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (outer, k // 2), generator=g, dtype=torch.uint8, device="cuda")
    if fmt == "nvfp4":
        if whole:
            s8 = torch.tensor([0.5, 1.0, 2.0], device="cuda")[torch.randint(0, 3, (outer, k // 16), generator=g,
                                                                            device="cuda")]
        else:
            s8 = (torch.exp(torch.randn((outer, k // 16), generator=g, device="cuda")) * 20).clamp(max=448)
        s8 = s8.to(torch.float8_e4m3fn)
        meta = torch.tensor([2688.0, 1.0] if whole else [0.37 * 2688, 0.37], device="cuda")
        w = nv.NVFP4Tensor(codes, s8.view(torch.uint8), meta, outer, k)
        s = s8.double() * float(meta[1])
    else:
        e = torch.randint(*((126, 129) if whole else (110, 130)), (outer, k // 32), generator=g, device="cuda")
        w = nv.MXFP4Tensor(codes, e.to(torch.uint8), outer, k)
        s = torch.exp2(e.double() - 127)
    return w, decoded(codes, s)


def decoded(codes, s):
    q = torch.stack([GRID[(codes & 15).long()], GRID[(codes >> 4).long()]], 2).view(codes.shape[0], s.shape[1], -1)
    return (q * s[..., None]).view(codes.shape[0], -1)


def experts_of(values, experts, transposed):
    if transposed:
        return values.view(values.shape[0], experts, -1).transpose(0, 1)
    return values.view(experts, -1, values.shape[1])


def offsets_of(sizes, dtype=torch.int32, first=0):
    return torch.tensor([first] + list(first + np.cumsum(sizes)), dtype=dtype, device="cuda")


def product(fmt, w, x, offsets, **kw):
    f = nv.nvfp4_grouped_matmul if fmt == "nvfp4" else nv.mxfp4_grouped_matmul
    return f(w, x, offsets, **kw)


def placed(values, pad, shift):
    rows, cols = values.shape
    flat = torch.full((shift + rows * (cols + pad),), 7.0, dtype=values.dtype, device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(values)
    return view


# N past whole tiles of 512, K past whole stages of 128, groups past whole tiles
# of 128; K below, at and above a stage
LARGE = [("nvfp4", 4136, 272, [1200, 0, 1, 900, 700]), ("mxfp4", 8200, 2080, [700, 33, 511]),
         ("nvfp4", 20520, 144, [300, 1, 90]), ("mxfp4", 4097, 32, [129, 2300]), ("nvfp4", 5121, 16, [127, 1, 2000]),
         ("nvfp4", 4609, 128, [2559]), ("mxfp4", 4608, 1184, [0, 1000, 0, 1559, 0])]


@pytest.mark.parametrize("fmt,n,k,sizes", LARGE)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (2, 2), (3, 1)])      # x as it lies, with a pitch, at odd places (copied)
def test_whole_numbers(fmt, n, k, sizes, transposed, pad, shift):
    """Multiples of 1/4 below 2^20: every product and sum is exact."""
    assert takes_large_tiles(n, k, sizes)
    experts, rows = len(sizes), sum(sizes)
    print(f"[prompt] whole {fmt} {n}x{k} {sizes} {transposed} {pad}", flush=True)
    w, values = stack(fmt, *((n, experts * k) if transposed else (experts * n, k)), seed=n, whole=True)
    values = experts_of(values, experts, transposed)
    g = torch.Generator(device="cuda").manual_seed(k)
    x = placed(torch.randint(-2, 3, (rows, k), generator=g, device="cuda").bfloat16(), pad, shift)
    y = product(fmt, w, x, offsets_of(sizes), out_dtype=torch.float32, transposed=transposed)
    half = product(fmt, w, x, offsets_of(sizes, torch.int64), transposed=transposed)
    assert torch.equal(half, y.bfloat16())
    at = 0
    for e, size in enumerate(sizes):
        want = x[at:at + size].double() @ values[e].t().contiguous()
        assert torch.equal(y[at:at + size].double(), want), (e, size)
        at += size


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("transposed", [False, True])
def test_values(fmt, transposed):
    """Rows in front of the groups and behind them: zeros, or left as they are in
    a given output, whatever x holds there."""
    n, k, sizes, first, rest = 4136, 288, [1000, 0, 1, 1300, 300], 3, 5
    assert takes_large_tiles(n, k, sizes)
    experts, rows = len(sizes), first + sum(sizes) + rest
    w, values = stack(fmt, *((n, experts * k) if transposed else (experts * n, k)), seed=3)
    values = experts_of(values, experts, transposed)
    x = torch.randn((rows, k), generator=torch.Generator("cuda").manual_seed(4), device="cuda").bfloat16()
    x[:first], x[rows - rest:] = float("nan"), float("inf")
    offsets = offsets_of(sizes, first=first)
    for out in (torch.float32, torch.bfloat16):
        y = product(fmt, w, x, offsets, out_dtype=out, transposed=transposed)
        wide = torch.full((rows, n + 9), 5.0, dtype=out, device="cuda")
        product(fmt, w, x, offsets, out_dtype=out, transposed=transposed, out=wide[:, 2:2 + n])
        inner = slice(first, rows - rest)
        assert torch.equal(wide[inner, 2:2 + n], y[inner])
        assert torch.all(wide[:first] == 5) and torch.all(wide[rows - rest:] == 5)
        assert torch.all(wide[:, :2] == 5) and torch.all(wide[:, 2 + n:] == 5)
        assert torch.all(y[:first] == 0) and torch.all(y[rows - rest:] == 0)
        at = first
        for e, size in enumerate(sizes):
            xd, wd = x[at:at + size].double(), values[e].t().contiguous()
            want, mass = xd @ wd, xd.abs() @ wd.abs()
            bound = (k + 3) * U * 1.01 * mass
            if out == torch.bfloat16:
                bound = bound + HALF_BF16 * (want.abs() + bound)
            assert ((y[at:at + size].double() - want).abs() <= bound + 1e-40).all(), e
            at += size


def test_mxfp4_scales_at_both_ends():
    """Scales of 2^-127 and 2^127, whose weights pass every 16-bit range, and the
    NaN code, in some rows of one expert alone: its tiles go twice."""
    n, k, sizes = 4136, 192, [1400, 1200]
    assert takes_large_tiles(n, k, sizes)
    w, _ = stack("mxfp4", 2 * n, k, 5)
    for row in (0, 31, 517, 4100):                                  # of the first expert, in several tiles and waves
        w.scales[row], w.scales[row + 1, 0], w.scales[row + 2, 3], w.scales[row + 3] = 254, 253, 255, 0
        w.scales[row + 4, 1], w.scales[row + 5, 5] = 1, 2
    w.codes[2, :4] = 0
    x = (1 + torch.rand((sum(sizes), k), device="cuda", generator=torch.Generator("cuda").manual_seed(6))) * 2.0 ** -20
    x = x.bfloat16()
    y = nv.mxfp4_grouped_matmul(w, x, offsets_of(sizes), out_dtype=torch.float32)
    scale = torch.exp2(w.scales.double() - 127)
    scale[w.scales == 255] = float("nan")
    values = experts_of(decoded(w.codes, scale), 2, False)
    at = 0
    for e, size in enumerate(sizes):
        nan = torch.isnan(values[e]).any(1)
        assert int(nan.sum()) == (4 if e == 0 else 0)
        got, xd, wd = y[at:at + size].double(), x[at:at + size].double(), values[e][~nan].t().contiguous()
        assert torch.isnan(got[:, nan]).all()
        want, mass = xd @ wd, xd.abs() @ wd.abs()
        # (a product below 2^-126 is off by a binary32 denormal step at most, 2^-149)
        assert ((got[:, ~nan] - want).abs() <= (k + 3) * U * 1.01 * mass + 2 * k * 2.0 ** -149).all()
        at += size


def test_infinite_and_nan_activations_stay_in_their_rows():
    n, k, sizes = 4136, 160, [1400, 1200]
    assert takes_large_tiles(n, k, sizes)
    w, _ = stack("nvfp4", 2 * n, k, 7)
    x = torch.randn((sum(sizes), k), device="cuda").bfloat16()
    want = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes))
    x[1, 5], x[sizes[0], k - 1] = float("nan"), float("inf")
    y = nv.nvfp4_grouped_matmul(w, x, offsets_of(sizes))
    good = torch.ones(sum(sizes), dtype=torch.bool, device="cuda")
    good[[1, sizes[0]]] = False
    assert torch.equal(y[good], want[good])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[sizes[0]]).all()


def test_captured_and_replayed():
    """The same graph for groups of other lengths."""
    n, k, sizes = 4136, 160, [1400, 0, 1200]
    w, _ = stack("nvfp4", 3 * n, k, 8)
    x = torch.randn((sum(sizes), k + 1), device="cuda").bfloat16()[:, :k]          # (at odd places: copied first)
    offsets = offsets_of(sizes)
    nv.nvfp4_grouped_matmul(w, x, offsets)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.nvfp4_grouped_matmul(w, x, offsets)
    for ends in ([0, 1400, 1400, 2600], [7, 7, 2000, 2001], [0, 0, 0, 0]):
        offsets.copy_(torch.tensor(ends, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, nv.nvfp4_grouped_matmul(w, x, offsets))


# ------------------------------------------------------------------ adapters

@pytest.mark.parametrize("rank", [8, 24, 40, 64])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_adapters_by_tiles_of_32_rows(rank, dt, wdt):
    """Whole numbers; segments that begin and end inside tiles."""
    n, k, adapters, sizes, index = 130, 300, 4, [4100, 0, 1, 2500, 1633, 31], [2, 0, 1, 2, -1, 0]
    first, rows = 5, 8300
    assert rows > 16 * 2 * cus() and rank <= 64 and first + sum(sizes) < rows
    g = torch.Generator(device="cuda").manual_seed(rank)

    def draw(*shape, keep=1.0):
        t = torch.randint(-1, 2, shape, generator=g, device="cuda")
        return t * (torch.rand(shape, generator=g, device="cuda") < keep)

    x, dy = placed(draw(rows, k).to(DT[dt]), 3, 1), placed(draw(rows, n).to(DT[dt]), 0, 0)
    a, b = draw(adapters, rank, k, keep=0.2).to(DT[wdt]), draw(adapters, n, rank, keep=0.2).to(DT[wdt])
    scale = torch.tensor([0.5, 1.0, 2.0, 0.25], device="cuda")
    offsets, which = offsets_of(sizes, first=first), torch.tensor(index, dtype=torch.int32, device="cuda")
    y, u = nv.nvfp4_adapters(x, a, b, offsets, which, scale, out_dtype=torch.float32)
    dx, da, db = nv.nvfp4_adapters_backward(dy, x.float(), u, a, b, offsets, which, scale)
    wy, wu = torch.zeros(y.shape, device="cuda").double(), torch.zeros(u.shape, device="cuda").double()
    wdx, wa = torch.zeros((rows, k), device="cuda").double(), torch.zeros(a.shape, device="cuda").double()
    wb = torch.zeros(b.shape, device="cuda").double()
    at = first
    for size, i in zip(sizes, index):
        s, at = slice(at, at + size), at + size
        if i < 0:
            continue
        xd, dd, ad, bd, sd = x[s].double(), dy[s].double(), a[i].double(), b[i].double(), float(scale[i])
        wu[s] = xd @ ad.t().contiguous()
        wy[s] = sd * (wu[s] @ bd.t().contiguous())
        gd = sd * (dd @ bd)
        wdx[s] = gd @ ad
        wa[i] += gd.t().contiguous() @ xd
        wb[i] += sd * (dd.t().contiguous() @ wu[s])
    for got, want in ((u, wu), (y, wy), (dx, wdx), (da, wa), (db, wb)):
        assert float(want.abs().max()) < 2 ** 22
        assert torch.equal(got.double(), want)


# ------------------------------------------------------------------ RMS norm

LAST_CACHE = 256 << 20


@pytest.mark.parametrize("cols", [480, 2048, 5120, 12320, 20480])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_rms_norm_past_the_caches(cols, dt, res):
    """More than the last cache holds: rows do not know of each other, so some of
    them come out bit for bit as in a small call; the sums over all rows are
    checked against float64 ((rows + 4) u of their magnitudes)."""
    size = {"bf16": 2, "f32": 4}
    rows = 1 + LAST_CACHE // (cols * (size[dt] + (2 * size[res] + 1 if res else size[dt])))
    g = torch.Generator(device="cuda").manual_seed(cols)

    def draw(d):
        return torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32).to(DT[d])

    print(f"[rms norm] {rows}x{cols} {dt} {res}", flush=True)
    x, r = draw(dt), None if res is None else draw(res)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    cuts = [slice(0, 3), slice(rows // 2, rows // 2 + 5), slice(rows - 4, rows)]
    y, rstd, *h = nv.nvfp4_rms_norm(x, w, r)
    m, m_rstd, *m_h = nv.mxfp8_rms_norm(x, w, r)
    assert torch.equal(rstd, m_rstd) and all(torch.equal(p, q) for p, q in zip(h, m_h))
    for at in cuts:
        part = None if r is None else r[at]
        ys, rs, *hs = nv.nvfp4_rms_norm(x[at], w, part)
        ms = nv.mxfp8_rms_norm(x[at], w, part)[0]
        assert torch.equal(ys, y[at]) and torch.equal(rs, rstd[at]) and all(torch.equal(p, q[at]) for p, q in zip(hs, h))
        assert torch.equal(ms.codes, m.codes[at]) and torch.equal(ms.scales, m.scales[at])
    if res is not None:                                            # in the residual's place
        out = r.clone()
        y2, rstd2, h2 = nv.nvfp4_rms_norm(x, w, out, residual_out=out)
        assert h2 is out and torch.equal(h2, h[0]) and torch.equal(y2, y) and torch.equal(rstd2, rstd)


@pytest.mark.parametrize("cols", [480, 5120, 12320])
@pytest.mark.parametrize("dt,dyt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("with_dh", [False, True])
def test_rms_norm_backward_past_the_caches(cols, dt, dyt, with_dh):
    size = {"bf16": 2, "f32": 4}
    rows = 1 + LAST_CACHE // (cols * ((3 if with_dh else 2) * size[dt] + size[dyt]))
    g = torch.Generator(device="cuda").manual_seed(cols)

    def draw(d):
        return torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32).to(DT[d])

    print(f"[rms norm] backward {rows}x{cols} {dt} {dyt} {with_dh}", flush=True)
    h, dy, dh = draw(dt), draw(dyt), draw(dt) if with_dh else None
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    rstd = nv.nvfp4_rms_norm(h, w)[1]
    dx, dw = nv.nvfp4_rms_norm_backward(dy, h, rstd, w, dh)
    for at in (slice(0, 3), slice(rows // 2, rows // 2 + 5), slice(rows - 4, rows)):
        small = nv.nvfp4_rms_norm_backward(dy[at], h[at], rstd[at], w, None if dh is None else dh[at])[0]
        assert torch.equal(small, dx[at])
    sums = torch.zeros((2, cols), dtype=torch.float64, device="cuda")
    for at in range(0, rows, 4096):
        t = dy[at:at + 4096].double() * h[at:at + 4096].double() * rstd[at:at + 4096, None].double()
        sums += torch.stack([t.sum(0), t.abs().sum(0)])
    assert torch.all((dw.double() - sums[0]).abs() <= (rows + 4) * U * sums[1])
    again = nv.nvfp4_rms_norm_backward(dy, h, rstd, w, dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
