"""GPU checks of the matrix-vector products where a workgroup goes through
several turns (weight rows' form) or tiles (several tokens' form), and where
the tiles' form multiplies in f16: many weight rows, all of them compared.

Each case states why it walks: the weight rows of a turn of the whole grid,
which the host checks against N, so that another cut of the work shows here.
Bounds: 1e-5 of the sum of magnitudes, as for any product."""
import math

import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _weights(fmt, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    if fmt == "nvfp4":
        scales = torch.randint(0, 0x7F, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
        return nv.NVFP4Tensor(codes, scales, torch.tensor([2.0, 2.0 / 2688], device="cuda"), n, k)
    scales = torch.randint(100, 135, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    return nv.MXFP4Tensor(codes, scales, n, k)


def _decoded(w, rows):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device="cuda")
    c = w.codes[rows]
    q = torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], 2).view(c.shape[0], w.k)
    if isinstance(w, nv.NVFP4Tensor):
        s = w.scales[rows].view(torch.float8_e4m3fn).double() * w.meta[1].double()
        return q.mul_(s.repeat_interleave(16, 1))
    return q.mul_(torch.exp2(w.scales[rows].double() - 127).repeat_interleave(32, 1))


def _run(w, x, out_dtype=torch.float32):
    return (nv.nvfp4_matvec if isinstance(w, nv.NVFP4Tensor) else nv.mxfp4_matvec)(w, x, out_dtype=out_dtype)


def _check(w, x, y, tokens=slice(None)):
    xd = x.double()
    step = max(1, 2 ** 26 // w.k)
    for r in range(0, w.outer, step):
        rows = slice(r, min(r + step, w.outer))
        wd = _decoded(w, rows)
        off = (y[:, rows].double() - xd @ wd.t()).abs()[tokens]
        assert torch.all(off <= 1e-5 * (xd.abs() @ wd.abs().t())[tokens]), rows


def _x(tokens, k, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, k), device="cuda", generator=g)
    return (x * (1 + 49 * (torch.rand((tokens, k), device="cuda", generator=g) < 0.01))).to(DT[dt])


# tokens, types, K, N, weight rows of a workgroup's turn, workgroups a CU
ROWS = [(1, "both", 512, 36901, 16, 3), (1, "both", 2064, 18491, 8, 3), (1, "both", 5120, 9311, 4, 3),
        (1, "both", 8192, 9311, 4, 3), (1, "both", 8208, 4651, 2, 3), (1, "both", 16400, 2351, 1, 3),
        (2, "both", 512, 36901, 16, 3), (2, "both", 2064, 18491, 8, 3), (2, "both", 5120, 12301, 4, 4),
        (2, "both", 8192, 9311, 4, 3), (2, "bf16", 8208, 4651, 2, 3), (3, "both", 496, 36901, 16, 3),
        (3, "both", 4096, 12303, 8, 3), (3, "both", 6128, 8301, 4, 4), (3, "both", 6160, 7001, 4, 3),
        (4, "both", 1008, 24401, 16, 3), (4, "both", 2064, 12001, 8, 3), (4, "both", 4112, 6047, 4, 4),
        (4, "both", 6160, 4041, 4, 3)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,types,k,n,turn,groups", ROWS)
def test_turns_of_weight_rows(tokens, types, k, n, turn, groups, fmt):
    assert n > turn * groups * _cus(), "one turn does it"
    k = (k + 31) // 32 * 32 if fmt == "mxfp4" else k
    w = _weights(fmt, n, k, k + tokens)
    for dt in ("bf16", "f32") if types == "both" else (types,):
        print(f"[matvec] rows {fmt} {tokens}x{n}x{k} {dt}", flush=True)
        x = _x(tokens, k, dt, n)
        _check(w, x, _run(w, x))


# K, N: short K puts up to 12 workgroups on a CU, long K one or two
TILES = [(128, 12), (400, 12), (1024, 12), (1040, 12), (2064, 3), (5120, 2), (6160, 2), (11280, 2)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [5, 6, 11, 16, 17])
@pytest.mark.parametrize("k,groups", TILES)
def test_walks_of_tiles(k, groups, tokens, dt, fmt):
    n = 16 * 3 * groups * _cus() + 5                   # three tiles and more for every workgroup
    k = (k + 31) // 32 * 32 if fmt == "mxfp4" else k
    print(f"[matvec] tiles {fmt} {tokens}x{n}x{k} {dt}", flush=True)
    w, x = _weights(fmt, n, k, k + tokens), _x(tokens, k, dt, n)
    y = _run(w, x)
    _check(w, x, y)
    assert torch.equal(_run(w, x, torch.bfloat16), y.to(torch.bfloat16))


def _many_rows(k, seed):
    """NVFP4 weights of 8 tiles and more for every workgroup, however many of
    them a CU takes (12 at most, one wave each), from where on columns whose
    values span at most 29 binades are multiplied in f16.  Every other row has
    no weight on the first 16 k."""
    w = _weights("nvfp4", 16 * 8 * 12 * _cus() + 9, k, seed)
    w.codes[::2, :8] = 0
    return w


def _spread(tokens, k, dt, spans, seed):
    """Token t: values of full 8 (f32: 24) bits in [1, 2) 2^-spans[t], and in the first 16 k some in [1, 2)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 1 + torch.rand((tokens, k), device="cuda", generator=g)
    x = torch.where(torch.rand((tokens, k), device="cuda", generator=g) < 0.5, -x, x)
    span = torch.tensor(spans, device="cuda")[:, None]
    at = torch.arange(k, device="cuda")[None]
    x = torch.where((at < 16) & (at % 3 == 0), x, torch.ldexp(x, -span))
    x = x.to(DT[dt])
    return torch.where(x.abs() == 2, x / 2, x) if dt == "bf16" else x    # (rounded up to 2: one binade more)


@pytest.mark.parametrize("k", [128, 400])
@pytest.mark.parametrize("tokens,dt", [(7, "bf16"), (16, "bf16"), (17, "bf16"), (5, "f32"), (7, "f32"), (16, "f32")])
def test_spans_of_a_column(tokens, dt, k):
    """The small values alone make the sums of every other row: they keep all
    their bits whether the columns fit f16 or not.  All tokens alike, then one
    among ordinary ones (which takes the wave's others along), zero tokens."""
    w = _many_rows(k, k)
    for span in (0, 20, 27, 28, 29, 30, 32, 40, 60):
        print(f"[matvec] span {span} {tokens}x{w.outer}x{k} {dt}", flush=True)
        x = _spread(tokens, k, dt, [span] * tokens, span)
        _check(w, x, _run(w, x))
    x = _spread(tokens, k, dt, [3] * (tokens - 1) + [45], 1)
    _check(w, x, _run(w, x))
    x = _spread(tokens, k, dt, [5] * tokens, 2)
    x[1] = 0
    x[3, 1:] = 0
    y = _run(w, x)
    _check(w, x, y)
    assert torch.all(y[1] == 0)


@pytest.mark.parametrize("tokens,dt", [(7, "bf16"), (16, "bf16"), (5, "f32"), (16, "f32")])
def test_tokens_of_different_size(tokens, dt):
    """Each column has its own power of two: tokens from 2^-100 to 2^90, some of
    whose elements are 0."""
    w = _many_rows(272, 3)
    x = _spread(tokens, 272, dt, [2] * tokens, 4)
    power = torch.linspace(-100, 90, tokens, device="cuda").round().int()[:, None]
    x = torch.ldexp(x.float(), power).to(DT[dt])
    x[:, 5::7] = 0
    _check(w, x, _run(w, x))

@pytest.mark.parametrize("tokens,dt", [(7, "bf16"), (17, "bf16"), (5, "f32"), (16, "f32")])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_non_finite_in_one_token(tokens, dt, value):
    w = _many_rows(160, 5)
    x = _spread(tokens, 160, dt, [6] * tokens, 6)
    x[2, 70] = value
    y = _run(w, x)
    x[2, 70] = 0
    _check(w, x, y, [t for t in range(tokens) if t != 2])
    col = torch.cat([_decoded(w, slice(r, r + 2 ** 17))[:, 70] for r in range(0, w.outer, 2 ** 17)])
    want = torch.where(col == 0, math.nan, col * value).float()        # inf times a zero weight is NaN
    assert torch.equal(y[2].isnan(), want.isnan())
    assert torch.equal(y[2][~want.isnan()], want[~want.isnan()])
