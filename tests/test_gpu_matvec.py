"""GPU checks of the matrix-vector products with 4-bit weights against the
float64 product of the exactly decoded weights.

Every product of a decoded weight and a bf16 (or split float32) activation is
exact in binary32; an output is a sum of K of them (three times as many parts
for float32 activations) that passes through at most one rounding per two
products and a few joins, so with u = 2^-24 it is within
    (K / 2 + 32) u sum|x w|     (float32 x: 3 (K / 2) + 32)
worst case, and with independent rounding errors near its square root: the
bound used is the smaller of that and 1e-5 sum|x w|, the GEMMs' contract.
bf16 outputs add half a bf16 step.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def _weights(fmt, n, k, seed):
    """Random codes and scales over their whole useful range: (tensor, decoded float64 [n, k])."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    q = np.empty((n, k))
    q[:, 0::2], q[:, 1::2] = GRID[codes & 15], GRID[codes >> 4]
    cu = torch.from_numpy(codes).cuda()
    if fmt == "nvfp4":
        scales = rng.integers(0, 0x7F, (n, k // 16), dtype=np.uint8)        # every finite E4M3 code, subnormals too
        s = torch.from_numpy(scales).view(torch.float8_e4m3fn).double().numpy()
        meta = torch.tensor([2.5, 2.5 / 2688], dtype=torch.float32)
        w = q * np.repeat(s, 16, 1) * meta[1].double().item()
        return nv.NVFP4Tensor(cu, torch.from_numpy(scales).cuda(), meta.cuda(), n, k), w
    scales = rng.integers(100, 135, (n, k // 32), dtype=np.uint8)
    w = q * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
    return nv.MXFP4Tensor(cu, torch.from_numpy(scales).cuda(), n, k), w


def _x(tokens, k, dtype, seed, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((tokens, k), generator=g) * (1 + 49 * (torch.rand((tokens, k), generator=g) < 0.01))
    flat = torch.full((shift + tokens * (k + pad),), float("nan"), dtype=dtype, device="cuda")
    view = flat[shift:].view(tokens, k + pad)[:, :k]
    view.copy_(v.to(dtype))
    return view


def _check(y, x, w, label):
    y, xd = y.detach(), x.double().cpu().numpy()
    k = w.shape[1]
    want, mass = xd @ w.T, np.abs(xd) @ np.abs(w).T
    parts = 3 if x.dtype == torch.float32 else 1
    bound = min((parts * k / 2 + 32) * U, 1e-5) * mass
    if y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    err = np.abs(y.double().cpu().numpy() - want)
    worst = np.max(err / (bound + 1e-40)) if err.size else 0.0
    print(f"[matvec] {label}: worst error / bound {worst:.3f}", flush=True)
    assert np.all(err <= bound + 1e-40), label


def _run(fmt, w, x, **kw):
    return (nv.nvfp4_matvec if fmt == "nvfp4" else nv.mxfp4_matvec)(w, x, **kw)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8, 16, 17, 40])
@pytest.mark.parametrize("n,k", [(1, 32), (16, 64), (17, 96), (33, 416), (130, 1056), (257, 5120)])
def test_against_decoded_product(fmt, dt, tokens, n, k):
    w, wd = _weights(fmt, n, k, n * 1000 + k)
    x = _x(tokens, k, DT[dt], tokens)
    print(f"[matvec] {fmt} {dt} {tokens}x{n}x{k}", flush=True)
    _check(_run(fmt, w, x, out_dtype=torch.float32), x, wd, "f32 out")
    _check(_run(fmt, w, x, out_dtype=torch.bfloat16), x, wd, "bf16 out")


@pytest.mark.parametrize("k", [16, 48, 80, 112, 144, 1040, 2064, 20496])
@pytest.mark.parametrize("tokens", [1, 4])
def test_nvfp4_odd_groups(k, tokens):
    """K an odd number of 16-groups: the last lane of a row holds half a load."""
    w, wd = _weights("nvfp4", 37, k, k)
    for dt in ("bf16", "f32"):
        x = _x(tokens, k, DT[dt], 7, pad=3, shift=1)
        _check(_run("nvfp4", w, x, out_dtype=torch.float32), x, wd, f"K={k} {dt}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n,k", [(40, 20480), (5000, 64), (4099, 1600), (3, 8192)])
def test_long_and_wide(fmt, n, k):
    w, wd = _weights(fmt, n, k, 3)
    for tokens in (1, 6, 16):
        x = _x(tokens, k, torch.bfloat16, 11)
        _check(_run(fmt, w, x), x, wd, f"{tokens}x{n}x{k}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
def test_output_view(fmt, out_dt):
    """An output with spare columns: they keep what they held."""
    n, k, tokens = 45, 192, 5
    w, wd = _weights(fmt, n, k, 13)
    x = _x(tokens, k, torch.bfloat16, 17, pad=5, shift=3)
    base = torch.full((tokens, n + 3), 9.0, dtype=DT[out_dt], device="cuda")
    y = _run(fmt, w, x, out_dtype=DT[out_dt], out=base[:, :n])
    _check(y, x, wd, "view")
    assert torch.all(base[:, n:] == 9.0)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens", [1, 3])
def test_non_finite_activations_stay_in_their_token(fmt, tokens):
    n, k = 50, 320
    w, wd = _weights(fmt, n, k, 19)
    for dt in ("bf16", "f32"):
        x = _x(tokens, k, DT[dt], 23)
        clean = _run(fmt, w, x, out_dtype=torch.float32)
        for value in (float("inf"), float("-inf"), float("nan")):
            bad = x.clone()
            bad[0, 37] = value
            y = _run(fmt, w, bad, out_dtype=torch.float32)
            # inf times a zero weight is NaN, as in the formula
            col = torch.from_numpy(wd[:, 37].copy()).cuda()
            want = torch.where(col == 0, float("nan"), col.float() * value)
            assert torch.equal(torch.isnan(y[0]), torch.isnan(want))
            sure = ~torch.isnan(want)
            assert torch.equal(y[0][sure], want[sure])
            assert torch.equal(y[1:], clean[1:])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_small_and_large_activations(dt):
    """Activations far below and above 1: products and parts keep their digits."""
    w, wd = _weights("nvfp4", 24, 256, 29)
    for scale in (2.0 ** -100, 2.0 ** 90):
        x = (_x(2, 256, torch.float32, 31) * scale).to(DT[dt])
        xd = x.double().cpu().numpy()
        got = _run("nvfp4", w, x, out_dtype=torch.float32).double().cpu().numpy()
        bound = 1e-5 * (np.abs(xd) @ np.abs(wd).T)
        assert np.all(np.abs(got - xd @ wd.T) <= bound)


def test_mx_scale_range():
    """The smallest scales that a product with ordinary activations keeps
    normal, and large ones."""
    rng = np.random.default_rng(37)
    n, k = 32, 128
    for lo, hi in ((1, 20), (230, 252)):
        codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
        scales = rng.integers(lo, hi, (n, k // 32), dtype=np.uint8)
        q = np.empty((n, k))
        q[:, 0::2], q[:, 1::2] = GRID[codes & 15], GRID[codes >> 4]
        wd = q * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
        w = nv.MXFP4Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), n, k)
        x = _x(3, k, torch.bfloat16, 41) * (2.0 ** 30 if lo == 1 else 2.0 ** -30)
        _check(nv.mxfp4_matvec(w, x, out_dtype=torch.float32), x, wd, f"scales {lo}..{hi}")


def test_zero_scale_groups():
    """Groups whose scale is 0 give 0, and a tensor of them zeros."""
    n, k = 20, 160
    w, _ = _weights("nvfp4", n, k, 43)
    w.scales.zero_()
    y = nv.nvfp4_matvec(w, _x(2, k, torch.bfloat16, 47))
    assert torch.all(y == 0)


def test_empty():
    w, _ = _weights("nvfp4", 8, 64, 53)
    assert nv.nvfp4_matvec(w, torch.empty((0, 64), device="cuda")).shape == (0, 8)
    none, _ = _weights("nvfp4", 0, 64, 53)
    assert nv.nvfp4_matvec(none, torch.ones((3, 64), device="cuda")).shape == (3, 0)
    flat = nv.NVFP4Tensor(torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                          torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                          torch.zeros(2, device="cuda"), 5, 0)
    assert torch.all(nv.nvfp4_matvec(flat, torch.empty((2, 0), device="cuda")) == 0)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantized_weights_round_trip(fmt):
    """Weights as the library's own quantizers write them."""
    wf = torch.randn((200, 512), generator=torch.Generator().manual_seed(59)).mul_(0.02).to(torch.bfloat16).cuda()
    w = nv.nvfp4_quantize(wf) if fmt == "nvfp4" else nv.mxfp4_quantize(wf)
    x = _x(4, 512, torch.bfloat16, 61)
    if fmt == "nvfp4":
        wd = nv.nvfp4_dequantize(w).double().cpu().numpy()
        # the decoded tensor is rounded once per element (u of it)
        _check(_run(fmt, w, x, out_dtype=torch.float32), x, wd, "quantized")
    else:
        codes, sc = w.codes.cpu().numpy(), w.scales.cpu().numpy().astype(np.float64)
        q = np.empty((200, 512))
        q[:, 0::2], q[:, 1::2] = GRID[codes & 15], GRID[codes >> 4]
        _check(_run(fmt, w, x, out_dtype=torch.float32), x, q * np.repeat(2.0 ** (sc - 127), 32, 1), "quantized")


def test_other_stream_and_repeat():
    w, _ = _weights("nvfp4", 600, 2048, 67)
    x = _x(7, 2048, torch.bfloat16, 71)
    want = nv.nvfp4_matvec(w, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.nvfp4_matvec(w, x, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(nv.nvfp4_matvec(w, x), want)


def test_graph_replays():
    w, _ = _weights("mxfp4", 300, 1024, 73)
    x = _x(2, 1024, torch.bfloat16, 79).contiguous()
    nv.mxfp4_matvec(w, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.mxfp4_matvec(w, x)
    for turn in range(4):
        x.copy_(_x(2, 1024, torch.bfloat16, 80 + turn))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, nv.mxfp4_matvec(w, x))


def test_offsets_past_32_bits():
    """5.2 GB of codes: sampled rows."""
    n, k = 2_040_005, 5120
    assert n * (k // 2) > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(83)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(1, 120, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
    meta = torch.tensor([1.0, 1 / 2688], device="cuda")
    x = _x(2, k, torch.bfloat16, 89)
    y = nv.nvfp4_matvec(nv.NVFP4Tensor(codes, scales, meta, n, k), x, out_dtype=torch.float32)
    for r in (0, n // 2, n - 40):
        c = codes[r:r + 40].cpu().numpy()
        q = np.empty((c.shape[0], k))
        q[:, 0::2], q[:, 1::2] = GRID[c & 15], GRID[c >> 4]
        s = scales[r:r + 40].cpu().view(torch.float8_e4m3fn).double().numpy()
        _check(y[:, r:r + 40], x, q * np.repeat(s, 16, 1) * meta[1].double().item(), f"rows from {r}")


@pytest.mark.parametrize("tokens", [1, 2, 7, 16])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [512, 1504])
def test_wide_range_within_a_token(dt, tokens, k):
    """Activations from 2^-60 to 2^60 side by side, the large ones under zero
    weights in half the rows: those rows' sums are of the small ones, which
    therefore have to keep all their bits."""
    n = 40
    w, wd = _weights("nvfp4", n, k, 97)
    x = _x(tokens, k, torch.float32, 101)
    for t in range(tokens):
        x[t, t % 16] = 2.0 ** 60
        x[t, 300 + t] = 0.0
        x[t, 20 + t] *= 2.0 ** -60
    if tokens > 2:
        x[1] = x[1].clamp(-1, 1) * 2.0 ** -40 + 0.0     # one token of ordinary spread between them
        x[2] = 0.0
    x = x.to(DT[dt])
    w.codes[: n // 2, :8] = 0
    wd[: n // 2, :16] = 0.0
    _check(_run("nvfp4", w, x, out_dtype=torch.float32), x, wd, f"{dt} {tokens} K={k}")


@pytest.mark.parametrize("tokens", [2, 16])
def test_ranges_of_k_join(tokens):
    """Long reductions are cut among workgroups and joined: K whole and not in
    the pieces that a cut has, an odd N, an output view."""
    for k in (6144, 7200, 20480 + 16, 24576):
        w, wd = _weights("nvfp4", 35, k, k)
        for dt in ("bf16", "f32"):
            x = _x(tokens, k, DT[dt], 103, pad=1)
            base = torch.full((tokens, 40), 9.0, dtype=torch.bfloat16, device="cuda")
            _check(_run("nvfp4", w, x, out_dtype=torch.bfloat16, out=base[:, :35]), x, wd, f"K={k} {dt}")
            assert torch.all(base[:, 35:] == 9.0)


@pytest.mark.parametrize("k", [128, 2032, 2048, 2064, 4096, 4112, 6144, 6160, 8192, 8208, 16384, 16400, 24576, 24592])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_few_tokens_at_every_length(dt, k):
    """One to five tokens where a row just fills, overfills or leaves part of
    the loads of the waves that share it; an odd number of weight rows."""
    w, wd = _weights("nvfp4", 11, k, k + 1)
    for tokens in (1, 2, 3, 4, 5):
        x = _x(tokens, k, DT[dt], 107 + tokens, pad=2, shift=1)
        _check(_run("nvfp4", w, x, out_dtype=torch.float32), x, wd, f"{dt} {tokens} K={k}")
