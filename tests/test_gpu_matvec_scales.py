"""GPU checks of the MXFP4 matrix-vector products over every E8M0 scale code:
0 (2^-127) to 254 (2^127), and 255, which is NaN.

A weight is 2^(code - 127) times at most 6, so it may lie above bf16's and
binary32's range; what counts is that its products with the activations do
not.  Bounds as for any scales: products are exact in binary32 where they are
normal numbers, the sum is within 1e-5 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOKENS = [1, 2, 3, 5, 8, 16, 17]
N = 37


def _weights(k, lo, hi, seed, special=()):
    """Random codes, scales from lo to hi; (rows, block, code) of `special` set afterwards."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, k // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi + 1, (N, k // 32), dtype=np.uint8)
    for row, block, code in special:
        scales[row, block] = code
    q = np.empty((N, k))
    q[:, 0::2], q[:, 1::2] = GRID[codes & 15], GRID[codes >> 4]
    w = nv.MXFP4Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), N, k)
    return w, q * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)


def _x(tokens, k, dt, scale):
    g = torch.Generator().manual_seed(tokens * 100 + k)
    return (torch.randn((tokens, k), generator=g) * scale).to(DT[dt]).cuda()


def _check(y, x, w, rows=slice(None)):
    xd = x.double().cpu().numpy()
    want, mass = (xd @ w.T)[:, rows], (np.abs(xd) @ np.abs(w).T)[:, rows]
    assert mass.max() < 3e38, "the case itself overflows"
    assert np.all(np.abs(y.double().cpu().numpy()[:, rows] - want) <= 1e-5 * mass)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [32, 96, 128, 416, 1056, 6176])
@pytest.mark.parametrize("lo,hi,scale", [(0, 3, 2.0 ** 60), (250, 254, 2.0 ** -40), (60, 254, 2.0 ** -40)])
def test_whole_range_of_scales(lo, hi, scale, k, dt):
    w, wd = _weights(k, lo, hi, k + lo)
    for tokens in TOKENS:
        print(f"[matvec] scales {lo}..{hi} {tokens}x{N}x{k} {dt}", flush=True)
        x = _x(tokens, k, dt, scale)
        _check(nv.mxfp4_matvec(w, x, out_dtype=torch.float32), x, wd)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [96, 1056])
def test_smallest_beside_largest(k, dt):
    """Rows of the smallest scales keep their digits beside a row of the
    largest, whose own sums overflow here."""
    w, wd = _weights(k, 0, 2, 5, [(9, b, 254) for b in range(k // 32)])
    rows = [r for r in range(N) if r != 9]
    wd[9] = 0.0
    for tokens in TOKENS:
        x = _x(tokens, k, dt, 2.0 ** 60)
        _check(nv.mxfp4_matvec(w, x, out_dtype=torch.float32), x, wd, rows)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [32, 96, 128, 1056])
def test_nan_scale(k, dt):
    """Code 255 makes its row NaN, zeros and all, and no other."""
    w, wd = _weights(k, 120, 130, 7, [(3, 0, 255), (20, k // 32 - 1, 255)])
    w.codes[20] = 0
    wd[[3, 20]] = 0.0
    rows = [r for r in range(N) if r not in (3, 20)]
    for tokens in TOKENS:
        x = _x(tokens, k, dt, 1.0)
        y = nv.mxfp4_matvec(w, x, out_dtype=torch.float32)
        assert torch.isnan(y[:, [3, 20]]).all()
        _check(y, x, wd, rows)
        assert torch.isnan(nv.mxfp4_matvec(w, x, out_dtype=torch.bfloat16)[:, [3, 20]]).all()
