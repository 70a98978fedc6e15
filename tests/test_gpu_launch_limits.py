"""GPU checks of sizes whose launches pass 2^32 threads: long rows in the last
kernel of the layer norm's backward pass."""
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def test_layer_norm_backward_of_long_rows():
    """dweight and dbias of 2^27 + 3 columns: sums of two products each, within
    4 u of their magnitudes; dx within the bound of its row sums, whose
    binary32 additions are cols / 8192 + 64 after each other."""
    rows, cols = 2, 2 ** 27 + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), device="cuda", generator=g, dtype=torch.float32).to(torch.bfloat16)
    dy = torch.randn((rows, cols), device="cuda", generator=g, dtype=torch.float32).to(torch.bfloat16)
    mean = torch.tensor([0.1, -0.2], device="cuda")
    rstd = torch.tensor([1.5, 0.75], device="cuda")
    print(f"[norm] backward {rows}x{cols}", flush=True)
    dx, dw, db = nv.nvfp4_layer_norm_backward(dy, x, mean, rstd)
    sums = torch.zeros((rows, 3), dtype=torch.float64, device="cuda")          # a, a h, |a h|
    pieces = [slice(c, min(c + 2 ** 24, cols)) for c in range(0, cols, 2 ** 24)]
    m, r = mean.double()[:, None], rstd.double()[:, None]
    for s in pieces:
        a, h = dy[:, s].double(), (x[:, s].double() - m) * r
        ah = a * h
        assert torch.all((dw[s].double() - ah.sum(0)).abs() <= 4 * U * ah.abs().sum(0) + 1e-30)
        assert torch.all((db[s].double() - a.sum(0)).abs() <= 4 * U * a.abs().sum(0) + 1e-30)
        sums += torch.stack([a.sum(1), ah.sum(1), ah.abs().sum(1) + a.abs().sum(1)], 1)
    s1, s2, mass = (sums[:, i:i + 1] / cols for i in range(3))
    off = (cols / 8192 + 64) * U * mass
    for s in pieces[:1] + pieces[-2:]:
        a, h = dy[:, s].double(), (x[:, s].double() - m) * r
        want = r * (a - s1 - h * s2)
        bound = r * (off * (1 + h.abs()) + 8 * U * (a.abs() + s1.abs() + (h * s2).abs()))
        assert torch.all((dx[:, s].double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound))
