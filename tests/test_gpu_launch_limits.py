"""GPU checks of sizes whose launches pass 2^32 threads: long rows in the last
kernel of the layer norm's backward pass, many short rows in distillation."""
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


def test_distillation_of_many_short_rows():
    """2^26 + 64 rows of 8 logits: every 64 rows are the same ones."""
    block, tokens = 64, 2 ** 26 + 64
    g = torch.Generator(device="cuda").manual_seed(2)
    z = (3 * torch.randn((block, 8), device="cuda", generator=g)).to(torch.bfloat16)
    idx = torch.randint(-1, 8, (block, 2), device="cuda", generator=g, dtype=torch.int32)
    t = torch.randn((block, 2), device="cuda", generator=g).to(torch.bfloat16)
    weight = torch.rand(block, device="cuda", generator=g)
    want = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    times = tokens // block
    z, idx, t, weight = z.repeat(times, 1), idx.repeat(times, 1), t.repeat(times, 1), weight.repeat(times)
    print(f"[distill] {tokens}x8", flush=True)
    step = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    loss, lse = nv.nvfp4_distill_topk(z, idx, t)
    for got, one in ((step[0], want[0]), (step[1], want[1]), (loss, want[0]), (lse, want[1])):
        assert torch.all(got.view(times, block) == one)
    for part in step[2].view(times, block, 8).split(2 ** 16):
        assert torch.all(part == want[2])
