"""GPU checks of the matrix-vector products at their edges."""
import math

import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [0.0, 1.0, math.inf, math.nan])
@pytest.mark.parametrize("tokens", [1, 3, 17])
def test_no_k_gives_zeros(tokens, g):
    """A sum over nothing is zero whatever the tensor scale of no weights is."""
    w = nv.NVFP4Tensor(torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                       torch.empty((5, 0), dtype=torch.uint8, device="cuda"),
                       torch.tensor([g, g], device="cuda"), 5, 0)
    for dt in (torch.float32, torch.bfloat16):
        y = nv.nvfp4_matvec(w, torch.empty((tokens, 0), device="cuda"), out_dtype=dt)
        assert y.shape == (tokens, 5) and torch.all(y == 0)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("k", [32, 96, 128, 1056, 5120])
def test_denormal_bf16_activations(k, fmt):
    """bf16 activations below the smallest normal number enter the product as
    they are: under weights of 2^100 (2^11 in NVFP4, whose tensor scale brings
    the rest) they make ordinary sums, each within 1e-5 of its magnitudes."""
    n = 21
    g = torch.Generator(device="cuda").manual_seed(k)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device="cuda")
    q = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], 2).view(n, k)
    if fmt == "mxfp4":
        scales = torch.randint(220, 230, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
        w = q * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
        wt, run, gain = nv.MXFP4Tensor(codes, scales, n, k), nv.mxfp4_matvec, 1.0
    else:
        scales = torch.randint(0x70, 0x7F, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
        w = q * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        gain = 2.0 ** 60
        wt, run = nv.NVFP4Tensor(codes, scales, torch.tensor([0.0, gain], device="cuda"), n, k), nv.nvfp4_matvec
    for tokens in (1, 2, 4, 7, 16):
        bits = torch.randint(1, 128, (tokens, k), device="cuda", generator=g)
        bits += 32768 * torch.randint(0, 2, (tokens, k), device="cuda", generator=g)
        x = bits.to(torch.int32).to(torch.uint16).view(torch.bfloat16)
        xd = (bits & 127).double() * 2.0 ** -133 * (1 - 2 * (bits >> 15).double())
        y = run(wt, x, out_dtype=torch.float32).double()
        want, mass = xd @ w.t() * gain, xd.abs() @ w.abs().t() * gain
        # (NVFP4's own sums lie at 2^-115 and above: normal numbers)
        assert torch.all((y - want).abs() <= 1e-5 * mass), tokens
