"""The weighted sum of a token's experts, on the CPU against float64.

The shares stay in float32 and the sum too, so that a bf16 result is off by its
own half step (2^-8 of the value) and binary32 roundings, top + 1 of 2^-24 of
the magnitudes (one for each product, top - 1 for the sum, one to spare)."""
import pytest
import torch

from gemm_amax_reduce_amd.experts import weighted_sum

U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,top,features", [(1, 1, 5), (7, 2, 64), (33, 8, 130), (0, 2, 16)])
def test_weighted_sum(dtype, tokens, top, features):
    g = torch.Generator().manual_seed(top)
    parts = torch.randn((tokens, top, features), generator=g).to(dtype).requires_grad_(True)
    share = torch.softmax(torch.randn((tokens, top), generator=g), 1).requires_grad_(True)
    y = weighted_sum(parts, share)
    pd, sd = (t.detach().double().requires_grad_(True) for t in (parts, share))
    yd = (pd * sd[:, :, None]).sum(1)
    mass = (pd.abs() * sd[:, :, None]).sum(1)
    half = HALF_BF16 if dtype == torch.bfloat16 else 0.0
    assert y.dtype == dtype and y.shape == (tokens, features)
    bound = (top + 1) * U * 1.01 * mass
    assert ((y.double() - yd).abs() <= bound + half * (yd.abs() + bound)).all()
    up = torch.randn(y.shape, generator=g).to(dtype)
    y.backward(up)
    yd.backward(up.double())
    assert parts.grad.dtype == dtype and share.grad.dtype == torch.float32
    assert ((parts.grad.double() - pd.grad).abs() <= (half + 2 * U) * 1.01 * pd.grad.abs()).all()
    mass = (up.double()[:, None].abs() * pd.abs()).sum(2)
    assert ((share.grad.double() - sd.grad).abs() <= (features + 1) * U * 1.01 * mass).all()
