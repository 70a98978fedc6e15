"""Temperatures whose reciprocal binary32 does not hold are refused."""
import pytest
import torch

import gemm_amax_reduce_amd as nv

A = 1 << 20
_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer argument tests run only without a GPU")


@_no_gpu
@pytest.mark.parametrize("tau,status", [(1e-40, -6), (2.0 ** -127, -6), (2.0 ** -126, -4), (1.0, -4), (1e30, -4)])
def test_smallest(tau, status):
    """-6: out of range; -4: as far as the launch, which fails without a GPU."""
    L = nv.lib()
    rows = (A, 1, 2, 8, 8, 2 * A, 64, 3 * A, 1, 1, tau)
    assert L.nvfp4_distill_topk(*rows, 4 * A, 4 * A, None, 0, None) == status
    assert L.nvfp4_distill_topk_backward(*rows, 4 * A, 4 * A, 8 * A, 8, None) == status
    assert L.nvfp4_distill_topk_step(*rows, 4 * A, 4 * A, 4 * A, 8 * A, 8, None, 0, None) == status


@pytest.mark.gpu
def test_cold_teacher_and_student():
    """At the smallest temperature shares are 0 and 1, or equal where logits are."""
    z = torch.tensor([[0.0, 0.0, -1.0, -2.0], [-1.0, 0.0, -3.0, -1.0]], device="cuda")
    idx, t = torch.tensor([[0, 1], [1, 2]], device="cuda"), torch.tensor([[0.0, 0.0], [5.0, 4.0]], device="cuda")
    tau = 2.0 ** -126
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, torch.ones(2, device="cuda"), temperature=tau)
    assert torch.all(loss == 0) and torch.all(grad == 0)
    assert torch.allclose(lse.double(), torch.tensor([2.0, 1.0], device="cuda").double().log(), atol=1e-6)
