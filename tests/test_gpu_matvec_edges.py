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
