"""GPU checks of the distillation loss on rows whose mask leaves nothing."""
import math

import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,vocab", [(3, 1), (3, 7), (4, 50), (5, 9000), (4, 32768), (130, 33001), (3, 70001),
                                          (130, 70001), (2, 140001)])
def test_log_sum_of_a_row_without_logits(dt, tokens, vocab):
    """log of an empty sum: -inf, whichever way the row goes and whether or not
    a gradient is asked for; a NaN among the masked ones shows, and other rows
    keep their values."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randn((tokens, vocab), device="cuda", generator=g).to(DT[dt])
    z[0] = -math.inf
    z[1] = -math.inf
    z[1, vocab // 2] = math.nan
    idx = torch.zeros((tokens, 2), dtype=torch.int64, device="cuda")
    idx[:2] = -1
    t = torch.zeros((tokens, 2), device="cuda")
    weight = torch.ones(tokens, device="cuda")
    print(f"[distill] {tokens}x{vocab} {dt}", flush=True)
    loss, lse = nv.nvfp4_distill_topk(z, idx, t)
    grad = nv.nvfp4_distill_topk_backward(z, idx, t, lse, weight)
    step = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    # binary32 sums of V / 256 + 64 terms after each other, u = 2^-24, factor 4
    bound = 4 * 2.0 ** -24 * (vocab / 256 + 64 + 20)
    want = torch.logsumexp(z.double(), 1)
    for los, ls, gr in ((loss, lse, grad), step):
        assert ls[0] == -math.inf
        assert torch.isnan(ls[1])
        assert torch.all((ls[2:].double() - want[2:]).abs() <= bound)
        assert torch.all(los[:2] == 0) and torch.all(gr[:2] == 0)
        assert torch.isfinite(los[2:]).all() and torch.isfinite(gr[2:]).all()
