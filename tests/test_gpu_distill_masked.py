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


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 0.5])
@pytest.mark.parametrize("tokens,vocab", [(3, 7), (3, 300), (5, 9000), (3, 70001)])
@pytest.mark.parametrize("level,spread", [("lowest", 0.0), (-1e9, 100.0), (-1e4, 2.0), (3000.0, 2.0), (3e5, 1.0)])
def test_backward_from_a_far_log_sum(level, spread, tokens, vocab, tau, dt):
    """A row that lies as a whole at the type's lowest value, or at a mask's
    value, has the shares of its differences, though a binary32 log-sum-exp
    of such a size (or its overflow, at temperatures below 1) no longer tells them.

    A share exp(z / tau - lse) formed from the row's maximum is off by
    E = 4 u (V / 256 + 64 + 70) of itself (u = 2^-24: the sum's roundings, the
    exponent's; factor 4), one formed from a saved lse below 4096 by 4 u |lse|
    more; the teacher's shares by 4 u (span / tau + 70); bf16 adds half a step."""
    u = 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(vocab)
    base = torch.finfo(DT[dt]).min if level == "lowest" else level
    z = (base + spread * torch.randn((tokens, vocab), device="cuda", generator=g)).to(DT[dt])
    idx = torch.randint(0, vocab, (tokens, 3), device="cuda", generator=g)
    t = torch.randn((tokens, 3), device="cuda", generator=g)
    weight = torch.rand(tokens, device="cuda", generator=g) + 0.5
    idx[0], weight[1] = -1, 0.0
    print(f"[distill] {tokens}x{vocab} {dt} tau {tau} level {level}", flush=True)
    loss, lse = nv.nvfp4_distill_topk(z, idx, t, temperature=tau)
    grad = nv.nvfp4_distill_topk_backward(z, idx, t, lse, weight, temperature=tau).double()
    zd = z.double() / tau
    want_lse = torch.logsumexp(zd, 1)
    q = torch.softmax(zd, 1)
    P = torch.zeros_like(q).scatter_add_(1, idx.clamp(min=0), torch.softmax(t.double() / tau, 1))
    live = torch.tensor([0.0, 0.0] + [1.0] * (tokens - 2), device="cuda", dtype=torch.float64)[:, None]
    scale = weight.double()[:, None] * tau * live
    near = torch.where(want_lse.abs() < 4096, want_lse.abs(), 0.0)[:, None]
    e = 4 * u * (vocab / 256 + 64 + 70 + near) + 4 * u * (8 / tau + 70)
    want, bound = scale * (q - P), scale * (q + P) * e + 1e-37
    if dt == "bf16":
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert torch.all((grad - want).abs() <= bound)
