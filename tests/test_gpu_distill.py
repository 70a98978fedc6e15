"""GPU checks of the distillation loss and its gradient against the definition
in float64, within a bound derived from binary32 arithmetic (u = 2^-24).

With R the largest |z - max z| / tau among the entries that matter (shares
above 1e-30: 70), a share exp(z / tau - lse) is off by the rounding of its
exponent (R u, and 4 u for the difference, the product and the exponential)
and of the sum (at most V / 256 + 64 roundings after each other, by threads,
waves and segments); the saved lse adds the rounding of its own value, which
the backward pass multiplies by tau again.  With room of a factor 4:
    E = 4 u (V / 256 + 64 + R + max|z| / tau + |lse|)
lse within E; loss within tau^2 (E + 4 u (R_t + R_q)) where R_t, R_q are the
spans of the teacher's and the student's logits at the list, in units of tau;
the gradient within weight tau (q + P) E', E' likewise, plus half a bf16 step.
"""
import numpy as np
import pytest
import torch

import gemm_amax_reduce_amd as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOWEST = {"bf16": torch.finfo(torch.bfloat16).min, "f32": torch.finfo(torch.float32).min}


def _reference(z, idx, t, tau):
    """(loss, lse, q, P, some) in float64 on the CPU; q the student's shares,
    P the teacher's by vocabulary entry."""
    z, t, idx = z.double().cpu().numpy(), t.double().cpu().numpy(), idx.cpu().numpy()
    tokens, vocab = z.shape
    with np.errstate(all="ignore"):
        zt = z / tau
        m = zt.max(1, keepdims=True)
        lse = (m + np.log(np.exp(zt - m).sum(1, keepdims=True)))[:, 0]
        q = np.exp(zt - lse[:, None])
    loss, P, some = np.zeros(tokens), np.zeros((tokens, vocab)), np.zeros(tokens, bool)
    for r in range(tokens):
        ok = (idx[r] >= 0) & (idx[r] < vocab) & (t[r] != -np.inf) if idx.shape[1] else np.zeros(0, bool)
        if not ok.any():
            continue
        some[r] = True
        with np.errstate(all="ignore"):
            a = t[r][ok] / tau
            lp = a - a.max()
            lp -= np.log(np.exp(lp).sum())
            p = np.exp(lp)
            at = idx[r][ok]
            live = p > 0
            loss[r] = tau * tau * np.sum(p[live] * (lp[live] - (zt[r][at[live]] - lse[r])))
            np.add.at(P[r], at, p)
    return loss, lse, q, P, some


def _bounds(z, idx, t, tau, lse):
    zd = z.double().cpu().numpy()
    big = np.abs(zd[np.isfinite(zd) & (np.abs(zd) < 1e30)]).max(initial=0.0)
    e = 4 * U * (z.shape[1] / 256 + 64 + 70 + big / tau + np.abs(lse))
    return e, 4 * U * (2 * big + 70 * tau + _span(t)) / tau


def _span(t):
    td = t.double().cpu().numpy()
    td = td[np.isfinite(td) & (np.abs(td) < 1e30)]
    return float(td.max(initial=0.0) - td.min(initial=0.0))


def _check(z, idx, t, tau, weight, outputs, label):
    loss, lse, grad = outputs
    want_loss, want_lse, q, P, some = _reference(z, idx, t, tau)
    e, lists = _bounds(z, idx, t, tau, want_lse)
    got = lse.double().cpu().numpy()
    assert np.all(np.abs(got - want_lse) <= e + 1e-40), label
    got = loss.double().cpu().numpy()
    worst = np.max(np.abs(got - want_loss) / (tau * tau * (e + lists) + 1e-40), initial=0.0)
    assert np.all(got[~some] == 0)
    if grad is not None:
        w = weight.double().cpu().numpy()[:, None] * some[:, None]
        with np.errstate(all="ignore"):
            want = np.where(w != 0, w * tau * (q - P), 0.0)
            bound = np.where(w != 0, np.abs(w) * tau * (q + P) * (e + lists)[:, None], 0.0) + 1e-37
        if grad.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
        g = grad.double().cpu().numpy()
        worst_g = np.max(np.abs(g - want) / bound, initial=0.0)
        print(f"[distill] {label}: worst error / bound, loss {worst:.3f} gradient {worst_g:.3f}", flush=True)
        assert np.all(np.abs(g - want) <= bound), label
        assert np.all(g[~some] == 0)
    assert worst <= 1, label


def _inputs(tokens, vocab, top, dt, seed, pad=0, shift=0, idx_dtype=torch.int64, t_dtype=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    full = spread * torch.randn((tokens, vocab), generator=g)
    flat = torch.full((shift + tokens * (vocab + pad),), float("nan"), dtype=DT[dt], device="cuda")
    z = flat[shift:].view(tokens, vocab + pad)[:, :vocab]
    z.copy_((full * 0.8 + torch.randn((tokens, vocab), generator=g)).to(DT[dt]))
    best = torch.topk(full, min(top, vocab), 1)
    idx, t = best.indices.to(idx_dtype), best.values.to(t_dtype)
    weight = torch.rand(tokens, generator=g) + 0.1
    if tokens > 2 and top:
        idx[1] = -1                                                   # a padding token
        idx[2, (idx.shape[1] + 1) // 2:] = -1                         # a short list
        weight[0] = 0.0
    return z, idx.cuda().contiguous(), t.cuda().contiguous(), weight.cuda()


def _all(z, idx, t, tau, weight):
    """Both ways to the gradient."""
    loss, lse = nv.nvfp4_distill_topk(z, idx, t, temperature=tau)
    grad = nv.nvfp4_distill_topk_backward(z, idx, t, lse, weight, temperature=tau)
    return (loss, lse, grad), nv.nvfp4_distill_topk_step(z, idx, t, weight, temperature=tau)


SIZES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 8, 8), (3, 9, 4), (6, 255, 1), (2, 2049, 64), (7, 4096, 20),
         (3, 8193, 5), (300, 1000, 16), (2, 32768, 64), (5, 50021, 200), (1, 131072, 1024)]


@pytest.mark.parametrize("tokens,vocab,top", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_loss_and_gradient(tokens, vocab, top, dt, tau):
    args = _inputs(tokens, vocab, top, dt, tokens * 7 + vocab)
    z, idx, t, weight = args
    print(f"[distill] {tokens}x{vocab} top {top} {dt} tau {tau}", flush=True)
    pair, step = _all(z, idx, t, tau, weight)
    _check(z, idx, t, tau, weight, pair, "pair")
    _check(z, idx, t, tau, weight, step, "step")


@pytest.mark.parametrize("dt,idx_dtype,t_dtype", [("bf16", torch.int32, torch.bfloat16),
                                                  ("f32", torch.int32, torch.bfloat16),
                                                  ("bf16", torch.int64, torch.float32)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 1), (27, 3)])
def test_types_strides_alignment(dt, idx_dtype, t_dtype, pad, shift):
    z, idx, t, weight = _inputs(6, 3001, 33, dt, 5, pad, shift, idx_dtype, t_dtype)
    base = torch.full((6, 3001 + 5), 9.0, dtype=DT[dt], device="cuda")
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, weight, temperature=0.7, out=base[:, :3001])
    _check(z, idx, t, 0.7, weight, (loss, lse, grad), "strided")
    assert torch.all(base[:, 3001:] == 9.0)
    grad2 = nv.nvfp4_distill_topk_backward(z, idx, t, lse, weight, temperature=0.7)
    _check(z, idx, t, 0.7, weight, (loss, lse, grad2), "strided backward")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 20001])
def test_masked_vocabulary(dt, vocab):
    """A padded vocabulary, masked by -inf or by the type's lowest value."""
    for mask in (float("-inf"), LOWEST[dt]):
        z, idx, t, weight = _inputs(4, vocab, 6, dt, 11)
        hide = torch.ones_like(z, dtype=torch.bool)
        hide.scatter_(1, idx.clamp(min=0), False)
        hide[:, : vocab // 2] = False
        z[hide] = mask
        pair, step = _all(z, idx, t, 1.0, weight)
        _check(z, idx, t, 1.0, weight, pair, "pair")
        _check(z, idx, t, 1.0, weight, step, "step")
        assert torch.all(step[2][hide] == 0) and torch.all(pair[2][hide] == 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_all_logits_lowest(dt):
    """A row held entirely at the type's lowest value is a uniform row."""
    z = torch.full((2, 300), LOWEST[dt], dtype=DT[dt], device="cuda")
    idx = torch.tensor([[5, 7], [1, 2]], device="cuda")
    t = torch.full((2, 2), torch.finfo(torch.float32).min, device="cuda")
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, torch.ones(2, device="cuda"))
    # p = 1/2 each, q = 1/300: loss = log(300 / 2), gradient 1/300 and 1/300 - 1/2
    assert np.allclose(loss.cpu().numpy(), np.log(150.0), rtol=1e-6)
    want = torch.full((2, 300), 1 / 300, dtype=torch.float64)
    want.scatter_add_(1, idx.cpu(), torch.full((2, 2), -0.5, dtype=torch.float64))
    tol = 2.0 ** -8 if dt == "bf16" else 1e-6
    assert torch.allclose(grad.double().cpu(), want, rtol=tol, atol=0)


@pytest.mark.parametrize("vocab", [50, 9000])
def test_empty_rows_ignore_their_logits(vocab):
    """No valid entry: loss 0 and gradient 0 even where the logits are NaN."""
    z, idx, t, weight = _inputs(5, vocab, 4, "f32", 13)
    idx[0], idx[3] = -1, vocab                     # past the end is absent, too
    t[4] = float("-inf")
    z[0], z[3, 5], z[4] = float("nan"), float("inf"), float("-inf")
    weight[:] = 0.5
    pair, step = _all(z, idx, t, 1.0, weight)
    for loss, _, grad in (pair, step):
        for r in (0, 1, 3, 4):
            assert loss[r] == 0 and torch.all(grad[r] == 0)
        assert torch.isfinite(loss).all() and torch.isfinite(grad).all()


def test_no_list_at_all():
    z = torch.randn((3, 64), device="cuda")
    idx, t = torch.empty((3, 0), dtype=torch.int64, device="cuda"), torch.empty((3, 0), device="cuda")
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, torch.ones(3, device="cuda"))
    assert torch.all(loss == 0) and torch.all(grad == 0)
    assert torch.allclose(lse, torch.logsumexp(z.double(), 1).float(), rtol=1e-5)


def test_no_tokens():
    z = torch.empty((0, 64), device="cuda")
    idx, t = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, torch.empty(0, device="cuda"))
    assert loss.shape == (0,) and lse.shape == (0,) and grad.shape == (0, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeated_indices_add(dt):
    z, idx, t, weight = _inputs(4, 5000, 12, dt, 17)
    idx[0, 3:7] = idx[0, 0]
    idx[3, :] = 4999
    weight[:] = 1.0
    pair, step = _all(z, idx, t, 1.0, weight)
    _check(z, idx, t, 1.0, weight, pair, "pair")
    _check(z, idx, t, 1.0, weight, step, "step")


def test_student_excludes_a_listed_entry():
    """The teacher wants an entry that the student masks: infinite loss, a
    finite gradient."""
    z, idx, t, weight = _inputs(1, 100, 3, "f32", 19)
    z[0, idx[0, 1]] = float("-inf")
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    assert torch.isinf(loss).all() and torch.isfinite(grad).all()
    p = torch.softmax(t.double(), 1)
    assert abs(grad[0, idx[0, 1]].item() + weight[0].item() * p[0, 1].item()) < 1e-6


def test_large_logits_and_sharp_lists():
    """Logits in the thousands, teacher shares down to nothing."""
    z, idx, t, weight = _inputs(4, 3000, 8, "f32", 23, spread=700.0)
    t[0, 4:] -= 1e5
    weight[:] = 1.0
    pair, step = _all(z, idx, t, 1.0, weight)
    _check(z, idx, t, 1.0, weight, pair, "pair")
    _check(z, idx, t, 1.0, weight, step, "step")


def test_nan_row_stays_alone():
    z, idx, t, weight = _inputs(4, 12000, 5, "bf16", 29)
    clean = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    bad = z.clone()
    bad[3, 7000] = float("nan")
    loss, lse, grad = nv.nvfp4_distill_topk_step(bad, idx, t, weight)
    assert torch.isnan(loss[3]) and torch.isnan(lse[3]) and torch.isnan(grad[3]).all()
    assert torch.equal(loss[:3], clean[0][:3]) and torch.equal(grad[:3], clean[2][:3])


def test_gradient_against_differences():
    tokens, vocab, tau = 3, 60, 1.7
    z, idx, t, weight = _inputs(tokens, vocab, 6, "f32", 31)
    _, step = _all(z, idx, t, tau, weight)
    grad = step[2].double().cpu().numpy()
    w = weight.double().cpu().numpy()
    v = torch.randn((tokens, vocab), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    h = 1e-4
    zd = z.double().cpu()
    hi, lo = _reference(zd + h * v, idx, t, tau)[0], _reference(zd - h * v, idx, t, tau)[0]
    numeric = (w * (hi - lo)).sum() / (2 * h)
    _, lse, q, P, some = _reference(z, idx, t, tau)
    e, lists = _bounds(z, idx, t, tau, lse)
    bound = ((w * some)[:, None] * tau * (q + P) * (e + lists)[:, None] * np.abs(v.numpy())).sum()
    # the differences' own error: third derivatives below 1 times the step squared
    assert abs((grad * v.numpy()).sum() - numeric) <= bound + h * h * (w[:, None] * np.abs(v.numpy()) ** 3).sum()


def test_rows_past_one_launch():
    """More rows than a grid dimension holds."""
    tokens = 65535 + 70
    z, idx, t, weight = _inputs(tokens, 9, 2, "f32", 37)
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    for s in (slice(0, 50), slice(65500, 65600), slice(tokens - 5, tokens)):
        _check(z[s], idx[s], t[s], 1.0, weight[s], (loss[s], lse[s], grad[s]), f"rows {s.start}")
    back = nv.nvfp4_distill_topk_backward(z, idx, t, lse, weight)
    # the two ways differ by 4 u (64 + 70 + 2 * 15) of a share, below 1 each here
    assert torch.allclose(back, grad, rtol=0, atol=2 * 4 * U * 164)


@pytest.mark.parametrize("dt,tokens,vocab", [("bf16", 8300, 8190), ("bf16", 2100, 32801), ("bf16", 1100, 65537),
                                             ("bf16", 521, 131101), ("f32", 8300, 4099), ("f32", 1040, 33001),
                                             ("f32", 500, 70003)])
def test_large_calls(dt, tokens, vocab):
    """More logits than the last cache holds; some of the rows are checked."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = (3 * torch.randn((tokens, vocab), generator=g, device="cuda")).to(DT[dt])
    idx = torch.randint(-1, vocab, (tokens, 20), generator=g, device="cuda")
    t = 2 * torch.randn((tokens, 20), generator=g, device="cuda")
    weight = torch.rand(tokens, generator=g, device="cuda")
    print(f"[distill] {tokens}x{vocab} {dt}", flush=True)
    rows = torch.tensor([0, 1, tokens // 2, tokens - 2, tokens - 1], device="cuda")
    for label, out in zip(("pair", "step"), _all(z, idx, t, 1.5, weight)):
        _check(z[rows], idx[rows], t[rows], 1.5, weight[rows], [o[rows] for o in out], label)


def test_other_stream_and_repeat():
    z, idx, t, weight = _inputs(9, 40000, 32, "bf16", 41)
    want = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    again = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.nvfp4_distill_topk_step(z, idx, t, weight, stream=side)
    back = nv.nvfp4_distill_topk_backward(z, idx, t, got[1], weight, stream=side)
    side.synchronize()
    for p, q, r in zip(want, again, got):
        assert torch.equal(p, q) and torch.equal(p, r)
    assert torch.equal(back, nv.nvfp4_distill_topk_backward(z, idx, t, want[1], weight))


def test_graph_replays():
    z, idx, t, weight = _inputs(6, 20000, 16, "bf16", 43)
    nv.nvfp4_distill_topk_step(z, idx, t, weight)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.nvfp4_distill_topk_step(z, idx, t, weight)
    for turn in range(4):
        z.copy_(_inputs(6, 20000, 16, "bf16", 50 + turn)[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, nv.nvfp4_distill_topk_step(z, idx, t, weight)):
            assert torch.equal(p, q)


def test_offsets_past_32_bits():
    """2.2e9 logits: sampled rows."""
    tokens, vocab = 17000, 131080
    assert tokens * vocab > 2 ** 31
    few, idx, t, weight = _inputs(17, vocab, 16, "bf16", 47)
    z = few.repeat(1000, 1)
    loss, lse, grad = nv.nvfp4_distill_topk_step(z, idx.repeat(1000, 1), t.repeat(1000, 1), weight.repeat(1000))
    for rep in (0, 499, 999):
        s = slice(17 * rep, 17 * rep + 17)
        _check(few, idx, t, 1.0, weight, (loss[s], lse[s], grad[s]), f"rows from {17 * rep}")
