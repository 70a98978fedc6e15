"""Measured cases of the operators that surround the 4-bit linear layer: layer
norm (forward; backward with the weight and bias gradients), matrix-vector
products with 4-bit weights, and distillation from a teacher's top logits.

``run`` computes each operator in its plain form (elementary torch operations
in float32, rounded once at the end) or, with ``own`` set, through the
package's entry points.  ``exact`` gives the same outputs from the definitions
in float64.

The widths are those of this repository's layer shapes (5120-wide model,
20480-wide MLP, the 32768 x 8192 sweep) or generic vocabularies; odd sizes and
padded row strides stand for vocabularies and batches that divide by nothing.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # the final norm of one answered token: launch latency
        {"name": "norm_1x5120", "op": "norm", "rows": 1, "cols": 5120, "pad": 0, "dtype": "bf16", "wdtype": "bf16",
         "amax": False},
        # a prompt's activations before the quantizer, which takes the maximum from here
        {"name": "norm_4096x5120_amax", "op": "norm", "rows": 4096, "cols": 5120, "pad": 0, "dtype": "bf16",
         "wdtype": "bf16", "amax": True},
        # the norm of a training batch in reverse
        {"name": "norm_bwd_8192x5120", "op": "norm_bwd", "rows": 8192, "cols": 5120, "pad": 0, "dtype": "bf16",
         "wdtype": "bf16"},
        # a ragged float32 batch, rows padded apart
        {"name": "norm_bwd_1537x5003", "op": "norm_bwd", "rows": 1537, "cols": 5003, "pad": 5, "dtype": "f32",
         "wdtype": "f32"},
        # the largest training batch, the sweep's tensor
        {"name": "norm_bwd_32768x8192", "op": "norm_bwd", "rows": 32768, "cols": 8192, "pad": 0, "dtype": "bf16",
         "wdtype": "f32"},
        # one token through the square projection: latency
        {"name": "matvec_1x5120x5120", "op": "matvec", "format": "nvfp4", "tokens": 1, "n": 5120, "k": 5120,
         "dtype": "bf16", "out": "bf16"},
        # one token through the MLP's wide projection
        {"name": "matvec_1x20480x5120", "op": "matvec", "format": "nvfp4", "tokens": 1, "n": 20480, "k": 5120,
         "dtype": "bf16", "out": "bf16"},
        # eight tokens answered together through a head of odd size, float32 logits; past the last-level cache
        {"name": "matvec_8x131075x5120", "op": "matvec", "format": "nvfp4", "tokens": 8, "n": 131075, "k": 5120,
         "dtype": "bf16", "out": "f32"},
        # a few tokens through the MLP's long reduction, MXFP4 weights, float32 activations
        {"name": "matvec_mx_5x5120x20480", "op": "matvec", "format": "mxfp4", "tokens": 5, "n": 5120, "k": 20480,
         "dtype": "f32", "out": "f32"},
        # the loss alone on a handful of held-out tokens: latency, few long rows
        {"name": "distill_loss_24x32768", "op": "distill", "kind": "loss", "tokens": 24, "vocab": 32768, "pad": 0,
         "top": 64, "dtype": "bf16", "tau": 1.0},
        # forward, then backward from the saved log-sum-exp, float32, odd vocabulary with padded rows
        {"name": "distill_pair_777x50021", "op": "distill", "kind": "pair", "tokens": 777, "vocab": 50021, "pad": 27,
         "top": 20, "dtype": "f32", "tau": 2.0},
        # loss and gradient of a training batch in one call
        {"name": "distill_step_4096x131072", "op": "distill", "kind": "step", "tokens": 4096, "vocab": 131072,
         "pad": 0, "top": 64, "dtype": "bf16", "tau": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "matvec", "distill"])
    if op in ("norm", "norm_bwd"):
        cols = _log_int(rng, 64, 20480)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, min(32768, 32768 * 8192 // cols // 2))
        case = {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 3, 16]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "wdtype": rng.choice(["bf16", "f32"])}
        if op == "norm":
            case["amax"] = rng.random() < 0.5
        return case
    if op == "matvec":
        fmt = rng.choice(["nvfp4", "mxfp4"])
        step = 16 if fmt == "nvfp4" else 32
        k = _log_int(rng, 256, 20480) // step * step
        n = _log_int(rng, 256, min(131075, 131075 * 5120 // k))
        return {"op": op, "format": fmt, "tokens": _log_int(rng, 1, 16), "n": n, "k": k,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
    vocab = _log_int(rng, 1000, 131072)
    if rng.random() < 0.5:
        vocab = vocab // 8 * 8
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 4096 * 131072 // vocab // (1 if dtype == "bf16" else 2)
    return {"op": op, "kind": rng.choice(["loss", "pair", "step"]), "tokens": _log_int(rng, 1, min(8192, most // 2)),
            "vocab": vocab, "pad": rng.choice([0, 0, 11, 64]), "top": _log_int(rng, 4, 256), "dtype": dtype,
            "tau": rng.choice([1.0, 1.0, 2.0, 0.7])}


# ------------------------------------------------------------------ inputs --

def _rows(rows, cols, pad, dtype):
    """An empty [rows, cols] matrix whose rows lie `pad` elements apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def _norm_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, dt, wdt = case["rows"], case["cols"], _DT[case["dtype"]], _DT[case["wdtype"]]
    # activations: unit spread about a channel's own offset, each row of its own size, a few channels far out
    v = torch.randn((rows, cols), device="cuda", generator=g)
    v *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=g))
    v += 0.3 * torch.randn((1, cols), device="cuda", generator=g)
    v *= 1 + 20.0 * (torch.rand((1, cols), device="cuda", generator=g) < 2e-3)
    x = _rows(rows, cols, case["pad"], dt)
    x.copy_(v)
    state = {"x": x,
             "weight": (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(wdt),
             "bias": (0.1 * torch.randn(cols, device="cuda", generator=g)).to(wdt)}
    if case["op"] == "norm_bwd":
        dy = _rows(rows, cols, case["pad"], dt)
        u = torch.rand((rows, cols), device="cuda", generator=g) - 0.5
        dy.copy_(-1e-3 * torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999)))   # Laplace, as dY is
        xf = x.float()
        mean = xf.mean(1)
        state.update(dy=dy, mean=mean, rstd=torch.rsqrt(((xf - mean[:, None]) ** 2).mean(1) + EPS))
    return state


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _matvec_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, k, m = case["n"], case["k"], case["tokens"]
    w = 0.02 * torch.randn((n, k), device="cuda", generator=g)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    if case["format"] == "nvfp4":
        amax = w.abs().max()
        blocks = w.view(n, k // 16, 16)
        s8 = (blocks.abs().amax(2) * (448.0 / amax)).to(torch.float8_e4m3fn)
        s = s8.float() * (amax / 2688.0)
        scales, meta = s8.view(torch.uint8), torch.stack([amax, amax / 2688.0])
    else:
        blocks = w.view(n, k // 32, 32)
        e = torch.ceil(torch.log2(blocks.abs().amax(2) / 6.0)).clamp(-127, 127)
        s = torch.exp2(e)
        scales, meta = (e + 127).to(torch.uint8), None
    blocks /= s[..., None].clamp(min=1e-30)
    codes = torch.bucketize(blocks.abs(), mids, out_int32=True).to(torch.uint8)
    codes |= (blocks < 0).to(torch.uint8) << 3
    codes = codes.view(n, k // 2, 2)
    codes = (codes[..., 0] | (codes[..., 1] << 4)).contiguous()
    x = torch.randn((m, k), device="cuda", generator=g)
    x *= 1 + 49.0 * (torch.rand((m, k), device="cuda", generator=g) < 1e-3)
    state = {"codes": codes, "scales": scales.contiguous(), "meta": meta, "x": x.to(_DT[case["dtype"]])}
    if own:
        import gemm_amax_reduce_amd as nv
        if case["format"] == "nvfp4":
            state["w"] = nv.NVFP4Tensor(codes, state["scales"], meta, n, k)
        else:
            state["w"] = nv.MXFP4Tensor(codes, state["scales"], n, k)
    return state


def _distill_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, v, top, dt = case["tokens"], case["vocab"], case["top"], _DT[case["dtype"]]
    z = _rows(t, v, case["pad"], dt)
    idx = torch.empty((t, top), dtype=torch.int64, device="cuda")
    tz = torch.empty((t, top), dtype=torch.float32, device="cuda")
    for r in range(0, t, 512):                     # the teacher's logits, of which the best are kept
        e = min(t, r + 512)
        full = 2.5 * torch.randn((e - r, v), device="cuda", generator=g)
        best = torch.topk(full, top, dim=1)
        idx[r:e], tz[r:e] = best.indices, best.values
        full *= 0.8                                # the student: near the teacher, with noise of its own
        full += torch.randn((e - r, v), device="cuda", generator=g)
        z[r:e].copy_(full)
    # shorter lists, padding tokens with none at all, and their weights
    count = torch.randint(max(1, top // 2), top + 1, (t, 1), device="cuda", generator=g)
    count[torch.rand((t, 1), device="cuda", generator=g) < 0.03] = 0
    idx[torch.arange(top, device="cuda")[None] >= count] = -1
    weight = (count[:, 0] > 0).float()
    weight /= weight.sum().clamp(min=1)
    return {"z": z, "idx": idx, "tz": tz, "weight": weight}


def prepare(case, seed):
    if case["op"] in ("norm", "norm_bwd"):
        state = _norm_inputs(case, seed)
    elif case["op"] == "matvec":
        state = _matvec_inputs(case, seed)
    else:
        state = _distill_inputs(case, seed)
    state["case"] = case
    return state


# ------------------------------------------------------------- plain forms --

def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = (d * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(_DT[c["dtype"]])
    return (y, mean, rstd, y.abs().max().float().reshape(1)) if c["amax"] else (y, mean, rstd)


def _plain_norm_bwd(s):
    x, dy, mean, rstd = s["x"].float(), s["dy"].float(), s["mean"][:, None], s["rstd"][:, None]
    xh = (x - mean) * rstd
    a = dy * s["weight"].float()
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _decode(s, dtype):
    """The 4-bit weights as a [n, k] matrix of `dtype`."""
    c = s["case"]
    lut = torch.tensor(_E2M1 + tuple(-q for q in _E2M1), dtype=dtype, device="cuda")
    codes = s["codes"]
    q = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], dim=2)
    if c["format"] == "nvfp4":
        scale = s["scales"].view(torch.float8_e4m3fn).to(dtype) * s["meta"][1].to(dtype)
    else:
        scale = torch.exp2(s["scales"].to(dtype) - 127)
    q = q.view(c["n"], scale.shape[1], -1)
    q *= scale[..., None]
    return q.view(c["n"], c["k"])


def _plain_matvec(s):
    return (s["x"].float() @ _decode(s, torch.float32).t()).to(_DT[s["case"]["out"]])


def _distill(s, dtype, weighted):
    """(loss, lse, gradient or None) in `dtype`, the gradient for the rows' weights."""
    c = s["case"]
    tau, v = c["tau"], c["vocab"]
    z = s["z"].to(dtype) / tau
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    valid = (s["idx"] >= 0) & (s["idx"] < v)
    some = valid.any(1)
    at = torch.where(valid, s["idx"], 0)
    t = s["tz"].to(dtype) / tau
    t = torch.where(valid, t, -math.inf)
    t = t - torch.where(some, t.amax(1), 0.0)[:, None]
    total = torch.where(some, torch.exp(t).sum(1), 1.0)[:, None]
    p = torch.exp(t) / total
    logp = torch.where(p > 0, t - torch.log(total), 0.0)
    loss = tau * tau * (p * (logp - (z.gather(1, at) - lse[:, None]))).sum(1)
    loss = torch.where(some, loss, 0.0)
    if not weighted:
        return loss, lse, None
    grad = torch.exp(z - lse[:, None])
    grad.scatter_add_(1, at, -p)
    grad *= torch.where(some, tau * s["weight"].to(dtype), 0.0)[:, None]
    return loss, lse, grad


def _plain_distill(s):
    loss, lse, grad = _distill(s, torch.float32, s["case"]["kind"] != "loss")
    return (loss, lse) if grad is None else (loss, lse, grad.to(s["z"].dtype))


# ---------------------------------------------------------------- one pass --

def run(state):
    c = state["case"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "matvec": _plain_matvec,
                "distill": _plain_distill}[c["op"]](state)
    import gemm_amax_reduce_amd as nv
    s = state
    if c["op"] == "norm":
        return nv.nvfp4_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, amax=c["amax"])
    if c["op"] == "norm_bwd":
        return nv.nvfp4_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if c["op"] == "matvec":
        matvec = nv.nvfp4_matvec if c["format"] == "nvfp4" else nv.mxfp4_matvec
        return matvec(s["w"], s["x"], out_dtype=_DT[c["out"]])
    if c["kind"] == "loss":
        return nv.nvfp4_distill_topk(s["z"], s["idx"], s["tz"], temperature=c["tau"])
    if c["kind"] == "step":
        return nv.nvfp4_distill_topk_step(s["z"], s["idx"], s["tz"], s["weight"], temperature=c["tau"])
    loss, lse = nv.nvfp4_distill_topk(s["z"], s["idx"], s["tz"], temperature=c["tau"])
    return loss, lse, nv.nvfp4_distill_topk_backward(s["z"], s["idx"], s["tz"], lse, s["weight"],
                                                     temperature=c["tau"])


def work(case):
    """What a pass cannot do without: each input read once, each output
    written once, and the operations of the formulas."""
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        n, s, ws = c["rows"] * c["cols"], _SIZE[c["dtype"]], _SIZE[c["wdtype"]]
        if c["op"] == "norm":
            return {"bytes": 2 * n * s + 2 * c["cols"] * ws + 8 * c["rows"] + (4 if c["amax"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * s + c["cols"] * (ws + 8) + 8 * c["rows"], "flops": 15 * n}
    if c["op"] == "matvec":
        m, n, k = c["tokens"], c["n"], c["k"]
        group = 16 if c["format"] == "nvfp4" else 32
        return {"bytes": n * k // 2 + n * (k // group) + m * k * _SIZE[c["dtype"]] + m * n * _SIZE[c["out"]],
                "flops": 2 * m * n * k}
    n, lists = c["tokens"] * c["vocab"], c["tokens"] * c["top"] * 12
    reads = n * _SIZE[c["dtype"]] + lists
    if c["kind"] == "loss":
        return {"bytes": reads + 8 * c["tokens"], "flops": 5 * n}
    return {"bytes": reads + n * _SIZE[c["dtype"]] + 12 * c["tokens"], "flops": 9 * n}


# ------------------------------------------------------ the 64-bit results --

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] == "norm":
        x = s["x"].double()
        mean = x.sum(1) / c["cols"]
        var = torch.square(x - mean[:, None]).sum(1) / c["cols"]
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = s["bias"].double() + s["weight"].double() * ((x - mean[:, None]) * rstd[:, None])
        if not c["amax"]:
            return y, mean, rstd
        # the maximum is that of the values as they are stored
        return y, mean, rstd, y.to(_DT[c["dtype"]]).double().abs().max().reshape(1)
    if c["op"] == "norm_bwd":
        r = s["rstd"].double()[:, None]
        xh = s["x"].double().sub_(s["mean"].double()[:, None]).mul_(r)
        dy = s["dy"].double()
        db, dw = dy.sum(0), (dy * xh).sum(0)
        a = dy.mul_(s["weight"].double())
        a_mean, a_xh = a.sum(1, keepdim=True) / c["cols"], (a * xh).sum(1, keepdim=True) / c["cols"]
        return a.sub_(a_mean).sub_(xh.mul_(a_xh)).mul_(r), dw, db
    if c["op"] == "matvec":
        x = s["x"].double()
        out = torch.empty((c["tokens"], c["n"]), dtype=torch.float64, device="cuda")
        grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        for r in range(0, c["n"], 8192):
            codes = s["codes"][r:r + 8192]
            w = torch.empty((codes.shape[0], c["k"]), dtype=torch.float64, device="cuda")
            for half, nib in ((0, codes & 15), (1, codes >> 4)):
                w[:, half::2] = grid[(nib & 7).long()] * (1 - 2 * (nib >> 3).double())
            sc = s["scales"][r:r + 8192]
            if c["format"] == "nvfp4":
                sc = sc.view(torch.float8_e4m3fn).double()
                w *= sc.repeat_interleave(16, 1)
                out[:, r:r + 8192] = (x @ w.t()) * s["meta"][1].double()
            else:
                w *= torch.pow(2.0, sc.double() - 127).repeat_interleave(32, 1)
                out[:, r:r + 8192] = x @ w.t()
        return out
    return _exact_distill(c, s)


def _exact_distill(c, s):
    t, v, tau = c["tokens"], c["vocab"], c["tau"]
    loss = torch.zeros(t, dtype=torch.float64, device="cuda")
    lse = torch.empty(t, dtype=torch.float64, device="cuda")
    grad = None if c["kind"] == "loss" else torch.empty((t, v), dtype=torch.float64, device="cuda")
    idx = s["idx"].clone()
    idx[(idx < 0) | (idx >= v)] = v                       # one column past the end takes what is absent
    for r in range(0, t, 256):
        i = idx[r:r + 256]
        z = s["z"][r:r + 256].double() / tau
        l = torch.logsumexp(z, 1)
        lse[r:r + 256] = l
        teacher = torch.full((i.shape[0], v + 1), -math.inf, dtype=torch.float64, device="cuda")
        teacher.scatter_(1, i, s["tz"][r:r + 256].double() / tau)
        teacher = teacher[:, :v]
        none = torch.isinf(teacher).all(1)
        logp = teacher - torch.logsumexp(teacher, 1, keepdim=True)
        p = torch.exp(logp)
        p[none] = 0.0
        terms = torch.where(p > 0, p * (logp - (z - l[:, None])), 0.0)
        loss[r:r + 256] = tau * tau * terms.sum(1)
        if grad is not None:
            grad[r:r + 256] = tau * s["weight"][r:r + 256].double()[:, None] * (torch.exp(z - l[:, None]) - p)
            grad[r:r + 256][none] = 0.0
    return (loss, lse) if grad is None else (loss, lse, grad)
