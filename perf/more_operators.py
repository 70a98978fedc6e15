"""Measured cases of the operators of a block around 4-bit layers: root-mean-
square norm with the residual's addition (forward, in 16 or 32 bits or in
MXFP8; backward), matrix products grouped by expert with 4-bit weights
(forward, data gradient, weight gradient), and low-rank adapters of many
requests beside a shared projection (forward and backward).

``run`` computes each operator in its plain form (elementary torch operations
in float32, rounded once at the end; rows of a group padded to a batch) or,
with ``own`` set, through the package's entry points.  ``exact`` gives the
same outputs from the definitions in float64.

The widths are those of this repository's layer shapes (5120-wide model,
20480-wide MLP) or generic; group sizes are drawn from a case's own values, so
that all its inputs have the same ones.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one answered token between two layers, residual added: launch latency
        {"name": "rms_1x5120", "op": "rms", "rows": 1, "cols": 5120, "pad": 0, "dtype": "bf16", "wdtype": "bf16",
         "residual": "bf16", "out": "bf16"},
        # a prompt's activations on their way into an MXFP8 product, the residual stream in float32
        {"name": "rms_mx8_4096x5120", "op": "rms", "rows": 4096, "cols": 5120, "pad": 0, "dtype": "bf16",
         "wdtype": "bf16", "residual": "f32", "out": "mxfp8"},
        # a training batch in reverse, with the residual stream's gradient
        {"name": "rms_bwd_8192x5120", "op": "rms_bwd", "rows": 8192, "cols": 5120, "pad": 0, "dtype": "bf16",
         "wdtype": "bf16", "dh": True},
        # a ragged float32 batch, rows padded apart
        {"name": "rms_bwd_1537x5003", "op": "rms_bwd", "rows": 1537, "cols": 5003, "pad": 5, "dtype": "f32",
         "wdtype": "f32", "dh": False},
        # eight answered tokens with two experts each: few rows a group, the weights are what is read
        {"name": "experts_16_of_32x2048x5120", "op": "experts", "format": "mxfp4", "experts": 32, "tokens": 16,
         "n": 2048, "k": 5120, "skew": 1.0, "rest": 0, "transposed": False, "dtype": "bf16", "out": "bf16"},
        # the data gradient of a ragged batch, experts without a row, the batch padded at its end
        {"name": "experts_dgrad_1531_of_24x5120x1280", "op": "experts", "format": "nvfp4", "experts": 24,
         "tokens": 1531, "n": 5120, "k": 1280, "skew": 2.0, "rest": 37, "transposed": True, "dtype": "f32",
         "out": "f32"},
        # a prompt through the wide projection of eight experts: the largest product
        {"name": "experts_4096_of_8x20480x5120", "op": "experts", "format": "nvfp4", "experts": 8, "tokens": 4096,
         "n": 20480, "k": 5120, "skew": 0.5, "rest": 0, "transposed": False, "dtype": "bf16", "out": "bf16"},
        # the experts' weight gradients of a training batch
        {"name": "experts_wgrad_8192_of_8x5120x5120", "op": "wgrad", "experts": 8, "tokens": 8192, "n": 5120,
         "k": 5120, "skew": 0.5, "rest": 0, "dtype": "bf16", "out": "f32"},
        # few rows for each of many experts, odd sizes, float32
        {"name": "experts_wgrad_777_of_16x1283x2050", "op": "wgrad", "experts": 16, "tokens": 777, "n": 1283,
         "k": 2050, "skew": 1.5, "rest": 5, "dtype": "f32", "out": "f32"},
        # 24 requests, one token each, beside the square projection: latency
        {"name": "adapters_24x5120x5120", "op": "adapters", "segments": 24, "tokens": 24, "adapters": 32, "rank": 16,
         "n": 5120, "k": 5120, "skew": 0.0, "rest": 0, "dtype": "bf16", "wdtype": "bf16", "base": True},
        # five prompts of odd lengths beside the wide projection
        {"name": "adapters_4099x20480x5120", "op": "adapters", "segments": 5, "tokens": 4099, "adapters": 4,
         "rank": 32, "n": 20480, "k": 5120, "skew": 1.0, "rest": 0, "dtype": "bf16", "wdtype": "bf16", "base": True},
        # a training batch of several adapters in reverse
        {"name": "adapters_bwd_8192x5120x5120", "op": "adapters_bwd", "segments": 12, "tokens": 8192, "adapters": 6,
         "rank": 16, "n": 5120, "k": 5120, "skew": 0.5, "rest": 0, "dtype": "bf16", "wdtype": "bf16", "base": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rms", "rms_bwd", "experts", "experts", "wgrad", "adapters", "adapters_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rms", "rms_bwd"):
        out = rng.choice(["mxfp8", "mxfp8", "bf16", "f32"])
        cols = _log_int(rng, 64, 20480)
        if rng.random() < 0.5 or (op == "rms" and out == "mxfp8"):
            cols = max(64, cols // 32 * 32)
        case = {"op": op, "rows": _log_int(rng, 1, min(32768, 100_000_000 // cols)), "cols": cols,
                "pad": rng.choice([0, 0, 3, 16]), "dtype": dtype, "wdtype": rng.choice(["bf16", "f32"])}
        if op == "rms":
            case.update(residual=rng.choice(["none", "bf16", "f32"]), out=out)
        else:
            case.update(dh=rng.random() < 0.5)
        return case
    if op == "experts":
        k = _log_int(rng, 256, 8192) // 32 * 32
        n = _log_int(rng, 256, 8192) // 32 * 32
        experts = _log_int(rng, 1, min(64, 400_000_000 // (n * k)))
        tokens = _log_int(rng, 1, min(8192, 200_000_000_000 // (n * k)))
        return {"op": op, "format": rng.choice(["nvfp4", "mxfp4"]), "experts": experts, "tokens": tokens, "n": n,
                "k": k, "skew": rng.choice([0.0, 0.5, 1.0, 2.0]), "rest": rng.choice([0, 0, 9]),
                "transposed": rng.random() < 0.4, "dtype": dtype, "out": rng.choice(["bf16", "f32"])}
    if op == "wgrad":
        k, n = _log_int(rng, 128, 8192), _log_int(rng, 128, 8192)
        if rng.random() < 0.6:
            k, n = max(128, k // 64 * 64), max(128, n // 64 * 64)
        return {"op": op, "experts": _log_int(rng, 1, min(64, 200_000_000 // (n * k))),
                "tokens": _log_int(rng, 1, min(8192, 100_000_000_000 // (n * k))), "n": n, "k": k,
                "skew": rng.choice([0.0, 0.5, 1.0, 2.0]), "rest": rng.choice([0, 0, 9]), "dtype": dtype,
                "out": rng.choice(["f32", "f32", "bf16"])}
    k, n = _log_int(rng, 256, 20480), _log_int(rng, 256, 20480)
    if rng.random() < 0.6:
        k, n = max(256, k // 64 * 64), max(256, n // 64 * 64)
    tokens = _log_int(rng, 1, min(8192, 100_000_000 // max(k, n)))
    return {"op": op, "segments": _log_int(rng, 1, min(64, tokens)), "tokens": tokens,
            "adapters": _log_int(rng, 1, 32), "rank": rng.choice([4, 8, 16, 16, 24, 32, 64]), "n": n, "k": k,
            "skew": rng.choice([0.0, 0.5, 1.0, 2.0]), "rest": rng.choice([0, 0, 9]), "dtype": dtype,
            "wdtype": rng.choice([dtype, "bf16", "f32"]), "base": rng.random() < 0.7}


# ------------------------------------------------------------------ inputs --

def _rows(rows, cols, pad, dtype):
    """An empty [rows, cols] matrix whose rows lie `pad` elements apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def _group_sizes(case):
    """How the case's rows fall on its groups: evenly up to one row (skew 0),
    or by shares with a spread of exp(skew), small ones of which get none."""
    groups = case["segments"] if "segments" in case else case["experts"]
    tokens = case["tokens"]
    rng = random.Random("%d %d %g" % (groups, tokens, case["skew"]))
    share = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(groups)]
    total, ends, at = sum(share), [], 0.0
    for s in share:
        at += s
        ends.append(int(tokens * at / total + 0.5))
    ends[-1] = tokens
    return [e - b for b, e in zip([0] + ends, ends)]


def _groups(case):
    """(offsets on the device, each row's place in a batch of groups padded
    to the longest, the longest): what the plain form batches by."""
    sizes = _group_sizes(case)
    size = torch.tensor(sizes, device="cuda")
    end = torch.cumsum(size, 0)
    offsets = torch.cat([end.new_zeros(1), end]).to(torch.int32)
    longest = max(max(sizes), 1)
    group = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), size)
    place = torch.arange(case["tokens"], device="cuda") - (end - size)[group] + group * longest
    return offsets, group, place, longest


def _tokens(g, rows, cols, dtype):
    """Activations: unit spread, a few entries far out."""
    x = torch.randn((rows, cols), device="cuda", generator=g)
    x *= 1 + 49.0 * (torch.rand((rows, cols), device="cuda", generator=g) < 1e-3)
    return x.to(dtype)


def _gradients(g, rows, cols, dtype):
    """Laplace, as gradients are."""
    u = torch.rand((rows, cols), device="cuda", generator=g) - 0.5
    return (-1e-3 * torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))).to(dtype)


def _rms_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, pad, dt = case["rows"], case["cols"], case["pad"], _DT[case["dtype"]]

    def stream(dtype, size):
        # each row of its own size, a few channels far out
        v = size * torch.randn((rows, cols), device="cuda", generator=g)
        v *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=g))
        v *= 1 + 20.0 * (torch.rand((1, cols), device="cuda", generator=g) < 2e-3)
        t = _rows(rows, cols, pad, dtype)
        t.copy_(v)
        return t

    state = {"x": stream(dt, 1.0), "weight": (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(
        _DT[case["wdtype"]])}
    if case["op"] == "rms":
        if case["residual"] != "none":
            state["residual"] = stream(_DT[case["residual"]], 3.0)
        return state
    state["dy"] = _rows(rows, cols, pad, dt)
    state["dy"].copy_(_gradients(g, rows, cols, dt))
    state["dh"] = _gradients(g, rows, cols, dt) if case["dh"] else None
    state["rstd"] = torch.rsqrt((state["x"].float() ** 2).mean(1) + EPS)
    return state


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _stack(case):
    """The stored layout of the experts' weights: (rows, k)."""
    if case["transposed"]:                       # [n][experts * k], blocks along each expert's k
        return case["n"], case["experts"] * case["k"]
    return case["experts"] * case["n"], case["k"]


def _experts_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    outer, k = _stack(case)
    codes = torch.empty((outer, k // 2), dtype=torch.uint8, device="cuda")
    nv4 = case["format"] == "nvfp4"
    block = 16 if nv4 else 32
    scales = torch.empty((outer, k // block), dtype=torch.uint8, device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    amax = torch.full((), 0.11, device="cuda")
    step = max(1, 100_000_000 // k)
    for r in range(0, outer, step):
        rows = min(step, outer - r)
        w = (0.02 * torch.randn((rows, k // block, block), device="cuda", generator=g)).clamp_(-0.11, 0.11)
        top = w.abs().amax(2)
        if nv4:
            s8 = (top * (448.0 / amax)).to(torch.float8_e4m3fn)
            s, scales[r:r + rows] = s8.float() * (amax / 2688.0), s8.view(torch.uint8)
        else:
            e = torch.ceil(torch.log2(top / 6.0)).clamp(-127, 127)
            s, scales[r:r + rows] = torch.exp2(e), (e + 127).to(torch.uint8)
        w /= s[..., None].clamp(min=1e-30)
        c = torch.bucketize(w.abs(), mids, out_int32=True).to(torch.uint8)
        c |= (w < 0).to(torch.uint8) << 3
        c = c.view(rows, k // 2, 2)
        codes[r:r + rows] = c[..., 0] | (c[..., 1] << 4)
    offsets, _, place, longest = _groups(case)
    return {"codes": codes, "scales": scales, "meta": torch.stack([amax, amax / 2688.0]), "offsets": offsets,
            "place": place, "longest": longest,
            "x": _tokens(g, case["tokens"] + case["rest"], case["k"], _DT[case["dtype"]])}


def _wgrad_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    offsets, _, place, longest = _groups(case)
    rows = case["tokens"] + case["rest"]
    return {"offsets": offsets, "place": place, "longest": longest,
            "x": _tokens(g, rows, case["k"], _DT[case["dtype"]]),
            "dy": _gradients(g, rows, case["n"], _DT[case["dtype"]])}


def _adapters_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    offsets, group, place, longest = _groups(case)
    dt, wdt = _DT[case["dtype"]], _DT[case["wdtype"]]
    rows, n, k, r, count = case["tokens"] + case["rest"], case["n"], case["k"], case["rank"], case["adapters"]
    index = torch.randint(0, count, (case["segments"],), device="cuda", generator=g)
    if case["segments"] <= count:                # requests of different users
        index = torch.randperm(count, device="cuda", generator=g)[:case["segments"]]
    index[torch.rand(case["segments"], device="cuda", generator=g) < 0.05] = -1       # and some without an adapter
    if case["segments"] == 1:
        index[0] = index[0].clamp(min=0)
    state = {"offsets": offsets, "place": place, "longest": longest, "group": group, "index": index.to(torch.int32),
             "x": _tokens(g, rows, k, dt),
             "a": (torch.randn((count, r, k), device="cuda", generator=g) / math.sqrt(k)).to(wdt),
             "b": (0.05 * torch.randn((count, n, r), device="cuda", generator=g)).to(wdt),
             "scale": 0.5 + 1.5 * torch.rand(count, device="cuda", generator=g), "base": None}
    if case["op"] == "adapters":
        if case["base"]:
            state["base"] = torch.randn((rows, n), device="cuda", generator=g).to(dt)
        return state
    if case["base"]:
        state["base"] = _gradients(g, rows, k, dt)
    state["dy"] = _gradients(g, rows, n, dt)
    # the forward pass' low-rank activations, zero where there is no adapter
    s = dict(state, case=case)
    state["u"] = _low_rank(s, s["x"], _of_segments(s, "a", torch.float32), torch.float32)
    return state


def prepare(case, seed):
    make = {"rms": _rms_inputs, "rms_bwd": _rms_inputs, "experts": _experts_inputs, "wgrad": _wgrad_inputs,
            "adapters": _adapters_inputs, "adapters_bwd": _adapters_inputs}[case["op"]]
    state = make(case, seed)
    state["case"] = case
    return state


# ------------------------------------------------------------- plain forms --

def _mxfp8(y):
    """MXFP8 of the rows of y: E4M3 values and E8M0 scales of 32 each."""
    blocks = y.view(y.shape[0], -1, 32)
    m, e = torch.frexp(blocks.abs().amax(2))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)         # 448 = 0.875 * 2^9
    e = torch.where(m > 0, e, -127)
    codes = torch.ldexp(blocks, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(y.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_rms(s):
    c = s["case"]
    h = s["x"]
    if c["residual"] != "none":
        h = (h.float() + s["residual"].float()).to(s["residual"].dtype)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + EPS)
    y = hf * rstd[:, None] * s["weight"].float()
    out = _mxfp8(y) if c["out"] == "mxfp8" else (y.to(_DT[c["out"]]),)
    return (*out, rstd, h) if c["residual"] != "none" else (*out, rstd)


def _plain_rms_bwd(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * r
    a = dy * s["weight"].float()
    dx = r * (a - n * (a * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["x"].dtype), (dy * n).sum(0)


def _padded(s, rows, groups):
    """The groups' rows as a float32 batch [groups, longest, columns]."""
    flat = torch.zeros((groups * s["longest"], rows.shape[1]), dtype=torch.float32, device="cuda")
    flat[s["place"]] = rows[:s["place"].shape[0]].float()
    return flat.view(groups, s["longest"], -1)


def _decode(s, dtype):
    """The 4-bit weights as [experts, n, k] of `dtype`."""
    c = s["case"]
    lut = torch.tensor(_E2M1 + tuple(-q for q in _E2M1), dtype=dtype, device="cuda")
    codes = s["codes"]
    q = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], dim=2)
    if c["format"] == "nvfp4":
        scale = s["scales"].view(torch.float8_e4m3fn).to(dtype) * s["meta"][1].to(dtype)
    else:
        scale = torch.exp2(s["scales"].to(dtype) - 127)
    q = q.view(codes.shape[0], scale.shape[1], -1)
    q *= scale[..., None]
    if c["transposed"]:
        return q.view(c["n"], c["experts"], c["k"]).transpose(0, 1)
    return q.view(c["experts"], c["n"], c["k"])


def _plain_experts(s):
    c = s["case"]
    y = torch.bmm(_padded(s, s["x"], c["experts"]), _decode(s, torch.float32).transpose(1, 2).contiguous())
    out = torch.zeros((c["tokens"] + c["rest"], c["n"]), dtype=_DT[c["out"]], device="cuda")
    out[:c["tokens"]] = y.view(-1, c["n"])[s["place"]].to(out.dtype)
    return out


def _plain_wgrad(s):
    c = s["case"]
    dy, x = _padded(s, s["dy"], c["experts"]), _padded(s, s["x"], c["experts"])
    return torch.bmm(dy.transpose(1, 2), x).to(_DT[c["out"]])


def _of_segments(s, name, dtype):
    """Each segment's own adapter, zeros where it has none."""
    at = s["index"].long()
    return s[name][at.clamp(min=0)].to(dtype) * (at >= 0).to(dtype)[:, None, None]


def _unpadded(s, batch, rows):
    out = torch.zeros((rows, batch.shape[2]), dtype=batch.dtype, device="cuda")
    out[:s["place"].shape[0]] = batch.reshape(-1, batch.shape[2])[s["place"]]
    return out


def _low_rank(s, x, a, dtype):
    """u = A x of every row (zeros in the rest)."""
    groups = s["case"]["segments"]
    u = torch.bmm(_padded(s, x, groups).to(dtype), a.transpose(1, 2).contiguous())
    return _unpadded(s, u, x.shape[0])


def _plain_adapters(s):
    c = s["case"]
    groups = c["segments"]
    u = _low_rank(s, s["x"], _of_segments(s, "a", torch.float32), torch.float32)
    b = _of_segments(s, "b", torch.float32) * s["scale"][s["index"].long().clamp(min=0)][:, None, None]
    y = _unpadded(s, torch.bmm(_padded(s, u, groups), b.transpose(1, 2).contiguous()), s["x"].shape[0])
    if s["base"] is not None:
        y += s["base"].float()
    return y.to(_DT[c["dtype"]]), u


def _plain_adapters_bwd(s):
    c = s["case"]
    groups = c["segments"]
    at = s["index"].long()
    used = (at >= 0).float()[:, None, None]
    scale = s["scale"][at.clamp(min=0)][:, None, None]
    a, b = _of_segments(s, "a", torch.float32), _of_segments(s, "b", torch.float32)
    x, dy, u = _padded(s, s["x"], groups), _padded(s, s["dy"], groups), _padded(s, s["u"], groups)
    g = torch.bmm(dy, b) * scale
    dx = _unpadded(s, torch.bmm(g, a), s["x"].shape[0])
    if s["base"] is not None:
        dx += s["base"].float()
    da = torch.zeros(s["a"].shape, dtype=torch.float32, device="cuda")
    db = torch.zeros(s["b"].shape, dtype=torch.float32, device="cuda")
    da.index_add_(0, at.clamp(min=0), torch.bmm(g.transpose(1, 2).contiguous(), x) * used)
    db.index_add_(0, at.clamp(min=0), torch.bmm(dy.transpose(1, 2).contiguous(), u) * (scale * used))
    return dx.to(_DT[c["dtype"]]), da, db


# ---------------------------------------------------------------- one pass --

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rms": _plain_rms, "rms_bwd": _plain_rms_bwd, "experts": _plain_experts, "wgrad": _plain_wgrad,
                "adapters": _plain_adapters, "adapters_bwd": _plain_adapters_bwd}[c["op"]](s)
    import gemm_amax_reduce_amd as nv
    if c["op"] == "rms":
        residual = s.get("residual")
        if c["out"] != "mxfp8":
            return nv.nvfp4_rms_norm(s["x"], s["weight"], residual, eps=EPS, out_dtype=_DT[c["out"]])
        q, *rest = nv.mxfp8_rms_norm(s["x"], s["weight"], residual, eps=EPS)
        return (q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu), *rest)
    if c["op"] == "rms_bwd":
        return nv.nvfp4_rms_norm_backward(s["dy"], s["x"], s["rstd"], s["weight"], dh=s["dh"])
    if c["op"] == "experts":
        outer, k = _stack(c)
        if c["format"] == "nvfp4":
            w, product = nv.NVFP4Tensor(s["codes"], s["scales"], s["meta"], outer, k), nv.nvfp4_grouped_matmul
        else:
            w, product = nv.MXFP4Tensor(s["codes"], s["scales"], outer, k), nv.mxfp4_grouped_matmul
        return product(w, s["x"], s["offsets"], out_dtype=_DT[c["out"]], transposed=c["transposed"])
    if c["op"] == "wgrad":
        return nv.nvfp4_grouped_wgrad(s["dy"], s["x"], s["offsets"], grad_dtype=_DT[c["out"]])
    if c["op"] == "adapters":
        return nv.nvfp4_adapters(s["x"], s["a"], s["b"], s["offsets"], s["index"], s["scale"], base=s["base"],
                                 out_dtype=_DT[c["dtype"]])
    return nv.nvfp4_adapters_backward(s["dy"], s["x"], s["u"], s["a"], s["b"], s["offsets"], s["index"], s["scale"],
                                      base=s["base"])


def work(case):
    """What a pass cannot do without: each input read once, each output
    written once, and the operations of the formulas."""
    c = case
    if c["op"] in ("rms", "rms_bwd"):
        n, s, ws = c["rows"] * c["cols"], _SIZE[c["dtype"]], _SIZE[c["wdtype"]]
        if c["op"] == "rms":
            h = 0 if c["residual"] == "none" else 2 * n * _SIZE[c["residual"]]
            y = n + n // 32 if c["out"] == "mxfp8" else n * _SIZE[c["out"]]
            return {"bytes": n * s + h + y + c["cols"] * ws + 4 * c["rows"], "flops": 5 * n}
        return {"bytes": (4 if c["dh"] else 3) * n * s + c["cols"] * (ws + 4) + 4 * c["rows"], "flops": 10 * n}
    if c["op"] in ("experts", "wgrad"):
        sizes = _group_sizes(c)
        active, s, out = sum(z > 0 for z in sizes), _SIZE[c["dtype"]], _SIZE[c["out"]]
        m, n, k = c["tokens"], c["n"], c["k"]
        if c["op"] == "wgrad":
            return {"bytes": m * (n + k) * s + c["experts"] * n * k * out, "flops": 2 * m * n * k}
        group = 16 if c["format"] == "nvfp4" else 32
        return {"bytes": active * n * (k // 2 + k // group) + m * k * s + (m + c["rest"]) * n * out,
                "flops": 2 * m * n * k}
    m, n, k, r = c["tokens"], c["n"], c["k"], c["rank"]
    s, w = _SIZE[c["dtype"]], min(c["segments"], c["adapters"]) * r * (n + k) * _SIZE[c["wdtype"]]
    if c["op"] == "adapters":
        return {"bytes": m * (k + (2 if c["base"] else 1) * n) * s + w + 4 * m * r, "flops": 2 * m * r * (n + k)}
    return {"bytes": m * (n + (3 if c["base"] else 2) * k) * s + w + 4 * m * r + 4 * c["adapters"] * r * (n + k),
            "flops": 4 * m * r * (n + k)}


# ------------------------------------------------------ the 64-bit results --

def exact(case, seed):
    s = prepare(case, seed)
    return {"rms": _exact_rms, "rms_bwd": _exact_rms_bwd, "experts": _exact_experts, "wgrad": _exact_wgrad,
            "adapters": _exact_adapters, "adapters_bwd": _exact_adapters_bwd}[case["op"]](case, s)


def _exact_rms(c, s):
    h = x = s["x"].double()
    if c["residual"] != "none":
        x = x + s["residual"].double()
        h = x.to(_DT[c["residual"]]).double()          # what is normed is the stream as it is stored
    rstd = 1.0 / torch.sqrt(torch.square(h).sum(1) / c["cols"] + EPS)
    y = s["weight"].double() * h * rstd[:, None]
    out = [y]
    if c["out"] == "mxfp8":
        b = y.view(c["rows"], -1, 32)
        top = b.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(-127, 127)
        e += (top > 448.0 * torch.pow(2.0, e)).double()          # the logarithm rounds next to a power of two
        e -= (top <= 448.0 * torch.pow(2.0, e - 1)).double()
        e = e.clamp(-127, 127)
        v = b * torch.pow(2.0, -e)
        ulp = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out = [(torch.round(v / ulp) * ulp).view(y.shape), torch.pow(2.0, e)[..., 0]]
    return (*out, rstd, x) if c["residual"] != "none" else (*out, rstd)


def _exact_rms_bwd(c, s):
    r = s["rstd"].double()[:, None]
    n = s["x"].double().mul_(r)
    a = s["dy"].double()
    dw = (a * n).sum(0)
    a *= s["weight"].double()
    dot = (a * n).sum(1, keepdim=True) / c["cols"]
    dx = a.sub_(n.mul_(dot)).mul_(r)
    if s["dh"] is not None:
        dx += s["dh"].double()
    return dx, dw


def _ranges(s):
    ends = s["offsets"].tolist()
    return list(zip(ends[:-1], ends[1:]))


def _exact_experts(c, s):
    out = torch.zeros((c["tokens"] + c["rest"], c["n"]), dtype=torch.float64, device="cuda")
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    nv4 = c["format"] == "nvfp4"
    block = 16 if nv4 else 32
    n, k = c["n"], c["k"]
    for e, (begin, end) in enumerate(_ranges(s)):
        if begin == end:
            continue
        if c["transposed"]:
            codes = s["codes"][:, e * (k // 2):(e + 1) * (k // 2)]
            scales = s["scales"][:, e * (k // block):(e + 1) * (k // block)]
        else:
            codes, scales = s["codes"][e * n:(e + 1) * n], s["scales"][e * n:(e + 1) * n]
        w = torch.empty((n, k), dtype=torch.float64, device="cuda")
        for half, nib in ((0, codes & 15), (1, codes >> 4)):
            w[:, half::2] = grid[(nib & 7).long()] * (1 - 2 * (nib >> 3).double())
        if nv4:
            w *= scales.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
            w *= s["meta"][1].double()
        else:
            w *= torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)
        out[begin:end] = s["x"][begin:end].double() @ w.t()
    return out


def _exact_wgrad(c, s):
    out = torch.zeros((c["experts"], c["n"], c["k"]), dtype=torch.float64, device="cuda")
    for e, (begin, end) in enumerate(_ranges(s)):
        out[e] = s["dy"][begin:end].double().t() @ s["x"][begin:end].double()
    return out


def _exact_adapters(c, s):
    y = torch.zeros((s["x"].shape[0], c["n"]), dtype=torch.float64, device="cuda")
    u = torch.zeros((s["x"].shape[0], c["rank"]), dtype=torch.float64, device="cuda")
    if s["base"] is not None:
        y += s["base"].double()
    for (begin, end), i in zip(_ranges(s), s["index"].tolist()):
        if i >= 0:
            u[begin:end] = s["x"][begin:end].double() @ s["a"][i].double().t()
            y[begin:end] += s["scale"][i].double() * (u[begin:end] @ s["b"][i].double().t())
    return y, u


def _exact_adapters_bwd(c, s):
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    if s["base"] is not None:
        dx += s["base"].double()
    for (begin, end), i in zip(_ranges(s), s["index"].tolist()):
        if i >= 0:
            dy = s["scale"][i].double() * s["dy"][begin:end].double()
            g = dy @ s["b"][i].double()
            dx[begin:end] += g @ s["a"][i].double()
            da[i] += g.t() @ s["x"][begin:end].double()
            db[i] += dy.t() @ s["u"][begin:end].double()
    return dx, da, db
