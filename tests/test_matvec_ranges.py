"""How the matrix-vector products cut K: the size query returns for every K,
also where K leaves half a lane's load (16) behind a whole number of slices,
and the products at such K are right.

A workgroup holds at most `most` slices of 512 (one slab of 16 columns) or
256 k (two or three slabs, float32 x of 6 tokens and more).  Where
K - 16 is a multiple of the slice and of every number of slices up to `most`,
no cut into equal ranges leaves more than 16 k for the last one.
"""
import json
import math
import subprocess
import sys

import pytest

import gemm_amax_reduce_amd as nv

MOST_K = (1 << 25) - 16
# tokens, dtype, k of a slice, slices of a workgroup at most
CUTS = [(16, nv.F32, 256, 8), (8, nv.F32, 256, 11), (5, nv.F32, 512, 11), (16, nv.BF16, 512, 11), (2, nv.BF16, 512, 11)]


def _hard(slice_k, most):
    """Every K <= MOST_K of the kind that no equal cut serves."""
    step = slice_k * math.lcm(*range(1, most + 1))
    return list(range(step + 16, MOST_K + 1, step))


def test_there_are_such_k():
    assert len(_hard(256, 8)) == 156 and len(_hard(256, 11)) == 4 and len(_hard(512, 11)) == 2


def test_size_query_returns():
    asked = [(16, k, tokens, dt) for tokens, dt, slice_k, most in CUTS for k in _hard(slice_k, most)]
    # in a process of its own, so that one that does not return ends
    code = ("import ctypes, json, sys\n"
            "f = ctypes.CDLL(sys.argv[1]).nvfp4_matvec_workspace_bytes\n"
            "f.argtypes, f.restype = [ctypes.c_int64] * 3 + [ctypes.c_int], ctypes.c_int64\n"
            "print(json.dumps([f(*a) for a in json.loads(sys.stdin.read())]))\n")
    done = subprocess.run([sys.executable, "-c", code, nv.LIB_PATH], input=json.dumps(asked), capture_output=True,
                          text=True, timeout=60, check=True)
    most_of = {(tokens, dt): slice_k * most for tokens, dt, slice_k, most in CUTS}
    for (n, k, tokens, dt), size in zip(asked, json.loads(done.stdout)):
        # [ranges][tokens][n] binary32 sums, with no more ranges than K needs
        assert size == 4 * tokens * n * -(-k // most_of[tokens, dt])


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,dt,k", [(16, "f32", 215056), (11, "f32", 430096), (16, "f32", 860176),
                                         (8, "f32", 7096336), (2, "bf16", 14192656), (16, "bf16", 14192656)])
def test_product_of_such_k(tokens, dt, k):
    """Every product is exact in binary32; with sums over K / (waves and lanes)
    added up in order and joined, 1e-5 of the sum of magnitudes as for any K.
    The last 48 k carry large activations, so that one left out, or taken
    twice, shows."""
    import torch
    n = 19
    g = torch.Generator(device="cuda").manual_seed(k % 1000 + tokens)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(0x28, 0x48, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
    meta = torch.tensor([2.0, 2.0 / 2688], device="cuda")
    x = torch.randn((tokens, k), device="cuda", generator=g)
    x[:, -48:] *= 1000.0
    x = x.to(torch.bfloat16 if dt == "bf16" else torch.float32)
    print(f"[matvec] {tokens}x{n}x{k} {dt}", flush=True)
    y = nv.nvfp4_matvec(nv.NVFP4Tensor(codes, scales, meta, n, k), x, out_dtype=torch.float32)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device="cuda")
    xd = x.double()
    for r in range(n):
        w = torch.stack([grid[(codes[r] & 15).int()], grid[(codes[r] >> 4).int()]], 1).flatten()
        w *= scales[r].view(torch.float8_e4m3fn).double().repeat_interleave(16) * meta[1].double()
        want, mass = xd @ w, xd.abs() @ w.abs()
        assert torch.all((y[:, r].double() - want).abs() <= 1e-5 * mass), r
        # the tail alone: within the same bound of it, its share of the sum is found
        assert torch.all(mass * 1e-5 < (xd[:, -16:].abs() @ w[-16:].abs()))
