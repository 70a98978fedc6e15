"""RMS norm, grouped products and low-rank adapters refuse invalid arguments
before anything is launched: the C ABI by status code (where no GPU is visible,
since the pointers are made up), the binding and the modules by NVFP4Error."""
import ctypes
import math

import pytest
import torch

import gemm_amax_reduce_amd as nv
from gemm_amax_reduce_amd.adapters import LowRankAdapters
from gemm_amax_reduce_amd.experts import NVFP4ExpertBlock, NVFP4Experts
from gemm_amax_reduce_amd.head import NVFP4Head, RMSNorm

FAKE = 1 << 20
_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer argument tests run only without a GPU")
NULL, SHAPE, ENUM, HIP, ALIGN, VALUE = -1, -2, -3, -4, -5, -6
LIMIT = (1 << 24) - 8                    # workgroups of a grid


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def _call(fn, good, **bad):
    """fn with the arguments of `good` (name -> value, in order), some replaced."""
    assert set(bad) <= set(good)
    return fn(*{**good, **bad}.values())


# ------------------------------------------------------------------ RMS norm

RMS = dict(x=FAKE, xd=1, rows=4, cols=64, ldx=64, res=2 * FAKE, rd=0, ldr=64, h=3 * FAKE, ldh=64, w=FAKE, wd=1, eps=1e-6,
           y=4 * FAKE, yd=1, ldy=64, rstd=5 * FAKE, stream=None)
RMS_SHARED = [(dict(xd=2), ENUM), (dict(wd=9), ENUM), (dict(rd=5), ENUM), (dict(cols=0), SHAPE), (dict(rows=-1), SHAPE),
              (dict(ldx=63), SHAPE), (dict(ldr=63), SHAPE), (dict(ldh=63), SHAPE), (dict(rows=1 << 40, ldx=1 << 30), SHAPE),
              (dict(eps=-1e-9), VALUE), (dict(eps=math.nan), VALUE), (dict(eps=math.inf), VALUE), (dict(x=None), NULL),
              (dict(h=None), NULL), (dict(rstd=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(res=2 * FAKE + 2), ALIGN),
              (dict(h=3 * FAKE + 2), ALIGN), (dict(w=FAKE + 1), ALIGN), (dict(rstd=FAKE + 2), ALIGN),
              (dict(h=FAKE), SHAPE),                                     # h where x is
              (dict(h=2 * FAKE + 4), SHAPE),                             # h one element into the residual
              (dict(h=2 * FAKE, ldh=65), SHAPE)]                         # in its place, at another pitch


@_no_gpu
@pytest.mark.parametrize("bad,status", RMS_SHARED + [
    (dict(yd=-1), ENUM), (dict(ldy=63), SHAPE), (dict(y=None), NULL), (dict(y=FAKE + 1), ALIGN), (dict(y=FAKE), SHAPE),
    (dict(y=2 * FAKE), SHAPE), (dict(y=3 * FAKE + 4 * 255), SHAPE), (dict(y=3 * FAKE + 4 * 256), HIP),
    (dict(h=2 * FAKE), HIP), (dict(rows=0, x=None, y=None, h=None, rstd=None), 0), (dict(res=None, rd=7), HIP)])
def test_rms_norm(L, bad, status):
    assert _call(L.nvfp4_rms_norm, RMS, **bad) == status


def _mx8(**bad):
    t = {**dict(codes=4 * FAKE, scales=5 * FAKE, outer=4, k=64), **bad}
    return nv._MXTensor(*t.values())


@_no_gpu
@pytest.mark.parametrize("bad,status", RMS_SHARED)
def test_rms_norm_mx8(L, bad, status):
    args = {k: v for k, v in {**RMS, **bad}.items() if k not in ("y", "yd", "ldy", "rstd", "stream")}
    rstd = bad.get("rstd", 6 * FAKE)
    assert L.mxfp8_rms_norm(*args.values(), ctypes.byref(_mx8()), rstd, None) == status


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(outer=5), SHAPE), (dict(k=32), SHAPE), (dict(codes=0), NULL), (dict(scales=0), NULL), (dict(codes=FAKE + 4), ALIGN),
    (dict(codes=FAKE), SHAPE), (dict(scales=3 * FAKE + 8), SHAPE), (dict(), HIP)])
def test_rms_norm_mx8_output(L, bad, status):
    args = [v for k, v in RMS.items() if k not in ("y", "yd", "ldy", "rstd", "stream")]
    assert L.mxfp8_rms_norm(*args, ctypes.byref(_mx8(**bad)), 6 * FAKE, None) == status
    assert L.mxfp8_rms_norm(*args, None, 6 * FAKE, None) == NULL
    odd = [v for k, v in {**RMS, "cols": 48}.items() if k not in ("y", "yd", "ldy", "rstd", "stream")]
    assert L.mxfp8_rms_norm(*odd, ctypes.byref(_mx8(k=48)), 6 * FAKE, None) == SHAPE


RMS_BACK = dict(dy=FAKE, dyd=1, lddy=64, h=2 * FAKE, hd=1, rows=4, cols=64, ldh=64, rstd=FAKE, w=FAKE, wd=1,
                dh=3 * FAKE, lddh=64, dx=4 * FAKE, lddx=64, dw=5 * FAKE, gd=0, ws=FAKE, bytes=1 << 30, stream=None)


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(dyd=3), ENUM), (dict(hd=3), ENUM), (dict(wd=3), ENUM), (dict(gd=3), ENUM), (dict(cols=0), SHAPE),
    (dict(rows=-1), SHAPE), (dict(lddy=1), SHAPE), (dict(ldh=1), SHAPE), (dict(lddh=1), SHAPE), (dict(lddx=1), SHAPE),
    (dict(rows=1000, bytes=0), SHAPE), (dict(rows=1000, ws=None), NULL), (dict(dy=None), NULL), (dict(h=None), NULL),
    (dict(rstd=None), NULL), (dict(dx=None), NULL), (dict(ws=FAKE + 8), ALIGN), (dict(dw=FAKE + 2), ALIGN),
    (dict(dx=FAKE + 1), ALIGN), (dict(dh=FAKE + 1), ALIGN), (dict(dx=FAKE), SHAPE), (dict(dx=2 * FAKE + 2), SHAPE),
    (dict(dx=3 * FAKE), SHAPE), (dict(), HIP), (dict(dh=None, lddh=0), HIP)])
def test_rms_norm_backward(L, bad, status):
    assert _call(L.nvfp4_rms_norm_backward, RMS_BACK, **bad) == status


@_no_gpu
def test_rms_norm_backward_workspace(L):
    size = L.nvfp4_rms_norm_backward_workspace_bytes
    assert size(-1, 64) == SHAPE and size(4, 0) == SHAPE and size(0, 64) >= 0
    need = size(1000, 64)
    assert need > 0
    assert _call(L.nvfp4_rms_norm_backward, RMS_BACK, rows=1000, bytes=need - 1) == SHAPE


# ---------------------------------------------------------- grouped products

GROUPED = dict(transposed=0, x=FAKE, xd=1, rows=40, ldx=64, off=FAKE, bits=64, experts=4, y=2 * FAKE, yd=1, ldy=16, zero=0,
               ws=FAKE, bytes=1 << 30, stream=None)
GROUPED_BAD = [
    (dict(xd=2), ENUM), (dict(yd=2), ENUM), (dict(bits=16), ENUM), (dict(experts=0), SHAPE), (dict(experts=-1), SHAPE),
    (dict(experts=3), SHAPE), (dict(experts=(1 << 20) + 1), SHAPE), (dict(rows=-1), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldy=15), SHAPE), (dict(rows=32 * LIMIT), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(off=None), NULL),
    (dict(x=FAKE + 1), ALIGN), (dict(yd=0, y=2 * FAKE + 2), ALIGN), (dict(off=FAKE + 4), ALIGN), (dict(ws=FAKE + 8), ALIGN),
    (dict(y=FAKE), SHAPE), (dict(y=FAKE + 2 * (39 * 64 + 63), ldy=64), SHAPE), (dict(), HIP), (dict(rows=0, x=None, y=None), 0)]


@_no_gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("bad,status", GROUPED_BAD)
def test_grouped_matmul(L, mx, bad, status):
    w = nv._MXTensor(FAKE, FAKE, 64, 64) if mx else nv._CTensor(FAKE, FAKE, FAKE, 64, 64)
    fn = L.mxfp4_grouped_matmul if mx else L.nvfp4_grouped_matmul
    assert fn(ctypes.byref(w), *{**GROUPED, **bad}.values()) == status


@_no_gpu
def test_grouped_matmul_weights(L):
    by, args = ctypes.byref, list(GROUPED.values())
    turned = list({**GROUPED, "transposed": 1, "ldx": 64, "ldy": 64}.values())
    assert L.nvfp4_grouped_matmul(None, *args) == NULL
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE, FAKE, 0, 64, 64)), *args) == NULL
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE, FAKE, FAKE, 64, 40)), *args) == SHAPE
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE + 4, FAKE, FAKE, 64, 64)), *args) == ALIGN
    # a transposed stack: the experts' columns are whole blocks
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE, FAKE, FAKE, 64, 4 * 48)), *turned) == HIP
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE, FAKE, FAKE, 64, 4 * 16 + 16)), *turned) == SHAPE
    assert L.mxfp4_grouped_matmul(None, *args) == NULL
    assert L.mxfp4_grouped_matmul(by(nv._MXTensor(FAKE, 0, 64, 64)), *args) == NULL
    assert L.mxfp4_grouped_matmul(by(nv._MXTensor(FAKE, FAKE, 64, 4 * 16)), *turned) == SHAPE
    long = {**GROUPED, "transposed": 1, "experts": 16, "ldx": 1 << 24}
    assert L.nvfp4_grouped_matmul(by(nv._CTensor(FAKE, FAKE, FAKE, 16, 16 << 24)), *long.values()) == SHAPE


@_no_gpu
def test_grouped_matmul_workspace(L):
    size = L.nvfp4_grouped_matmul_workspace_bytes
    assert size(4, 16, 64, 40, 7) == ENUM
    for bad in ((0, 16, 64, 40), (4, -1, 64, 40), (4, 16, 40, 40), (4, 16, 64, -1), (4, 16, 1 << 25, 40),
                (4, 16, 64, 32 * LIMIT)):
        assert size(*bad, 1) == SHAPE, bad
    assert size(4, 0, 64, 40, 1) >= 0 and size(4, 16, 0, 40, 1) >= 0 and size(4, 16, 64, 0, 1) >= 0
    need = size(4, 16, 64, 4000, 0)                     # many float32 rows: their parts
    assert need > 0
    by = ctypes.byref(nv._CTensor(FAKE, FAKE, FAKE, 64, 64))
    f32 = {**GROUPED, "xd": 0, "rows": 4000, "y": 4 * FAKE}
    assert L.nvfp4_grouped_matmul(by, *{**f32, "bytes": need - 1}.values()) == SHAPE
    assert L.nvfp4_grouped_matmul(by, *{**f32, "bytes": need, "ws": None}.values()) == NULL


WGRAD = dict(dy=FAKE, dyd=1, lddy=48, x=2 * FAKE, xd=1, ldx=64, rows=40, n=48, k=64, off=FAKE, bits=32, experts=4,
             dw=3 * FAKE, dwd=0, ws=FAKE, bytes=1 << 30, stream=None)


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(dyd=2), ENUM), (dict(xd=2), ENUM), (dict(dwd=2), ENUM), (dict(bits=8), ENUM), (dict(lddy=47), SHAPE),
    (dict(ldx=63), SHAPE), (dict(rows=-1), SHAPE), (dict(n=-1), SHAPE), (dict(k=-1), SHAPE), (dict(experts=0), SHAPE),
    (dict(experts=(1 << 20) + 1), SHAPE),
    (dict(n=1 << 25, lddy=1 << 25), SHAPE), (dict(k=1 << 25, ldx=1 << 25), SHAPE), (dict(experts=1 << 20, n=1 << 12, lddy=1 << 12), SHAPE), (dict(dy=None), NULL),
    (dict(x=None), NULL), (dict(dw=None), NULL), (dict(off=None), NULL), (dict(dy=FAKE + 1), ALIGN),
    (dict(dw=3 * FAKE + 2), ALIGN), (dict(off=FAKE + 2), ALIGN), (dict(ws=FAKE + 8), ALIGN), (dict(dw=FAKE), SHAPE),
    (dict(dw=2 * FAKE - 4), SHAPE), (dict(dyd=0, lddy=48, bytes=0), SHAPE), (dict(dyd=0, ws=None), NULL), (dict(), HIP),
    (dict(rows=0, dy=None, x=None), HIP), (dict(n=0, dw=None), 0)])
def test_grouped_wgrad(L, bad, status):
    assert _call(L.nvfp4_grouped_wgrad, WGRAD, **bad) == status


@_no_gpu
def test_grouped_wgrad_workspace(L):
    size = L.nvfp4_grouped_wgrad_workspace_bytes
    assert size(4, 48, 64, 40, 2, 1) == ENUM and size(4, 48, 64, 40, 1, 2) == ENUM
    for bad in ((0, 48, 64, 40), (4, -1, 64, 40), (4, 48, -1, 40), (4, 48, 64, -1)):
        assert size(*bad, 1, 1) == SHAPE
    need = size(4, 48, 64, 40, 0, 1)
    assert need > 0
    assert _call(L.nvfp4_grouped_wgrad, WGRAD, dyd=0, bytes=need - 1) == SHAPE


# ------------------------------------------------------------------ adapters

SET = dict(a=FAKE, b=2 * FAKE, wd=1, adapters=3, rank=8, n=48, scale=FAKE, off=FAKE, index=FAKE, bits=64, segments=2)
ADAPT = dict(x=3 * FAKE, xd=1, rows=10, k=64, ldx=64, **SET, base=4 * FAKE, bd=1, ldb=48, y=5 * FAKE, yd=1, ldy=48,
             u=6 * FAKE, stream=None)
ADAPT_BACK = dict(dy=3 * FAKE, dyd=1, lddy=48, x=4 * FAKE, xd=1, rows=10, k=64, ldx=64, u=5 * FAKE, **SET, base=6 * FAKE,
                  bd=1, ldb=64, dx=7 * FAKE, dxd=1, lddx=64, da=8 * FAKE, db=9 * FAKE, gd=0, ws=FAKE, bytes=1 << 30,
                  stream=None)
SET_BAD = [
    (dict(wd=2), ENUM), (dict(bits=16), ENUM), (dict(xd=2), ENUM), (dict(bd=2), ENUM), (dict(rank=0), SHAPE),
    (dict(rank=129), SHAPE), (dict(adapters=0), SHAPE), (dict(adapters=65536), SHAPE), (dict(n=-1), SHAPE), (dict(k=-1), SHAPE),
    (dict(rows=-1), SHAPE), (dict(segments=0), SHAPE), (dict(segments=(1 << 20) + 1), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldb=40), SHAPE), (dict(rows=16 * LIMIT), SHAPE), (dict(x=None), NULL), (dict(a=None), NULL), (dict(b=None), NULL),
    (dict(off=None), NULL), (dict(index=None), NULL), (dict(u=None), NULL), (dict(a=FAKE + 1), ALIGN),
    (dict(wd=0, b=2 * FAKE + 2), ALIGN), (dict(scale=FAKE + 2), ALIGN), (dict(off=FAKE + 4), ALIGN),
    (dict(index=FAKE + 4), ALIGN), (dict(x=3 * FAKE + 1), ALIGN), (dict(u=6 * FAKE + 2), ALIGN), (dict(), HIP),
    (dict(base=None, bd=9, ldb=0), HIP), (dict(scale=None), HIP)]


@_no_gpu
@pytest.mark.parametrize("bad,status", SET_BAD)
def test_adapters_shared(L, bad, status):
    assert _call(L.nvfp4_adapters, ADAPT, **bad) == status
    assert _call(L.nvfp4_adapters_backward, ADAPT_BACK, **bad) == status


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(yd=2), ENUM), (dict(ldy=47), SHAPE), (dict(y=None), NULL), (dict(y=5 * FAKE + 1), ALIGN), (dict(y=3 * FAKE), SHAPE),
    (dict(y=4 * FAKE), HIP), (dict(y=4 * FAKE, ldy=50), SHAPE), (dict(y=4 * FAKE, yd=0), SHAPE), (dict(y=4 * FAKE + 2), SHAPE),
    (dict(u=3 * FAKE), SHAPE), (dict(u=4 * FAKE), SHAPE), (dict(u=5 * FAKE), SHAPE),
    (dict(rows=0, x=None, y=None, u=None, off=None, index=None), 0)])
def test_adapters(L, bad, status):
    assert _call(L.nvfp4_adapters, ADAPT, **bad) == status


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(dyd=2), ENUM), (dict(dxd=2), ENUM), (dict(gd=2), ENUM), (dict(lddy=47), SHAPE), (dict(lddx=63), SHAPE),
    (dict(bytes=0), SHAPE), (dict(ws=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(da=None), NULL),
    (dict(db=None), NULL), (dict(ws=FAKE + 8), ALIGN), (dict(da=8 * FAKE + 2), ALIGN), (dict(dx=7 * FAKE + 1), ALIGN),
    (dict(dx=6 * FAKE), HIP), (dict(dx=6 * FAKE, lddx=66), SHAPE), (dict(dx=4 * FAKE), SHAPE), (dict(dx=3 * FAKE), SHAPE),
    (dict(da=9 * FAKE), SHAPE), (dict(da=4 * FAKE), SHAPE), (dict(db=5 * FAKE), SHAPE), (dict(db=7 * FAKE), SHAPE),
    (dict(da=FAKE), SHAPE), (dict(db=2 * FAKE), SHAPE)])
def test_adapters_backward(L, bad, status):
    assert _call(L.nvfp4_adapters_backward, ADAPT_BACK, **bad) == status


@_no_gpu
def test_adapters_backward_workspace(L):
    size = L.nvfp4_adapters_backward_workspace_bytes
    good = dict(rows=10, n=48, k=64, rank=8, adapters=3, segments=2, wd=1)
    assert _call(size, good, wd=2) == ENUM
    for bad in (dict(rows=-1), dict(n=-1), dict(k=-1), dict(rank=0), dict(rank=129), dict(adapters=0),
                dict(adapters=65536), dict(segments=0)):
        assert _call(size, good, **bad) == SHAPE, bad
    need = _call(size, good)
    assert need > 0
    assert _call(L.nvfp4_adapters_backward, ADAPT_BACK, bytes=need - 1) == SHAPE
    assert _call(L.nvfp4_adapters_backward, ADAPT_BACK, bytes=need) == HIP


# ----------------------------------------------- outputs that meet something

APART = {
    "rms": (RMS, dict(y="x res h w rstd", h="x w", rstd="x res h w y")),
    "rms_back": (dict(RMS_BACK, rstd=6 * FAKE, w=7 * FAKE, ws=8 * FAKE),
                 dict(dx="dy h dh rstd w dw", dw="dy h dh rstd w dx")),
    "adapters": (dict(ADAPT, scale=7 * FAKE, off=8 * FAKE, index=9 * FAKE),
                 dict(y="x a b scale off index u", u="x a b scale off index base y")),
    "adapters_back": (dict(ADAPT_BACK, scale=10 * FAKE, off=11 * FAKE, index=12 * FAKE, ws=13 * FAKE),
                      dict(dx="dy x u a b scale off index da db", da="dy x u a b scale off index base dx db",
                           db="dy x u a b scale off index base dx da")),
}
CALLS = {"rms": "nvfp4_rms_norm", "rms_back": "nvfp4_rms_norm_backward", "adapters": "nvfp4_adapters",
         "adapters_back": "nvfp4_adapters_backward"}


@_no_gpu
@pytest.mark.parametrize("which,out,other", [(which, out, other) for which, (_, pairs) in APART.items()
                                             for out, others in pairs.items() for other in others.split()])
def test_outputs_do_not_meet(L, which, out, other):
    """Each output at another argument's place, and 8 bytes in front of it; with
    all of them a megabyte apart the call gets as far as its launch."""
    good = APART[which][0]
    fn = getattr(L, CALLS[which])
    assert _call(fn, good) == HIP
    assert _call(fn, good, **{out: good[other]}) == SHAPE
    assert _call(fn, good, **{out: good[other] - 8}) == SHAPE


@_no_gpu
@pytest.mark.parametrize("other", ["x", "res", "h", "w", "rstd"])
@pytest.mark.parametrize("out", ["codes", "scales"])
def test_mx8_outputs_do_not_meet(L, out, other):
    good = {**RMS, "w": 8 * FAKE, "rstd": 6 * FAKE}
    args = [v for k, v in good.items() if k not in ("y", "yd", "ldy", "rstd", "stream")]
    call = lambda **t: L.mxfp8_rms_norm(*args, ctypes.byref(_mx8(**t)), good["rstd"], None)
    assert call() == HIP
    assert call(**{out: good[other]}) == SHAPE
    assert call(codes=4 * FAKE, scales=4 * FAKE + 255) == SHAPE and call(codes=4 * FAKE, scales=4 * FAKE + 256) == HIP
    assert call(codes=4 * FAKE, scales=4 * FAKE - 7) == SHAPE and call(codes=4 * FAKE, scales=4 * FAKE - 8) == HIP


@_no_gpu
@pytest.mark.parametrize("rows", [1, 2, 4])
@pytest.mark.parametrize("ld", [4, 9, 40])
def test_a_block_in_the_gaps_of_a_matrix(L, rows, ld):
    """u (a block of rows * rank * 4 bytes) at every place around dx [rows][ld]
    of 4 float32 columns: refused where elements meet, and there alone."""
    k, rank = 4, 3
    dx = {FAKE + 4 * (r * ld + c) for r in range(rows) for c in range(k)}
    good = dict(ADAPT_BACK, rows=rows, k=k, ldx=k, rank=rank, n=2, lddy=2, dyd=0, xd=0, base=None, dx=FAKE, dxd=0, lddx=ld,
                a=20 * FAKE, b=21 * FAKE, scale=None, off=22 * FAKE, index=23 * FAKE, ws=24 * FAKE)
    for shift in range(-4 * (rows * rank + 2), 4 * (rows * ld + 2), 4):
        u = {FAKE + shift + 4 * i for i in range(rows * rank)}
        assert _call(L.nvfp4_adapters_backward, good, u=FAKE + shift) == (SHAPE if u & dx else HIP), shift


@_no_gpu
@pytest.mark.parametrize("rows", [1, 3])
def test_matrices_side_by_side(L, rows):
    """y against h, and dx against dy, in one buffer: refused where elements
    meet (of two pitches, where the whole ranges do)."""
    cols = 5
    for ldh, ldy in ((5, 5), (12, 12), (12, 9)):
        at = lambda p, ld: {p + 4 * (r * ld + c) for r in range(rows) for c in range(cols)}
        for shift in range(-4 * 40, 4 * 40, 4):
            meets = bool(at(FAKE, ldh) & at(FAKE + shift, ldy))
            fwd = _call(L.nvfp4_rms_norm, RMS, rows=rows, cols=cols, ldx=cols, x=9 * FAKE, w=None, ldr=cols, h=FAKE, ldh=ldh,
                        y=FAKE + shift, yd=0, ldy=ldy)
            back = _call(L.nvfp4_rms_norm_backward, RMS_BACK, rows=rows, cols=cols, rstd=6 * FAKE, w=None, hd=0, ldh=cols,
                         dh=None, dy=FAKE, dyd=0, lddy=ldh, dx=FAKE + shift, lddx=ldy)
            for got in (fwd, back):
                if meets or ldh == ldy:
                    assert got == (SHAPE if meets else HIP), (ldh, ldy, shift)
                else:
                    assert got in (SHAPE, HIP)


@pytest.mark.gpu
def test_gradients_in_the_place_of_u_are_refused():
    x, dy = torch.randn((6, 8), device="cuda"), torch.randn((6, 40), device="cuda")
    a, b = torch.randn((2, 8, 8), device="cuda"), torch.randn((2, 40, 8), device="cuda")
    off, index = torch.tensor([0, 4, 6], device="cuda"), torch.tensor([1, 0], device="cuda")
    y, u = nv.nvfp4_adapters(x, a, b, off, index)
    with pytest.raises(nv.NVFP4Error, match="shape"):
        nv.nvfp4_adapters_backward(dy, x, u, a, b, off, index, out=u)
    with pytest.raises(nv.NVFP4Error, match="shape"):
        nv.nvfp4_adapters(x, a, b, off, index, out=b.view(-1)[:240].view(6, 40))
    wide = torch.zeros((6, 100), device="cuda")
    wide[:, 60:] = dy                                          # dx beside dy in one buffer
    want = nv.nvfp4_adapters_backward(dy, x, u, a, b, off, index)
    got = nv.nvfp4_adapters_backward(wide[:, 60:], x, u, a, b, off, index, out=wide[:, 3:11])
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(wide[:, 60:], dy)


# ------------------------------------------------------- binding and modules


def test_binding_refuses_cpu_tensors():
    x, one = torch.zeros(4, 32), torch.zeros(4)
    w = nv.NVFP4Tensor(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(2), 8,
                       32)
    off, index = torch.tensor([0, 4]), torch.tensor([0])
    a, b = torch.zeros(1, 2, 32), torch.zeros(1, 32, 2)
    for call in (lambda: nv.nvfp4_rms_norm(x), lambda: nv.mxfp8_rms_norm(x), lambda: nv.nvfp4_rms_norm_backward(x, x, one),
                 lambda: nv.nvfp4_grouped_matmul(w, x, off), lambda: nv.nvfp4_grouped_wgrad(x, x, off),
                 lambda: nv.nvfp4_adapters(x, a, b, off, index),
                 lambda: nv.nvfp4_adapters_backward(x, x, torch.zeros(4, 2), a, b, off, index)):
        with pytest.raises(nv.NVFP4Error, match="GPU"):
            call()


def test_modules_refuse_shapes():
    x = torch.zeros(4, 32)
    off, index = torch.tensor([0, 2, 4]), torch.tensor([0])
    low = LowRankAdapters(2, 32, 48, 4)
    head = NVFP4Head(32, 48, norm="rms")
    for call, match in ((lambda: RMSNorm(33)(x), "33 features"), (lambda: RMSNorm(32)(x, x[:3]), "residual"),
                        (lambda: NVFP4Head(32, 48, norm="batch"), "norm"),
                        (lambda: head.answer(x, None, adapters=low), "offsets"),
                        (lambda: NVFP4Experts(2, 40, 32), "16"), (lambda: NVFP4Experts(2, 32, 40), "16"),
                        (lambda: NVFP4Experts(2, 16, 32)(x, off), "rows, 16"),
                        (lambda: NVFP4Experts(3, 32, 32)(x, off), "4 entries"),
                        (lambda: NVFP4ExpertBlock(2, 3, 32, 32), "top"),
                        (lambda: low(x[:, :31], None, off, index), "32 features"),
                        (lambda: low(x, x, off, index), "base")):
        with pytest.raises(nv.NVFP4Error, match=match):
            call()


@pytest.mark.parametrize("convert", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16().float(), lambda m: m.double(),
                                     lambda m: torch.nn.Sequential(m).to("cpu", torch.bfloat16)[0]])
def test_adapters_keep_their_scale_in_float32(convert):
    low = LowRankAdapters(3, 32, 48, 4)
    low.scale.copy_(torch.tensor([0.1, 1 / 3, 7.0]))
    want = low.scale.clone()
    out = convert(low)
    assert out is low and low.scale.dtype == torch.float32 and torch.equal(low.scale, want)
    assert "scale" in dict(low.named_buffers()) and torch.equal(low.state_dict()["scale"], want)
    low.to("meta")
    assert low.scale.is_meta and low.scale.dtype == torch.float32


@pytest.mark.gpu
def test_binding_refuses_bad_tensors():
    x = torch.zeros((4, 32), device="cuda")
    one = torch.zeros(4, device="cuda")
    off, index = torch.tensor([0, 2, 4], device="cuda"), torch.tensor([0, 1], device="cuda")
    w = nv.nvfp4_quantize(torch.ones((32, 32), device="cuda"))
    mx = nv.mxfp4_quantize(torch.ones((32, 32), device="cuda"))
    a, b = torch.zeros((2, 3, 32), device="cuda"), torch.zeros((2, 48, 3), device="cuda")
    u = torch.zeros((4, 3), device="cuda")
    dy = torch.zeros((4, 48), device="cuda")
    bad = [
        (lambda: nv.nvfp4_rms_norm(x.half()), "dtype"),
        (lambda: nv.nvfp4_rms_norm(x.t()), "row-major"),
        (lambda: nv.nvfp4_rms_norm(x, one), "vector of 32"),
        (lambda: nv.nvfp4_rms_norm(x, None, x[:3]), "shape"),
        (lambda: nv.nvfp4_rms_norm(x, residual_out=x), "residual"),
        (lambda: nv.nvfp4_rms_norm(x, eps=-1.0), "range"),
        (lambda: nv.nvfp4_rms_norm(x, out=x), "shape"),
        (lambda: nv.nvfp4_rms_norm(x, out_dtype=torch.float16), "output dtype"),
        (lambda: nv.mxfp8_rms_norm(x[:, :24]), "multiple of 32"),
        (lambda: nv.nvfp4_rms_norm_backward(x[:3], x, one), "shape"),
        (lambda: nv.nvfp4_rms_norm_backward(x, x, one[:3]), "rstd"),
        (lambda: nv.nvfp4_rms_norm_backward(x, x, one, dh=x.bfloat16()), "dtype"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, off.float()), "int32 or int64"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, off[:1]), "vector"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, off.cpu()), "GPU|cuda"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, torch.tensor([0, 1, 2, 4], device="cuda")), "experts"),
        (lambda: nv.nvfp4_grouped_matmul(w, x[:, :16], off), "columns"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, off, transposed=True), "columns"),
        (lambda: nv.nvfp4_grouped_matmul(w, x, off, out=torch.empty((4, 15), device="cuda")), "shape"),
        (lambda: nv.mxfp4_grouped_matmul(mx, x.half(), off), "dtype"),
        (lambda: nv.nvfp4_grouped_wgrad(x[:3], x, off), "rows"),
        (lambda: nv.nvfp4_grouped_wgrad(x, x, off, out=torch.empty((2, 32, 31), device="cuda")), "shape"),
        (lambda: nv.nvfp4_grouped_wgrad(x, x, off, torch.float16), "dtype"),
        (lambda: nv.nvfp4_adapters(x, a[0], b, off, index), "3-D"),
        (lambda: nv.nvfp4_adapters(x, a, b[:, :, :2], off, index), "shape"),
        (lambda: nv.nvfp4_adapters(x, a, b.bfloat16(), off, index), "same dtype"),
        (lambda: nv.nvfp4_adapters(x, a, b, off, index.int()), "index"),
        (lambda: nv.nvfp4_adapters(x, a, b, off, index[:1]), "index"),
        (lambda: nv.nvfp4_adapters(x[:, :31], a, b, off, index), "columns"),
        (lambda: nv.nvfp4_adapters(x, a, b, off, index, one[:1]), "scale"),
        (lambda: nv.nvfp4_adapters(x, a, b, off, index, base=x), "shape"),
        (lambda: nv.nvfp4_adapters_backward(x, x, u, a, b, off, index), "shape"),
        (lambda: nv.nvfp4_adapters_backward(dy, x, u[:3], a, b, off, index), "u must|u "),
        (lambda: nv.nvfp4_adapters_backward(dy, x, u, a, b, off, index, out=x), "shape"),
    ]
    for i, (call, match) in enumerate(bad):
        with pytest.raises(nv.NVFP4Error, match=match):
            call()
            pytest.fail(f"case {i} was not refused")
