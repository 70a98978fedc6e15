"""The operators around the linear layer refuse invalid arguments before
anything is launched: the C ABI by status code (where no GPU is visible, since
the pointers are made up), the binding by NVFP4Error."""
import ctypes
import math

import pytest
import torch

import gemm_amax_reduce_amd as nv

FAKE = 0x10000
_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer argument tests run only without a GPU")
NULL, SHAPE, ENUM, ALIGN, VALUE = -1, -2, -3, -5, -6


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def _call(fn, good, **bad):
    """fn with the arguments of `good` (name -> value, in order), some replaced."""
    assert set(bad) <= set(good)
    return fn(*{**good, **bad}.values())


NORM = dict(x=FAKE, xd=1, rows=4, cols=64, ldx=64, w=FAKE, b=FAKE, wd=1, eps=1e-5, y=FAKE, yd=1, ldy=64, mean=FAKE,
            rstd=FAKE, amax=FAKE, ws=FAKE, bytes=1 << 20, stream=None)


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(xd=2), ENUM), (dict(wd=9), ENUM), (dict(yd=-1), ENUM), (dict(cols=0), SHAPE), (dict(rows=-1), SHAPE),
    (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE), (dict(rows=1 << 40, ldx=1 << 30), SHAPE),
    (dict(cols=(1 << 31) + 1, ldx=1 << 32, ldy=1 << 32), SHAPE), (dict(eps=-1e-9), VALUE), (dict(eps=math.nan), VALUE),
    (dict(eps=math.inf), VALUE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(mean=None), NULL),
    (dict(rstd=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(xd=0, x=FAKE + 2), ALIGN), (dict(w=FAKE + 1), ALIGN),
    (dict(amax=FAKE + 2), ALIGN), (dict(mean=FAKE + 2), ALIGN),
    (dict(rows=9, bytes=0), SHAPE), (dict(rows=9, ws=None), NULL), (dict(ws=FAKE + 2), ALIGN)])
def test_layer_norm(L, bad, status):
    assert _call(L.nvfp4_layer_norm, NORM, **bad) == status


BACK = dict(dy=FAKE, dyd=1, lddy=64, x=FAKE, xd=1, rows=4, cols=64, ldx=64, mean=FAKE, rstd=FAKE, w=FAKE, wd=1,
            dx=FAKE, lddx=64, dw=FAKE, db=FAKE, gd=0, ws=FAKE, bytes=1 << 30, stream=None)


@_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(dyd=3), ENUM), (dict(xd=3), ENUM), (dict(wd=3), ENUM), (dict(gd=3), ENUM), (dict(cols=0), SHAPE),
    (dict(rows=-1), SHAPE), (dict(lddy=1), SHAPE), (dict(ldx=1), SHAPE), (dict(lddx=1), SHAPE), (dict(rows=1000, bytes=0), SHAPE),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL),
    (dict(dx=None), NULL), (dict(rows=1000, ws=None), NULL), (dict(ws=FAKE + 8), ALIGN), (dict(dw=FAKE + 2), ALIGN),
    (dict(dx=FAKE + 1), ALIGN)])
def test_layer_norm_backward(L, bad, status):
    assert _call(L.nvfp4_layer_norm_backward, BACK, **bad) == status


@_no_gpu
def test_workspace_sizes(L):
    assert L.nvfp4_layer_norm_backward_workspace_bytes(-1, 64) == SHAPE
    assert L.nvfp4_layer_norm_backward_workspace_bytes(4, 0) == SHAPE
    assert L.nvfp4_layer_norm_backward_workspace_bytes(0, 64) >= 0
    need = L.nvfp4_layer_norm_backward_workspace_bytes(1000, 64)
    assert need > 0
    assert _call(L.nvfp4_layer_norm_backward, BACK, rows=1000, bytes=need - 1) == SHAPE
    assert L.nvfp4_layer_norm_workspace_bytes(-1, 64) == SHAPE
    assert L.nvfp4_layer_norm_workspace_bytes(4, 0) == SHAPE
    assert L.nvfp4_layer_norm_workspace_bytes(0, 64) == L.nvfp4_layer_norm_workspace_bytes(1, 64) == 0
    assert L.nvfp4_layer_norm_workspace_bytes(5, 64) == 20
    assert L.nvfp4_distill_topk_workspace_bytes(-1, 64) == SHAPE
    assert L.nvfp4_distill_topk_workspace_bytes(4, 0) == SHAPE
    assert L.nvfp4_distill_topk_workspace_bytes(4, 1 << 31) == SHAPE
    assert L.nvfp4_distill_topk_workspace_bytes(0, 64) == 0


MV = dict(x=FAKE, xd=1, tokens=2, ldx=64, y=FAKE, yd=0, ldy=8, ws=None, bytes=0, stream=None)


@_no_gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(xd=4), ENUM), (dict(yd=4), ENUM), (dict(tokens=-1), SHAPE), (dict(tokens=1048561), SHAPE),
    (dict(ldx=63), SHAPE), (dict(ldy=7), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=FAKE + 1), ALIGN),
    (dict(y=FAKE + 2), ALIGN), (dict(ws=FAKE + 8), ALIGN)])
def test_matvec(L, mx, bad, status):
    w = nv._MXTensor(FAKE, FAKE, 8, 64) if mx else nv._CTensor(FAKE, FAKE, FAKE, 8, 64)
    fn = L.mxfp4_matvec if mx else L.nvfp4_matvec
    assert fn(ctypes.byref(w), *{**MV, **bad}.values()) == status


@_no_gpu
def test_matvec_weights(L):
    args = list(MV.values())
    by = ctypes.byref
    assert L.nvfp4_matvec(None, *args) == NULL
    assert L.nvfp4_matvec(by(nv._CTensor(FAKE, FAKE, 0, 8, 64)), *args) == NULL
    assert L.nvfp4_matvec(by(nv._CTensor(0, FAKE, FAKE, 8, 64)), *args) == NULL
    assert L.nvfp4_matvec(by(nv._CTensor(FAKE, FAKE, FAKE, 8, 40)), *args) == SHAPE
    assert L.nvfp4_matvec(by(nv._CTensor(FAKE + 4, FAKE, FAKE, 8, 64)), *args) == ALIGN
    assert L.mxfp4_matvec(None, *args) == NULL
    assert L.mxfp4_matvec(by(nv._MXTensor(FAKE, FAKE, 8, 48)), *args) == SHAPE
    assert L.mxfp4_matvec(by(nv._MXTensor(FAKE, 0, 8, 64)), *args) == NULL
    assert L.mxfp4_matvec(by(nv._MXTensor(FAKE + 8, FAKE, 8, 64)), *args) == ALIGN


ROWS = dict(z=FAKE, zd=1, tokens=4, vocab=100, ldz=100, idx=FAKE, bits=64, t=FAKE, td=0, top=8, tau=1.0)
FORWARD = dict(**ROWS, loss=FAKE, lse=FAKE, ws=FAKE, bytes=1 << 20, stream=None)
BACKWARD = dict(**ROWS, lse=FAKE, dloss=FAKE, dz=2 * FAKE, lddz=100, stream=None)
STEP = dict(**ROWS, weight=FAKE, loss=FAKE, lse=FAKE, dz=2 * FAKE, lddz=100, ws=FAKE, bytes=1 << 20, stream=None)
SHARED = [(dict(zd=2), ENUM), (dict(td=2), ENUM), (dict(bits=16), ENUM), (dict(vocab=0), SHAPE),
          (dict(vocab=1 << 31, ldz=1 << 31), SHAPE), (dict(tokens=-1), SHAPE), (dict(ldz=99), SHAPE),
          (dict(top=-1), SHAPE), (dict(top=1025), SHAPE), (dict(tau=0.0), VALUE), (dict(tau=-1.0), VALUE),
          (dict(tau=math.nan), VALUE), (dict(tau=math.inf), VALUE), (dict(z=None), NULL), (dict(idx=None), NULL),
          (dict(t=None), NULL), (dict(lse=None), NULL), (dict(z=FAKE + 1), ALIGN), (dict(idx=FAKE + 4), ALIGN),
          (dict(t=FAKE + 2), ALIGN), (dict(lse=FAKE + 2), ALIGN)]


@_no_gpu
@pytest.mark.parametrize("bad,status", SHARED)
def test_distill_shared(L, bad, status):
    assert _call(L.nvfp4_distill_topk, FORWARD, **bad) == status
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, **bad) == status
    assert _call(L.nvfp4_distill_topk_step, STEP, **bad) == status


@_no_gpu
def test_distill_own_arguments(L):
    assert _call(L.nvfp4_distill_topk, FORWARD, loss=None) == NULL
    long = dict(vocab=1 << 20, ldz=1 << 20)            # rows that need a workspace
    assert L.nvfp4_distill_topk_workspace_bytes(4, 100) == 0 < L.nvfp4_distill_topk_workspace_bytes(4, 1 << 20)
    assert _call(L.nvfp4_distill_topk, FORWARD, **long, ws=None) == NULL
    assert _call(L.nvfp4_distill_topk, FORWARD, **long, bytes=0) == SHAPE
    assert _call(L.nvfp4_distill_topk, FORWARD, ws=FAKE + 8) == ALIGN
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, dloss=None) == NULL
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, dz=None) == NULL
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, lddz=99) == SHAPE
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, dz=FAKE) == SHAPE               # in place
    assert _call(L.nvfp4_distill_topk_backward, BACKWARD, dz=FAKE + 798) == SHAPE         # last element
    assert _call(L.nvfp4_distill_topk_step, STEP, weight=None) == NULL
    assert _call(L.nvfp4_distill_topk_step, STEP, loss=None) == NULL
    assert _call(L.nvfp4_distill_topk_step, STEP, dz=FAKE + 100) == SHAPE
    assert _call(L.nvfp4_distill_topk_step, STEP, **{**long, "lddz": 1 << 20, "dz": 1 << 30}, bytes=0) == SHAPE
    assert _call(L.nvfp4_distill_topk_step, STEP, dz=2 * FAKE + 1) == ALIGN


def test_status_string():
    assert nv.lib().nvfp4_status_string(VALUE) == b"scalar argument out of range"


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 32)
    idx, t = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    one = torch.zeros(4)
    w = nv.NVFP4Tensor(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(2), 8,
                       32)
    for call in (lambda: nv.nvfp4_layer_norm(x), lambda: nv.nvfp4_layer_norm_backward(x, x, one, one),
                 lambda: nv.nvfp4_matvec(w, x), lambda: nv.nvfp4_distill_topk(x, idx, t),
                 lambda: nv.nvfp4_distill_topk_backward(x, idx, t, one, one),
                 lambda: nv.nvfp4_distill_topk_step(x, idx, t, one)):
        with pytest.raises(nv.NVFP4Error, match="GPU"):
            call()


@pytest.mark.gpu
def test_binding_refuses_bad_tensors():
    x = torch.zeros((4, 32), device="cuda")
    one = torch.zeros(4, device="cuda")
    idx, t = torch.zeros((4, 2), dtype=torch.int64, device="cuda"), torch.zeros((4, 2), device="cuda")
    w = nv.nvfp4_quantize(torch.ones((8, 32), device="cuda"))
    mx = nv.mxfp4_quantize(torch.ones((8, 32), device="cuda"))
    bad = [
        (lambda: nv.nvfp4_layer_norm(x.half()), "dtype"),
        (lambda: nv.nvfp4_layer_norm(x[0]), "2-D"),
        (lambda: nv.nvfp4_layer_norm(x.t()), "row-major"),
        (lambda: nv.nvfp4_layer_norm(x[:1].expand(4, 32)), "overlap"),
        (lambda: nv.nvfp4_layer_norm(x, one), "vector of 32"),
        (lambda: nv.nvfp4_layer_norm(x, torch.zeros(32)), "GPU"),
        (lambda: nv.nvfp4_layer_norm(x, x[0], x[0].bfloat16()), "same dtype"),
        (lambda: nv.nvfp4_layer_norm(x, eps=-1.0), "range"),
        (lambda: nv.nvfp4_layer_norm(x, out_dtype=torch.float16), "output dtype"),
        (lambda: nv.nvfp4_layer_norm(x, out=torch.empty((4, 31), device="cuda")), "shape"),
        (lambda: nv.nvfp4_layer_norm(torch.empty((3, 0), device="cuda")), "shape"),
        (lambda: nv.nvfp4_layer_norm_backward(x[:3], x, one, one), "shape"),
        (lambda: nv.nvfp4_layer_norm_backward(x, x, one[:3], one), "mean"),
        (lambda: nv.nvfp4_layer_norm_backward(x, x, one, one.double()), "rstd"),
        (lambda: nv.nvfp4_matvec(w, x[:, :16]), "columns"),
        (lambda: nv.nvfp4_matvec(w, x.half()), "dtype"),
        (lambda: nv.mxfp4_matvec(mx, x, out=torch.empty((4, 7), device="cuda")), "shape"),
        (lambda: nv.nvfp4_distill_topk(x, idx.float(), t), "int32 or int64"),
        (lambda: nv.nvfp4_distill_topk(x, idx[:3], t[:3]), "shape"),
        (lambda: nv.nvfp4_distill_topk(x, idx, t[:, :1]), "shape"),
        (lambda: nv.nvfp4_distill_topk(x, idx, t.half()), "dtype"),
        (lambda: nv.nvfp4_distill_topk(x, idx.t().contiguous().t(), t), "contiguous"),
        (lambda: nv.nvfp4_distill_topk(x, idx, t, temperature=0.0), "range"),
        (lambda: nv.nvfp4_distill_topk_step(x, idx, t, one.double()), "weight"),
        (lambda: nv.nvfp4_distill_topk_step(x, idx, t, one, out=x), "shape"),
        (lambda: nv.nvfp4_distill_topk_backward(x, idx, t, one, one[:2]), "dloss"),
    ]
    for i, (call, match) in enumerate(bad):
        with pytest.raises(nv.NVFP4Error, match=match):
            call()
            pytest.fail(f"case {i} was not refused")


@_no_gpu
def test_matvec_size_limits(L):
    k = 1 << 25
    args = list({**MV, "ldx": k}.values())
    assert L.nvfp4_matvec(ctypes.byref(nv._CTensor(FAKE, FAKE, FAKE, 8, k)), *args) == SHAPE
    assert L.mxfp4_matvec(ctypes.byref(nv._MXTensor(FAKE, FAKE, 8, k)), *args) == SHAPE


@_no_gpu
def test_matvec_workspace(L):
    size = L.nvfp4_matvec_workspace_bytes
    assert size(8, 64, 2, 7) == ENUM
    for bad in ((-1, 64, 2), (8, 40, 2), (8, -16, 2), (8, 64, -1), (8, 64, 1048561), (8, 1 << 25, 2)):
        assert size(*bad, 1) == SHAPE
    assert size(8, 64, 1, 1) == 0 and size(0, 64, 2, 1) == 0 and size(8, 64, 0, 0) == 0 and size(8, 16, 2, 0) == 0
    k = 1 << 20
    need = size(8, k, 2, 1)
    assert need > 0 and need % 4 == 0
    w = nv._CTensor(FAKE, FAKE, FAKE, 8, k)
    args = {**MV, "ldx": k}
    assert L.nvfp4_matvec(ctypes.byref(w), *{**args, "ws": FAKE, "bytes": need - 1}.values()) == SHAPE
    assert L.nvfp4_matvec(ctypes.byref(w), *{**args, "bytes": need}.values()) == NULL
