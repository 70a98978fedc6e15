"""Python binding of the MI355X NVFP4 linear-layer library (``libnvfp4.so``).

Argument marshalling only: every step of quantize / dequantize / GEMM runs in
the gfx950 kernels behind the C ABI of ``include/nvfp4.h``.  torch supplies
device memory and the current HIP stream.  There is no CPU fallback: if the
library is not built, or no GPU is visible, the calls raise.

Names follow the C ABI: ``nvfp4_quantize``, ``nvfp4_rht_quantize``,
``nvfp4_dequantize``, ``nvfp4_gemm``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

__all__ = ["NVFP4Tensor", "NVFP4Error", "nvfp4_quantize", "nvfp4_rht_quantize", "nvfp4_quantize_dual", "nvfp4_amax",
           "nvfp4_quantize_amax", "MXFP4Tensor", "mxfp4_quantize", "mxfp4_gemm", "MXFP8Tensor", "mxfp8_quantize",
           "mxfp8_gemm",
           "nvfp4_dequantize", "nvfp4_gemm", "nvfp4_gemm_ws", "nvfp4_gemm_noalloc", "gemm_workspace",
           "nvfp4_layer_norm", "nvfp4_layer_norm_backward", "nvfp4_rms_norm", "mxfp8_rms_norm",
           "nvfp4_rms_norm_backward", "nvfp4_matvec", "mxfp4_matvec", "nvfp4_grouped_matmul", "mxfp4_grouped_matmul",
           "nvfp4_grouped_wgrad", "nvfp4_adapters", "nvfp4_adapters_backward", "nvfp4_distill_topk",
           "nvfp4_distill_topk_backward", "nvfp4_distill_topk_step",
           "lib", "LIB_PATH", "F32", "BF16", "RNE", "SR"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

F32, BF16 = 0, 1
RNE, SR = 0, 1


class NVFP4Error(RuntimeError):
    pass


class _CTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("outer", ctypes.c_int64), ("k", ctypes.c_int64)]


class _MXTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("outer", ctypes.c_int64),
                ("k", ctypes.c_int64)]


_lib = None

# every symbol the header declares
EXPORTS = ("nvfp4_quantize", "nvfp4_rht_quantize", "nvfp4_amax", "nvfp4_quantize_amax", "nvfp4_quantize_dual",
           "mxfp4_quantize", "mxfp4_gemm", "nvfp4_dequantize", "nvfp4_gemm", "nvfp4_gemm_ws",
           "nvfp4_gemm_workspace_bytes", "nvfp4_gemm_noalloc", "mxfp8_quantize", "mxfp8_gemm", "nvfp4_layer_norm",
           "nvfp4_layer_norm_workspace_bytes", "nvfp4_layer_norm_backward", "nvfp4_layer_norm_backward_workspace_bytes",
           "nvfp4_rms_norm", "mxfp8_rms_norm", "nvfp4_rms_norm_backward", "nvfp4_rms_norm_backward_workspace_bytes",
           "nvfp4_matvec", "mxfp4_matvec",
           "nvfp4_matvec_workspace_bytes", "nvfp4_grouped_matmul", "mxfp4_grouped_matmul",
           "nvfp4_grouped_matmul_workspace_bytes", "nvfp4_grouped_wgrad", "nvfp4_grouped_wgrad_workspace_bytes",
           "nvfp4_adapters", "nvfp4_adapters_backward",
           "nvfp4_adapters_backward_workspace_bytes", "nvfp4_distill_topk", "nvfp4_distill_topk_backward",
           "nvfp4_distill_topk_step", "nvfp4_distill_topk_workspace_bytes", "nvfp4_probe_mfma", "nvfp4_probe_philox", "nvfp4_status_string")


def lib() -> ctypes.CDLL:
    """Load ``libnvfp4.so`` (build it with ``gemm_amax_reduce_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise NVFP4Error(f"{LIB_PATH} is missing: run gemm_amax_reduce_amd/build.py "
                             "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        i64, u64, vp, ci = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int
        pt = ctypes.POINTER(_CTensor)
        L.nvfp4_quantize.argtypes = [vp, ci, i64, i64, ci, ci, u64, u64, pt, vp]
        L.nvfp4_quantize.restype = ci
        L.nvfp4_rht_quantize.argtypes = [vp, ci, i64, i64, ci, ci, u64, u64, ctypes.c_uint16, pt, vp]
        L.nvfp4_rht_quantize.restype = ci
        mt = ctypes.POINTER(_MXTensor)
        L.mxfp4_quantize.argtypes = [vp, ci, i64, i64, ci, mt, vp]
        L.mxfp4_quantize.restype = ci
        L.mxfp4_gemm.argtypes = [mt, mt, vp, ci, i64, vp]
        L.mxfp4_gemm.restype = ci
        L.mxfp8_quantize.argtypes = [vp, ci, i64, i64, ci, mt, vp]
        L.mxfp8_quantize.restype = ci
        L.mxfp8_gemm.argtypes = [mt, mt, vp, ci, i64, vp]
        L.mxfp8_gemm.restype = ci
        L.nvfp4_amax.argtypes = [vp, ci, i64, i64, ci, ci, ctypes.c_uint16, vp, vp]
        L.nvfp4_amax.restype = ci
        L.nvfp4_quantize_amax.argtypes = [vp, ci, i64, i64, ci, ci, u64, u64, ci, ctypes.c_uint16, vp, pt, vp]
        L.nvfp4_quantize_amax.restype = ci
        L.nvfp4_quantize_dual.argtypes = [vp, ci, i64, i64, ci, u64, u64, pt, ci, ctypes.c_uint16, ci, u64, u64,
                                          pt, vp]
        L.nvfp4_quantize_dual.restype = ci
        L.nvfp4_dequantize.argtypes = [pt, vp, ci, vp]
        L.nvfp4_dequantize.restype = ci
        L.nvfp4_gemm.argtypes = [pt, pt, vp, ci, i64, vp]
        L.nvfp4_gemm.restype = ci
        L.nvfp4_gemm_ws.argtypes = [pt, pt, vp, ci, i64, vp, i64, vp]
        L.nvfp4_gemm_ws.restype = ci
        L.nvfp4_gemm_workspace_bytes.argtypes = []
        L.nvfp4_gemm_noalloc.argtypes = [pt, pt, vp, ci, i64, vp]
        L.nvfp4_gemm_noalloc.restype = ci
        L.nvfp4_gemm_workspace_bytes.restype = i64
        cf = ctypes.c_float
        L.nvfp4_layer_norm.argtypes = [vp, ci, i64, i64, i64, vp, vp, ci, cf, vp, ci, i64, vp, vp, vp, vp, i64, vp]
        L.nvfp4_layer_norm_workspace_bytes.argtypes = [i64, i64]
        L.nvfp4_layer_norm_workspace_bytes.restype = i64
        L.nvfp4_layer_norm.restype = ci
        L.nvfp4_layer_norm_backward.argtypes = [vp, ci, i64, vp, ci, i64, i64, i64, vp, vp, vp, ci, vp, i64, vp, vp,
                                                ci, vp, i64, vp]
        L.nvfp4_layer_norm_backward.restype = ci
        L.nvfp4_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
        L.nvfp4_layer_norm_backward_workspace_bytes.restype = i64
        rms = [vp, ci, i64, i64, i64, vp, ci, i64, vp, i64, vp, ci, cf]      # x, residual, h, weight, eps
        L.nvfp4_rms_norm.argtypes = rms + [vp, ci, i64, vp, vp]
        L.nvfp4_rms_norm.restype = ci
        L.mxfp8_rms_norm.argtypes = rms + [mt, vp, vp]
        L.mxfp8_rms_norm.restype = ci
        L.nvfp4_rms_norm_backward.argtypes = [vp, ci, i64, vp, ci, i64, i64, i64, vp, vp, ci, vp, i64, vp, i64, vp, ci,
                                              vp, i64, vp]
        L.nvfp4_rms_norm_backward.restype = ci
        L.nvfp4_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
        L.nvfp4_rms_norm_backward_workspace_bytes.restype = i64
        L.nvfp4_matvec.argtypes = [pt, vp, ci, i64, i64, vp, ci, i64, vp, i64, vp]
        L.nvfp4_matvec.restype = ci
        L.mxfp4_matvec.argtypes = [mt, vp, ci, i64, i64, vp, ci, i64, vp, i64, vp]
        L.mxfp4_matvec.restype = ci
        L.nvfp4_matvec_workspace_bytes.argtypes = [i64, i64, i64, ci]
        L.nvfp4_matvec_workspace_bytes.restype = i64
        groups = [ci, vp, ci, i64, i64, vp, ci, i64, vp, ci, i64, ci, vp, i64, vp]
        L.nvfp4_grouped_matmul.argtypes = [pt] + groups
        L.nvfp4_grouped_matmul.restype = ci
        L.mxfp4_grouped_matmul.argtypes = [mt] + groups
        L.mxfp4_grouped_matmul.restype = ci
        L.nvfp4_grouped_matmul_workspace_bytes.argtypes = [i64, i64, i64, i64, ci]
        L.nvfp4_grouped_matmul_workspace_bytes.restype = i64
        L.nvfp4_grouped_wgrad.argtypes = [vp, ci, i64, vp, ci, i64, i64, i64, i64, vp, ci, i64, vp, ci, vp, i64, vp]
        L.nvfp4_grouped_wgrad.restype = ci
        L.nvfp4_grouped_wgrad_workspace_bytes.argtypes = [i64, i64, i64, i64, ci, ci]
        L.nvfp4_grouped_wgrad_workspace_bytes.restype = i64
        low = [vp, vp, ci, i64, i64, i64, vp, vp, vp, ci, i64]               # adapters, scale, segments
        L.nvfp4_adapters.argtypes = [vp, ci, i64, i64, i64] + low + [vp, ci, i64, vp, ci, i64, vp, vp]
        L.nvfp4_adapters.restype = ci
        L.nvfp4_adapters_backward.argtypes = ([vp, ci, i64, vp, ci, i64, i64, i64, vp] + low +
                                              [vp, ci, i64, vp, ci, i64, vp, vp, ci, vp, i64, vp])
        L.nvfp4_adapters_backward.restype = ci
        L.nvfp4_adapters_backward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64, ci]
        L.nvfp4_adapters_backward_workspace_bytes.restype = i64
        rows = [vp, ci, i64, i64, i64, vp, ci, vp, ci, i64, cf]       # logits, indices, teacher, temperature
        L.nvfp4_distill_topk.argtypes = rows + [vp, vp, vp, i64, vp]
        L.nvfp4_distill_topk.restype = ci
        L.nvfp4_distill_topk_backward.argtypes = rows + [vp, vp, vp, i64, vp]
        L.nvfp4_distill_topk_backward.restype = ci
        L.nvfp4_distill_topk_step.argtypes = rows + [vp, vp, vp, vp, i64, vp, i64, vp]
        L.nvfp4_distill_topk_step.restype = ci
        L.nvfp4_distill_topk_workspace_bytes.argtypes = [i64, i64]
        L.nvfp4_distill_topk_workspace_bytes.restype = i64
        L.nvfp4_probe_mfma.argtypes = [i64, vp, vp]
        L.nvfp4_probe_mfma.restype = ci
        L.nvfp4_probe_philox.argtypes = [i64, vp, vp]
        L.nvfp4_probe_philox.restype = ci
        L.nvfp4_status_string.argtypes = [ci]
        L.nvfp4_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = lib().nvfp4_status_string(rc).decode()
        raise NVFP4Error(f"{what} failed: {msg} ({rc})")


def _stream_handle(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


def _require_device(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise NVFP4Error(f"{name} must be a GPU tensor (no CPU path exists)")


def _require_buffer(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int, device: torch.device):
    """A caller-supplied device buffer the kernels write or read whole: the
    C ABI cannot see its size, so it is checked here."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise NVFP4Error(f"{name} must be a GPU tensor on {device}")
    if t.dtype != dtype:
        raise NVFP4Error(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous() or t.numel() < numel:
        raise NVFP4Error(f"{name} must be contiguous with at least {numel} elements")


def _vector(t, name: str, dtype: torch.dtype, numel: int, device: torch.device) -> int:
    """The address of a device vector that the kernels read whole
    (_require_buffer says what is wrong with one that they cannot)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.numel() >= numel
            and t.device == device and t.is_contiguous()):
        _require_buffer(t, name, dtype, numel, device)
    return t.data_ptr()


def _out_code(dtype) -> int:
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise NVFP4Error(f"unsupported output dtype {dtype} (float32 or bfloat16)")


def _require_matrix_out(out: torch.Tensor, rows: int, cols: int, dtype, device: torch.device) -> int:
    """Check a caller-supplied [rows][cols] output view (row stride >= cols)
    and return its leading dimension."""
    if not isinstance(out, torch.Tensor) or not out.is_cuda or out.device != device:
        raise NVFP4Error(f"out must be a GPU tensor on {device}")
    if out.dtype != dtype:
        raise NVFP4Error(f"out has dtype {out.dtype}, expected {dtype}")
    if out.dim() != 2 or tuple(out.shape) != (rows, cols):
        raise NVFP4Error(f"out must have shape ({rows}, {cols}), got {tuple(out.shape)}")
    if cols > 1 and out.stride(1) != 1:
        raise NVFP4Error("out must be row-major (unit column stride)")
    if rows > 1 and out.stride(0) < cols:
        raise NVFP4Error("out rows overlap (row stride < columns)")
    return out.stride(0) if rows > 1 else max(cols, 1)


class NVFP4Tensor:
    """Device buffers of one NVFP4 tensor in its quantized [outer][k] layout:
    ``codes`` u8 [outer, k/2], ``scales`` u8 [outer, k/16], ``meta`` f32 [2]
    = (amax, g)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, meta: torch.Tensor, outer: int, k: int):
        self.codes, self.scales, self.meta = codes, scales, meta
        self.outer, self.k = int(outer), int(k)

    @classmethod
    def empty(cls, outer: int, k: int, device=None) -> "NVFP4Tensor":
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        codes = torch.empty((outer, k // 2), dtype=torch.uint8, device=device)
        scales = torch.empty((outer, k // 16), dtype=torch.uint8, device=device)
        meta = torch.empty(2, dtype=torch.float32, device=device)
        return cls(codes, scales, meta, outer, k)

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def _c(self) -> _CTensor:
        if self.outer < 0 or self.k < 0 or self.k % 16:
            raise NVFP4Error(f"invalid NVFP4 shape ({self.outer}, {self.k})")
        dev = self.codes.device
        return _CTensor(_vector(self.codes, "codes", torch.uint8, self.outer * (self.k // 2), dev),
                        _vector(self.scales, "scales", torch.uint8, self.outer * (self.k // 16), dev),
                        _vector(self.meta, "meta", torch.float32, 2, dev), self.outer, self.k)

    @property
    def shape(self):
        return (self.outer, self.k)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise NVFP4Error(f"unsupported input dtype {t.dtype} (f32 or bf16)")


def _rounding_code(r) -> int:
    if isinstance(r, str):
        r = {"rne": RNE, "sr": SR}[r.lower()]
    return int(r)


def _same_device(q, x: torch.Tensor):
    if q.device != x.device:
        raise NVFP4Error(f"output on {q.device}, input on {x.device}")


def _quantize(x, axis, rounding, seed, offset, rht, sign_mask, out, stream):
    _require_device(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    rows, cols = x.shape
    outer, k = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = NVFP4Tensor.empty(outer, k, device=x.device)
    _same_device(out, x)
    ct = out._c()
    with torch.cuda.device(x.device):
        if rht:
            rc = lib().nvfp4_rht_quantize(x.data_ptr(), _dtype_code(x), rows, cols, axis, _rounding_code(rounding),
                                          seed, offset, sign_mask & 0xFFFF, ctypes.byref(ct),
                                          _stream_handle(stream, x.device))
        else:
            rc = lib().nvfp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, axis, _rounding_code(rounding),
                                      seed, offset, ctypes.byref(ct), _stream_handle(stream, x.device))
    _check(rc, "nvfp4_rht_quantize" if rht else "nvfp4_quantize")
    return out


def nvfp4_quantize(x: torch.Tensor, axis: int = 1, rounding="rne", seed: int = 0, offset: int = 0,
                   out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """Quantize a 2-D f32/bf16 GPU tensor to NVFP4 (see include/nvfp4.h)."""
    return _quantize(x, axis, rounding, seed, offset, False, 0, out, stream)


def nvfp4_rht_quantize(x: torch.Tensor, sign_mask: int, axis: int = 1, rounding="rne", seed: int = 0,
                       offset: int = 0, out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """Quantize after the 16-point random Hadamard transform along k."""
    return _quantize(x, axis, rounding, seed, offset, True, sign_mask, out, stream)


def nvfp4_amax(x: torch.Tensor, axis: int = 1, rht: bool = False, sign_mask: int = 0,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The tensor amax of x on `axis` (after the RHT if rht), as f32 [1] on x's device."""
    _require_device(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _require_buffer(out, "out", torch.float32, 1, x.device)
    rows, cols = x.shape
    with torch.cuda.device(x.device):
        _check(lib().nvfp4_amax(x.data_ptr(), _dtype_code(x), rows, cols, axis, int(bool(rht)), sign_mask & 0xFFFF,
                                out.data_ptr(), _stream_handle(stream, x.device)), "nvfp4_amax")
    return out


def nvfp4_quantize_amax(x: torch.Tensor, amax: torch.Tensor, axis: int = 1, rounding="rne", seed: int = 0,
                        offset: int = 0, rht: bool = False, sign_mask: int = 0,
                        out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """Quantize with the tensor amax supplied (device f32, element 0)."""
    _require_device(x, "x")
    _require_device(amax, "amax")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    _require_buffer(amax, "amax", torch.float32, 1, x.device)
    rows, cols = x.shape
    outer, k = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = NVFP4Tensor.empty(outer, k, device=x.device)
    _same_device(out, x)
    ct = out._c()
    with torch.cuda.device(x.device):
        _check(lib().nvfp4_quantize_amax(x.data_ptr(), _dtype_code(x), rows, cols, axis, _rounding_code(rounding),
                                         seed, offset, int(bool(rht)), sign_mask & 0xFFFF, amax.data_ptr(),
                                         ctypes.byref(ct), _stream_handle(stream, x.device)), "nvfp4_quantize_amax")
    return out


def nvfp4_quantize_dual(x: torch.Tensor, rounding1="rne", seed1: int = 0, offset1: int = 0,
                        rht0: bool = False, sign_mask0: int = 0, rounding0="rne", seed0: int = 0,
                        offset0: int = 0, out1: NVFP4Tensor | None = None, out0: NVFP4Tensor | None = None,
                        stream=None) -> tuple[NVFP4Tensor, NVFP4Tensor]:
    """Both layouts of x with one amax read: (axis-1 tensor, axis-0 tensor),
    bit-identical to the two single quantizations (see include/nvfp4.h)."""
    _require_device(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    rows, cols = x.shape
    if out1 is None:
        out1 = NVFP4Tensor.empty(rows, cols, device=x.device)
    if out0 is None:
        out0 = NVFP4Tensor.empty(cols, rows, device=x.device)
    _same_device(out1, x)
    _same_device(out0, x)
    c1, c0 = out1._c(), out0._c()
    with torch.cuda.device(x.device):
        rc = lib().nvfp4_quantize_dual(x.data_ptr(), _dtype_code(x), rows, cols, _rounding_code(rounding1), seed1,
                                       offset1, ctypes.byref(c1), int(bool(rht0)), sign_mask0 & 0xFFFF,
                                       _rounding_code(rounding0), seed0, offset0, ctypes.byref(c0),
                                       _stream_handle(stream, x.device))
    _check(rc, "nvfp4_quantize_dual")
    return out1, out0


def nvfp4_dequantize(q: NVFP4Tensor, dtype=torch.float32, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Decode to f32/bf16 in the quantized [outer][k] layout."""
    code = _out_code(dtype)
    dev = q.device
    if out is None:
        out = torch.empty((q.outer, q.k), dtype=dtype, device=dev)
    _require_buffer(out, "out", dtype, q.outer * q.k, dev)
    ct = q._c()
    with torch.cuda.device(dev):
        _check(lib().nvfp4_dequantize(ctypes.byref(ct), out.data_ptr(), code, _stream_handle(stream, dev)),
               "nvfp4_dequantize")
    return out


def nvfp4_gemm(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """C = A . B^T for A [M, K] and B [N, K] NVFP4 tensors, f32 accumulation."""
    code = _out_code(out_dtype)
    dev = a.device
    if b.device != dev:
        raise NVFP4Error(f"operands on {a.device} and {b.device}")
    if out is None:
        out = torch.empty((a.outer, b.outer), dtype=out_dtype, device=dev)
    ldc = _require_matrix_out(out, a.outer, b.outer, out_dtype, dev)
    ca, cb = a._c(), b._c()
    with torch.cuda.device(dev):
        _check(lib().nvfp4_gemm(ctypes.byref(ca), ctypes.byref(cb), out.data_ptr(), code, ldc,
                                _stream_handle(stream, dev)), "nvfp4_gemm")
    return out


_workspaces: dict = {}
# of one, what the kernel needs zero-filled (its flags)
_WORKSPACE_FLAGS = 1 << 16


def gemm_workspace(device=None, stream=None) -> torch.Tensor:
    """The split-tail GEMM workspace for one (device, stream): allocated
    zero-filled on first use and kept (the kernel leaves it zero-filled).
    Calls on one stream run in order, so a workspace per stream is never
    used by two calls at once.  Under capture it is a new one, its flags
    cleared by the graph itself, and is not kept: graphs captured on one stream
    may be replayed in any order, on any streams."""
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with _on(device, stream):                    # its memory and its clearing are the stream's
        return _stream_workspace(device, stream if stream is not None else torch.cuda.current_stream(device))


def _stream_workspace(device, s) -> torch.Tensor:
    size = int(lib().nvfp4_gemm_workspace_bytes())
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        ws[:_WORKSPACE_FLAGS].zero_()
        return ws
    key = (device, int(s.cuda_stream))
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros(size, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def nvfp4_gemm_ws(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C = A . B^T with a workspace (same result contract as nvfp4_gemm):
    the tiles of a partly filled last round split into K ranges where that
    is faster; `workspace` defaults to the one of (device, stream)."""
    code = _out_code(out_dtype)
    dev = a.device
    if b.device != dev:
        raise NVFP4Error(f"operands on {a.device} and {b.device}")
    if out is None:
        out = torch.empty((a.outer, b.outer), dtype=out_dtype, device=dev)
    ldc = _require_matrix_out(out, a.outer, b.outer, out_dtype, dev)
    ws = workspace if workspace is not None else gemm_workspace(dev, stream)
    _require_buffer(ws, "workspace", torch.uint8, int(lib().nvfp4_gemm_workspace_bytes()), dev)
    ca, cb = a._c(), b._c()
    with torch.cuda.device(dev):
        _check(lib().nvfp4_gemm_ws(ctypes.byref(ca), ctypes.byref(cb), out.data_ptr(), code, ldc, ws.data_ptr(),
                                   ws.numel(), _stream_handle(stream, dev)), "nvfp4_gemm_ws")
    return out


def nvfp4_gemm_noalloc(a: NVFP4Tensor, b: NVFP4Tensor, out: torch.Tensor, out_dtype=torch.float32,
                       stream=None) -> torch.Tensor:
    """nvfp4_gemm_ws with the library's own per-GPU workspace: allocates
    nothing (the caller supplies `out`).  Calls overlapping in time on one
    GPU race."""
    code = _out_code(out_dtype)
    dev = a.device
    if b.device != dev:
        raise NVFP4Error(f"operands on {a.device} and {b.device}")
    ldc = _require_matrix_out(out, a.outer, b.outer, out_dtype, dev)
    ca, cb = a._c(), b._c()
    with torch.cuda.device(dev):
        _check(lib().nvfp4_gemm_noalloc(ctypes.byref(ca), ctypes.byref(cb), out.data_ptr(), code, ldc,
                                        _stream_handle(stream, dev)), "nvfp4_gemm_noalloc")
    return out


def nvfp4_probe_mfma(iters: int, stream=None) -> float:
    """Run the MFMA ceiling probe (include/nvfp4.h) once on the current device
    and return its rate in TFLOP/s, timed with events on the probe's stream.
    A measurement helper for the benchmark, not part of the method."""
    dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.empty(1024 * 256, dtype=torch.float32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(s):
        _check(lib().nvfp4_probe_mfma(min(iters, 8), out.data_ptr(), _stream_handle(s, dev)), "nvfp4_probe_mfma")
        e0.record(s)
        _check(lib().nvfp4_probe_mfma(iters, out.data_ptr(), _stream_handle(s, dev)), "nvfp4_probe_mfma")
        e1.record(s)
    e1.synchronize()
    return 1024 * 4 * iters * 32 * 32768 / (e0.elapsed_time(e1) * 1e-3) / 1e12


def nvfp4_probe_philox(calls: int, stream=None) -> float:
    """Run the Philox probe (include/nvfp4.h) once for `calls` counters on the
    current device and return its time in ms (events on the probe's stream).
    A measurement helper for the benchmark, not part of the method."""
    dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.empty(4096 * 256, dtype=torch.int32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(s):
        _check(lib().nvfp4_probe_philox(min(calls, 1 << 20), out.data_ptr(), _stream_handle(s, dev)),
               "nvfp4_probe_philox")
        e0.record(s)
        _check(lib().nvfp4_probe_philox(calls, out.data_ptr(), _stream_handle(s, dev)), "nvfp4_probe_philox")
        e1.record(s)
    e1.synchronize()
    return e0.elapsed_time(e1)


class MXFP4Tensor:
    """Device buffers of one MXFP4 tensor in its quantized [outer][k] layout:
    ``codes`` u8 [outer, k/2], ``scales`` u8 [outer, k/32] (E8M0)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, outer: int, k: int):
        self.codes, self.scales, self.outer, self.k = codes, scales, int(outer), int(k)

    @classmethod
    def empty(cls, outer: int, k: int, device=None) -> "MXFP4Tensor":
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        return cls(torch.empty((outer, k // 2), dtype=torch.uint8, device=device),
                   torch.empty((outer, k // 32), dtype=torch.uint8, device=device), outer, k)

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def _c(self) -> _MXTensor:
        if self.outer < 0 or self.k < 0 or self.k % 32:
            raise NVFP4Error(f"invalid MXFP4 shape ({self.outer}, {self.k})")
        dev = self.codes.device
        return _MXTensor(_vector(self.codes, "codes", torch.uint8, self.outer * (self.k // 2), dev),
                         _vector(self.scales, "scales", torch.uint8, self.outer * (self.k // 32), dev), self.outer,
                         self.k)


def mxfp4_quantize(x: torch.Tensor, axis: int = 1, out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """Quantize a 2-D f32/bf16 GPU tensor to MXFP4 (see include/nvfp4.h)."""
    _require_device(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    rows, cols = x.shape
    outer, k = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = MXFP4Tensor.empty(outer, k, device=x.device)
    _same_device(out, x)
    ct = out._c()
    with torch.cuda.device(x.device):
        _check(lib().mxfp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, axis, ctypes.byref(ct),
                                    _stream_handle(stream, x.device)), "mxfp4_quantize")
    return out


def mxfp4_gemm(a: MXFP4Tensor, b: MXFP4Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """C = A . B^T for MXFP4 A [M, K] and B [N, K] (K % 256 == 0), f32 accumulation."""
    code = _out_code(out_dtype)
    dev = a.device
    if b.device != dev:
        raise NVFP4Error(f"operands on {a.device} and {b.device}")
    if out is None:
        out = torch.empty((a.outer, b.outer), dtype=out_dtype, device=dev)
    ldc = _require_matrix_out(out, a.outer, b.outer, out_dtype, dev)
    ca, cb = a._c(), b._c()
    with torch.cuda.device(dev):
        _check(lib().mxfp4_gemm(ctypes.byref(ca), ctypes.byref(cb), out.data_ptr(), code, ldc,
                                _stream_handle(stream, dev)), "mxfp4_gemm")
    return out



class MXFP8Tensor:
    """Device buffers of one MXFP8 tensor in its quantized [outer][k] layout:
    ``codes`` u8 [outer, k] (E4M3), ``scales`` u8 [outer, k/32] (E8M0).  The
    C struct has the same fields as the MXFP4 one."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, outer: int, k: int):
        self.codes, self.scales, self.outer, self.k = codes, scales, int(outer), int(k)

    @classmethod
    def empty(cls, outer: int, k: int, device=None) -> "MXFP8Tensor":
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        return cls(torch.empty((outer, k), dtype=torch.uint8, device=device),
                   torch.empty((outer, k // 32), dtype=torch.uint8, device=device), outer, k)

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def _c(self) -> _MXTensor:
        if self.outer < 0 or self.k < 0 or self.k % 32:
            raise NVFP4Error(f"invalid MXFP8 shape ({self.outer}, {self.k})")
        dev = self.codes.device
        _require_buffer(self.codes, "codes", torch.uint8, self.outer * self.k, dev)
        _require_buffer(self.scales, "scales", torch.uint8, self.outer * (self.k // 32), dev)
        return _MXTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.outer, self.k)


def mxfp8_quantize(x: torch.Tensor, axis: int = 1, out: MXFP8Tensor | None = None, stream=None) -> MXFP8Tensor:
    """Quantize a 2-D f32/bf16 GPU tensor to MXFP8 (see include/nvfp4.h)."""
    _require_device(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise NVFP4Error("x must be a contiguous 2-D tensor")
    rows, cols = x.shape
    outer, k = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = MXFP8Tensor.empty(outer, k, device=x.device)
    _same_device(out, x)
    ct = out._c()
    with torch.cuda.device(x.device):
        _check(lib().mxfp8_quantize(x.data_ptr(), _dtype_code(x), rows, cols, axis, ctypes.byref(ct),
                                    _stream_handle(stream, x.device)), "mxfp8_quantize")
    return out


def mxfp8_gemm(a: MXFP8Tensor, b: MXFP8Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """C = A . B^T for MXFP8 A [M, K] and B [N, K] (K % 128 == 0), f32 accumulation."""
    code = _out_code(out_dtype)
    dev = a.device
    if b.device != dev:
        raise NVFP4Error(f"operands on {a.device} and {b.device}")
    if out is None:
        out = torch.empty((a.outer, b.outer), dtype=out_dtype, device=dev)
    ldc = _require_matrix_out(out, a.outer, b.outer, out_dtype, dev)
    ca, cb = a._c(), b._c()
    with torch.cuda.device(dev):
        _check(lib().mxfp8_gemm(ctypes.byref(ca), ctypes.byref(cb), out.data_ptr(), code, ldc,
                                _stream_handle(stream, dev)), "mxfp8_gemm")
    return out


# ----------------------------------------------------------------------------
# The operators around the 4-bit linear layer.  Their inputs are matrices with
# unit column stride and any row stride of at least their width.  Outputs and
# scratch are allocated for the stream the call runs on, so memory freed by
# another stream's unfinished work is not reused.
# ----------------------------------------------------------------------------

_here = contextlib.nullcontext()
_current_device = torch.cuda.current_device


def _on(device: torch.device, stream):
    """The context that makes `device` and `stream` current; nothing to do
    (and nothing to pay) where they are already."""
    if stream is not None:
        if stream.device != device:
            raise NVFP4Error(f"stream of {stream.device}, tensors on {device}")
        return torch.cuda.stream(stream)
    return _here if _current_device() == device.index else torch.cuda.device(device)


def _require_matrix(t: torch.Tensor, name: str, device: torch.device | None = None, shape=None) -> int:
    """A [rows, cols] GPU matrix with unit column stride and rows that do not
    overlap; returns its leading dimension."""
    if not isinstance(t, torch.Tensor):
        raise NVFP4Error(f"{name} must be a tensor")
    _require_device(t, name)
    if device is not None and t.device != device:
        raise NVFP4Error(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 2:
        raise NVFP4Error(f"{name} must be a 2-D tensor, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise NVFP4Error(f"{name} must have shape {shape}, got {(rows, cols)}")
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise NVFP4Error(f"{name} must be row-major (unit column stride)")
    if rows <= 1:
        return max(cols, 1)
    if s0 < cols:
        raise NVFP4Error(f"{name}: rows overlap (row stride < columns)")
    return s0


def _param(t, name: str, cols: int, device: torch.device):
    """A parameter vector or None: (pointer, dtype code)."""
    if t is None:
        return None, F32
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.shape[0] != cols:
        raise NVFP4Error(f"{name} must be a vector of {cols} elements")
    return _vector(t, name, t.dtype, cols, device), _dtype_code(t)


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without building a Stream object (2.5 us less
# of the 11 that a small call costs), where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_handle(device: torch.device) -> int:
    """The handle of `device`'s current stream (the one _on made current)."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return int(torch.cuda.current_stream(device).cuda_stream)


def nvfp4_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     eps: float = 1e-5, out_dtype=None, amax: bool = False, out: torch.Tensor | None = None,
                     stream=None):
    """Layer norm of the rows of x [rows, cols] (f32/bf16): (y, mean, rstd),
    y in `out_dtype` (x's by default), mean and rstd f32 [rows].  With amax,
    (y, mean, rstd, amax): the f32 [1] maximum of |y| that
    nvfp4_quantize_amax takes on axis 1 (see include/nvfp4.h)."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    rows, cols = x.shape
    out_dtype = x.dtype if out_dtype is None else out_dtype
    ycode = _out_code(out_dtype)
    wp, wcode = _param(weight, "weight", cols, dev)
    bp, bcode = _param(bias, "bias", cols, dev)
    if wp is None:
        wcode = bcode
    elif bp is not None and bcode != wcode:
        raise NVFP4Error("weight and bias must have the same dtype")
    with _on(dev, stream):
        if out is None:
            y, ldy = torch.empty((rows, cols), dtype=out_dtype, device=dev), max(cols, 1)
        else:
            y, ldy = out, _require_matrix_out(out, rows, cols, out_dtype, dev)
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        top, ws, need = None, None, 0
        if amax:
            top = torch.empty(1, dtype=torch.float32, device=dev)
            need = lib().nvfp4_layer_norm_workspace_bytes(rows, cols)
            if need > 0:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _check(lib().nvfp4_layer_norm(x.data_ptr(), _dtype_code(x), rows, cols, ldx, wp, bp, wcode, eps, y.data_ptr(),
                                      ycode, ldy, mean.data_ptr(), rstd.data_ptr(), _ptr(top), _ptr(ws), need,
                                      _current_handle(dev)), "nvfp4_layer_norm")
    return (y, mean, rstd, top) if amax else (y, mean, rstd)


def nvfp4_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                              weight: torch.Tensor | None = None, grad_dtype=torch.float32, stream=None):
    """The gradients of nvfp4_layer_norm: (dx in x's dtype, dweight, dbias),
    the latter [cols] in `grad_dtype`."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    rows, cols = x.shape
    lddy = _require_matrix(dy, "dy", dev, (rows, cols))
    mp = _vector(mean, "mean", torch.float32, rows, dev)
    rp = _vector(rstd, "rstd", torch.float32, rows, dev)
    wp, wcode = _param(weight, "weight", cols, dev)
    gcode = _out_code(grad_dtype)
    need = lib().nvfp4_layer_norm_backward_workspace_bytes(rows, cols)
    if need < 0:
        _check(need, "nvfp4_layer_norm_backward")
    with _on(dev, stream):
        dx = x.new_empty((rows, cols))
        dweight = torch.empty(cols, dtype=grad_dtype, device=dev)
        dbias = torch.empty(cols, dtype=grad_dtype, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
        _check(lib().nvfp4_layer_norm_backward(dy.data_ptr(), _dtype_code(dy), lddy, x.data_ptr(), _dtype_code(x),
                                               rows, cols, ldx, mp, rp, wp, wcode,
                                               dx.data_ptr(), cols, dweight.data_ptr(), dbias.data_ptr(), gcode,
                                               _ptr(ws), need, _current_handle(dev)),
               "nvfp4_layer_norm_backward")
    return dx, dweight, dbias


def _rms_args(x, weight, residual, residual_out):
    """Checks what the two RMS norm calls share; returns (x's device, h or
    None, the leading C arguments up to the weight's dtype, h's place in
    them).  h is made by the caller's stream where it is not given."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    rows, cols = x.shape
    wp, wcode = _param(weight, "weight", cols, dev)
    if residual is None:
        if residual_out is not None:
            raise NVFP4Error("residual_out needs a residual")
        return dev, None, [x.data_ptr(), _dtype_code(x), rows, cols, ldx, None, F32, max(cols, 1), None, max(cols, 1),
                           wp, wcode]
    ldr = _require_matrix(residual, "residual", dev, (rows, cols))
    rcode = _dtype_code(residual)
    if residual_out is None:
        h, ldh = residual.new_empty((rows, cols)), max(cols, 1)
    else:
        h, ldh = residual_out, _require_matrix_out(residual_out, rows, cols, residual.dtype, dev)
    return dev, h, [x.data_ptr(), _dtype_code(x), rows, cols, ldx, residual.data_ptr(), rcode, ldr, h.data_ptr(), ldh,
                    wp, wcode]


def _stream_device(x, stream):
    """_on for the device of an input that is yet to be checked."""
    return _on(x.device, stream) if isinstance(x, torch.Tensor) and x.is_cuda else _here


def nvfp4_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, out_dtype=None, out: torch.Tensor | None = None,
                   residual_out: torch.Tensor | None = None, stream=None):
    """RMS norm of the rows of x [rows, cols] (f32/bf16), or of the sum
    h = x + residual: (y, rstd), with a residual (y, rstd, h).  y in
    `out_dtype` (x's by default), rstd f32 [rows], h in the residual's dtype,
    new or in `residual_out`, which may be the residual (see include/nvfp4.h)."""
    with _stream_device(x, stream):
        dev, h, args = _rms_args(x, weight, residual, residual_out)
        rows, cols = x.shape
        out_dtype = x.dtype if out_dtype is None else out_dtype
        ycode = _out_code(out_dtype)
        if out is None:
            y, ldy = torch.empty((rows, cols), dtype=out_dtype, device=dev), max(cols, 1)
        else:
            y, ldy = out, _require_matrix_out(out, rows, cols, out_dtype, dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        _check(lib().nvfp4_rms_norm(*args, eps, y.data_ptr(), ycode, ldy, rstd.data_ptr(), _current_handle(dev)),
               "nvfp4_rms_norm")
    return (y, rstd) if h is None else (y, rstd, h)


def mxfp8_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, out: "MXFP8Tensor | None" = None, residual_out: torch.Tensor | None = None,
                   stream=None):
    """nvfp4_rms_norm with y in MXFP8 on axis 1 (cols a multiple of 32)."""
    with _stream_device(x, stream):
        dev, h, args = _rms_args(x, weight, residual, residual_out)
        rows, cols = x.shape
        if cols % 32:
            raise NVFP4Error(f"MXFP8 needs a multiple of 32 columns, got {cols}")
        if out is None:
            out = MXFP8Tensor.empty(rows, cols, device=dev)
        _same_device(out, x)
        ct = out._c()
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        _check(lib().mxfp8_rms_norm(*args, eps, ctypes.byref(ct), rstd.data_ptr(), _current_handle(dev)),
               "mxfp8_rms_norm")
    return (out, rstd) if h is None else (out, rstd, h)


def nvfp4_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor | None = None,
                            dh: torch.Tensor | None = None, grad_dtype=torch.float32, stream=None):
    """The gradients of nvfp4_rms_norm: (dx in h's dtype, dweight [cols] in
    `grad_dtype`).  h is what was normed (x itself without a residual), dh the
    gradient that reaches it from the residual stream; dx is the gradient of
    x and of the residual alike."""
    ldh = _require_matrix(h, "h")
    dev = h.device
    rows, cols = h.shape
    lddy = _require_matrix(dy, "dy", dev, (rows, cols))
    rp = _vector(rstd, "rstd", torch.float32, rows, dev)
    wp, wcode = _param(weight, "weight", cols, dev)
    lddh = max(cols, 1)
    if dh is not None:
        lddh = _require_matrix(dh, "dh", dev, (rows, cols))
        if dh.dtype != h.dtype:
            raise NVFP4Error(f"dh must have h's dtype {h.dtype}, got {dh.dtype}")
    gcode = _out_code(grad_dtype)
    need = lib().nvfp4_rms_norm_backward_workspace_bytes(rows, cols)
    if need < 0:
        _check(need, "nvfp4_rms_norm_backward")
    with _on(dev, stream):
        dx = h.new_empty((rows, cols))
        dweight = torch.empty(cols, dtype=grad_dtype, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
        _check(lib().nvfp4_rms_norm_backward(dy.data_ptr(), _dtype_code(dy), lddy, h.data_ptr(), _dtype_code(h), rows,
                                             cols, ldh, rp, wp, wcode, _ptr(dh), lddh, dx.data_ptr(), max(cols, 1),
                                             dweight.data_ptr(), gcode, _ptr(ws), need, _current_handle(dev)),
               "nvfp4_rms_norm_backward")
    return dx, dweight


def _matvec(fn, what, w, x, out_dtype, out, stream):
    ldx = _require_matrix(x, "x")
    dev = x.device
    if w.device != dev:
        raise NVFP4Error(f"weights on {w.device}, x on {dev}")
    tokens, k = x.shape
    if k != w.k:
        raise NVFP4Error(f"x must have {w.k} columns, got {k}")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    code = _out_code(out_dtype)
    cw, xcode = w._c(), _dtype_code(x)
    need = lib().nvfp4_matvec_workspace_bytes(w.outer, k, tokens, xcode)
    if need < 0:
        _check(need, what)
    with _on(dev, stream):
        y = torch.empty((tokens, w.outer), dtype=out_dtype, device=dev) if out is None else out
        ldy = _require_matrix_out(y, tokens, w.outer, out_dtype, dev) if out is not None else max(w.outer, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(fn(ctypes.byref(cw), x.data_ptr(), xcode, tokens, ldx, y.data_ptr(), code, ldy, _ptr(ws), need,
                  _current_handle(dev)), what)
    return y


def nvfp4_matvec(w: NVFP4Tensor, x: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y [tokens, N] = x . W^T for unquantized x [tokens, K] (f32/bf16, made
    for 1 to 16 tokens) and NVFP4 weights W [N, K]; y in `out_dtype` (x's by
    default)."""
    return _matvec(lib().nvfp4_matvec, "nvfp4_matvec", w, x, out_dtype, out, stream)


def mxfp4_matvec(w: MXFP4Tensor, x: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """nvfp4_matvec with MXFP4 weights."""
    return _matvec(lib().mxfp4_matvec, "mxfp4_matvec", w, x, out_dtype, out, stream)


def _group_args(offsets, device):
    """(address, index bits, number of groups) of a vector of group offsets."""
    if not isinstance(offsets, torch.Tensor) or offsets.dtype not in (torch.int32, torch.int64):
        raise NVFP4Error("offsets must be an int32 or int64 tensor")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise NVFP4Error(f"offsets must be a vector of the groups' ends behind a first start, got "
                         f"{tuple(offsets.shape)}")
    groups = offsets.shape[0] - 1
    return (_vector(offsets, "offsets", offsets.dtype, groups + 1, device), 32 if offsets.dtype is torch.int32 else 64,
            groups)


def _grouped_matmul(fn, what, w, x, offsets, out_dtype, transposed, out, stream):
    ldx = _require_matrix(x, "x")
    dev = x.device
    if w.device != dev:
        raise NVFP4Error(f"weights on {w.device}, x on {dev}")
    op, bits, experts = _group_args(offsets, dev)
    rows, k = x.shape
    stacked = w.k if transposed else w.outer
    if stacked % experts:
        raise NVFP4Error(f"a stack of {stacked} {'columns' if transposed else 'rows'} is not one of {experts} experts")
    n, want = (w.outer, w.k // experts) if transposed else (w.outer // experts, w.k)
    if k != want:
        raise NVFP4Error(f"x must have {want} columns, got {k}")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    code = _out_code(out_dtype)
    cw, xcode = w._c(), _dtype_code(x)
    need = lib().nvfp4_grouped_matmul_workspace_bytes(experts, n, k, rows, xcode)
    if need < 0:
        _check(need, what)
    with _on(dev, stream):
        y = torch.empty((rows, n), dtype=out_dtype, device=dev) if out is None else out
        ldy = max(n, 1) if out is None else _require_matrix_out(y, rows, n, out_dtype, dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(fn(ctypes.byref(cw), int(bool(transposed)), x.data_ptr(), xcode, rows, ldx, op, bits, experts,
                  y.data_ptr(), code, ldy, int(out is None), _ptr(ws), need, _current_handle(dev)), what)
    return y


def nvfp4_grouped_matmul(w: NVFP4Tensor, x: torch.Tensor, offsets: torch.Tensor, out_dtype=None,
                         transposed: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [rows, N] = x . W_e^T for the rows offsets[e] .. offsets[e + 1] - 1 of
    unquantized x [rows, K] (f32/bf16) and each expert's NVFP4 weights W_e
    [N, K]: w is [experts * N, K], or with `transposed` [N, experts * K] (the
    stack [experts * K, N] quantized on axis 0, for the data gradient).
    offsets: int32/int64 [experts + 1] on the GPU, not decreasing.  Rows of no
    group are zeros, and left as they are in a given `out`."""
    return _grouped_matmul(lib().nvfp4_grouped_matmul, "nvfp4_grouped_matmul", w, x, offsets, out_dtype, transposed,
                           out, stream)


def mxfp4_grouped_matmul(w: MXFP4Tensor, x: torch.Tensor, offsets: torch.Tensor, out_dtype=None,
                         transposed: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_grouped_matmul with MXFP4 weights."""
    return _grouped_matmul(lib().mxfp4_grouped_matmul, "mxfp4_grouped_matmul", w, x, offsets, out_dtype, transposed,
                           out, stream)


def nvfp4_grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, grad_dtype=torch.float32,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient [experts, N, K] of a stack of experts' weights in
    `grad_dtype`: the sum of dy[t]^T x[t] over each group's rows of dy
    [rows, N] and x [rows, K]."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    rows, k = x.shape
    lddy = _require_matrix(dy, "dy", dev)
    if dy.shape[0] != rows:
        raise NVFP4Error(f"dy must have {rows} rows, got {dy.shape[0]}")
    n = dy.shape[1]
    op, bits, experts = _group_args(offsets, dev)
    code = _out_code(grad_dtype)
    need = lib().nvfp4_grouped_wgrad_workspace_bytes(experts, n, k, rows, _dtype_code(dy), _dtype_code(x))
    if need < 0:
        _check(need, "nvfp4_grouped_wgrad")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((experts, n, k), dtype=grad_dtype, device=dev)
        elif not isinstance(out, torch.Tensor) or tuple(out.shape) != (experts, n, k):
            raise NVFP4Error(f"out must have shape ({experts}, {n}, {k})")
        dp = _vector(out, "out", grad_dtype, experts * n * k, dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(lib().nvfp4_grouped_wgrad(dy.data_ptr(), _dtype_code(dy), lddy, x.data_ptr(), _dtype_code(x), ldx, rows, n,
                                         k, op, bits, experts, dp, code, _ptr(ws), need, _current_handle(dev)),
               "nvfp4_grouped_wgrad")
    return out


def _adapter_args(a, b, offsets, index, scale, device):
    """Checks the adapters and their segments; returns (n, k, rank, the C
    arguments from a to segments)."""
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise NVFP4Error(f"{name} must be a 3-D tensor")
    adapters, rank, k = a.shape
    n = b.shape[1]
    if b.shape[0] != adapters or b.shape[2] != rank:
        raise NVFP4Error(f"b must have shape ({adapters}, N, {rank}), got {tuple(b.shape)}")
    if b.dtype != a.dtype:
        raise NVFP4Error(f"a and b must have the same dtype, got {a.dtype} and {b.dtype}")
    code = _dtype_code(a)
    op, bits, segments = _group_args(offsets, device)
    if not isinstance(index, torch.Tensor) or index.dtype != offsets.dtype or tuple(index.shape) != (segments,):
        raise NVFP4Error(f"index must be a vector of {segments} elements of offsets' dtype {offsets.dtype}")
    sp = None if scale is None else _vector(scale, "scale", torch.float32, adapters, device)
    return n, k, rank, [_vector(a, "a", a.dtype, adapters * rank * k, device),
                        _vector(b, "b", b.dtype, adapters * n * rank, device), code, adapters, rank, n, sp, op,
                        _vector(index, "index", index.dtype, segments, device), bits, segments]


def _base_args(base, rows, cols, device):
    """(address or None, dtype code, leading dimension)."""
    if base is None:
        return None, F32, max(cols, 1)
    ld = _require_matrix(base, "base", device, (rows, cols))
    return base.data_ptr(), _dtype_code(base), ld


def nvfp4_adapters(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, index: torch.Tensor,
                   scale: torch.Tensor | None = None, base: torch.Tensor | None = None, out_dtype=None,
                   out: torch.Tensor | None = None, stream=None):
    """Low-rank adapters beside a shared projection: (y, u) with u = A x f32
    [rows, rank] and y = base + scale B u, for the rows offsets[i] ..
    offsets[i + 1] - 1 of x [rows, K] (f32/bf16) and adapter index[i] (-1 =
    none: y = base, u = 0).  a [adapters, rank, K], b [adapters, N, rank]
    (f32/bf16), scale f32 [adapters]; base [rows, N], the shared projection's
    result, or None (0); offsets and index int32/int64 on the GPU.  y in
    `out_dtype` (base's by default, else x's), new or in `out`, which may be
    base (see include/nvfp4.h)."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    n, k, rank, weights = _adapter_args(a, b, offsets, index, scale, dev)
    rows = x.shape[0]
    if x.shape[1] != k:
        raise NVFP4Error(f"x must have {k} columns, got {x.shape[1]}")
    bp, bcode, ldb = _base_args(base, rows, n, dev)
    if out_dtype is None:
        out_dtype = (x if base is None else base).dtype
    ycode = _out_code(out_dtype)
    with _on(dev, stream):
        y = torch.empty((rows, n), dtype=out_dtype, device=dev) if out is None else out
        ldy = max(n, 1) if out is None else _require_matrix_out(y, rows, n, out_dtype, dev)
        u = torch.empty((rows, rank), dtype=torch.float32, device=dev)
        _check(lib().nvfp4_adapters(x.data_ptr(), _dtype_code(x), rows, k, ldx, *weights, bp, bcode, ldb, y.data_ptr(),
                                    ycode, ldy, u.data_ptr(), _current_handle(dev)), "nvfp4_adapters")
    return y, u


def nvfp4_adapters_backward(dy: torch.Tensor, x: torch.Tensor, u: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                            offsets: torch.Tensor, index: torch.Tensor, scale: torch.Tensor | None = None,
                            base: torch.Tensor | None = None, grad_dtype=torch.float32,
                            out: torch.Tensor | None = None, stream=None):
    """The gradients of nvfp4_adapters: (dx, da, db).  dx [rows, K] in x's
    dtype is base (the shared projection's own gradient, or 0) plus the
    adapters' part, new or in `out`, which may be base; da and db in
    `grad_dtype`, of a's and b's shapes."""
    ldx = _require_matrix(x, "x")
    dev = x.device
    n, k, rank, weights = _adapter_args(a, b, offsets, index, scale, dev)
    rows = x.shape[0]
    if x.shape[1] != k:
        raise NVFP4Error(f"x must have {k} columns, got {x.shape[1]}")
    lddy = _require_matrix(dy, "dy", dev, (rows, n))
    up = _vector(u, "u", torch.float32, rows * rank, dev)
    bp, bcode, ldb = _base_args(base, rows, k, dev)
    gcode = _out_code(grad_dtype)
    need = lib().nvfp4_adapters_backward_workspace_bytes(rows, n, k, rank, a.shape[0], index.shape[0], weights[2])
    if need < 0:
        _check(need, "nvfp4_adapters_backward")
    with _on(dev, stream):
        dx = x.new_empty((rows, k)) if out is None else out
        lddx = max(k, 1) if out is None else _require_matrix_out(dx, rows, k, x.dtype, dev)
        da = torch.empty(a.shape, dtype=grad_dtype, device=dev)
        db = torch.empty(b.shape, dtype=grad_dtype, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check(lib().nvfp4_adapters_backward(dy.data_ptr(), _dtype_code(dy), lddy, x.data_ptr(), _dtype_code(x), rows, k,
                                             ldx, up, *weights, bp, bcode, ldb, dx.data_ptr(), _dtype_code(dx), lddx,
                                             da.data_ptr(), db.data_ptr(), gcode, _ptr(ws), need, _current_handle(dev)),
               "nvfp4_adapters_backward")
    return dx, da, db


def _distill_args(logits, indices, teacher, temperature):
    """Checks the inputs that the distillation calls share; returns their
    leading C arguments."""
    ldz = _require_matrix(logits, "logits")
    dev = logits.device
    tokens, vocab = logits.shape
    if not isinstance(indices, torch.Tensor) or indices.dtype not in (torch.int32, torch.int64):
        raise NVFP4Error("indices must be an int32 or int64 tensor")
    if indices.dim() != 2 or indices.shape[0] != tokens:
        raise NVFP4Error(f"indices must have shape ({tokens}, top), got {tuple(indices.shape)}")
    if not isinstance(teacher, torch.Tensor) or teacher.shape != indices.shape:
        raise NVFP4Error("teacher must be a tensor of indices' shape")
    top = indices.shape[1]
    return (logits.data_ptr(), _dtype_code(logits), tokens, vocab, ldz,
            _vector(indices, "indices", indices.dtype, tokens * top, dev), 32 if indices.dtype is torch.int32 else 64,
            _vector(teacher, "teacher", teacher.dtype, tokens * top, dev), _dtype_code(teacher), top, temperature)


def _distill_workspace(tokens: int, vocab: int, device):
    """(tensor or None, address or None, size) of the scratch memory."""
    need = lib().nvfp4_distill_topk_workspace_bytes(tokens, vocab)
    if need < 0:
        _check(need, "nvfp4_distill_topk")
    if need == 0:
        return None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), need


def nvfp4_distill_topk(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                       temperature: float = 1.0, stream=None):
    """The distillation loss of logits [tokens, vocab] (f32/bf16) against a
    teacher's best logits [tokens, top] at `indices` (-1 = no entry):
    (loss, lse), f32 [tokens] (see include/nvfp4.h)."""
    args = _distill_args(logits, indices, teacher, temperature)
    dev = logits.device
    tokens, vocab = logits.shape
    with _on(dev, stream):
        loss = torch.empty(tokens, dtype=torch.float32, device=dev)
        lse = torch.empty(tokens, dtype=torch.float32, device=dev)
        ws, wsp, need = _distill_workspace(tokens, vocab, dev)
        _check(lib().nvfp4_distill_topk(*args, loss.data_ptr(), lse.data_ptr(), wsp, need,
                                        _current_handle(dev)), "nvfp4_distill_topk")
    return loss, lse


def nvfp4_distill_topk_backward(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                                lse: torch.Tensor, dloss: torch.Tensor, temperature: float = 1.0,
                                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of sum_t dloss_t loss_t with respect to the logits, in
    their dtype, from the forward call's lse."""
    args = _distill_args(logits, indices, teacher, temperature)
    dev = logits.device
    tokens, vocab = logits.shape
    lp = _vector(lse, "lse", torch.float32, tokens, dev)
    gp = _vector(dloss, "dloss", torch.float32, tokens, dev)
    with _on(dev, stream):
        dz = logits.new_empty((tokens, vocab)) if out is None else out
        ldd = _require_matrix_out(dz, tokens, vocab, logits.dtype, dev) if out is not None else max(vocab, 1)
        _check(lib().nvfp4_distill_topk_backward(*args, lp, gp, dz.data_ptr(), ldd,
                                                 _current_handle(dev)), "nvfp4_distill_topk_backward")
    return dz


def nvfp4_distill_topk_step(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                            weight: torch.Tensor, temperature: float = 1.0, out: torch.Tensor | None = None,
                            stream=None):
    """Loss and gradient in one call: (loss, lse, dlogits), dlogits being the
    gradient of sum_t weight_t loss_t (weight f32 [tokens])."""
    args = _distill_args(logits, indices, teacher, temperature)
    dev = logits.device
    tokens, vocab = logits.shape
    gp = _vector(weight, "weight", torch.float32, tokens, dev)
    with _on(dev, stream):
        dz = logits.new_empty((tokens, vocab)) if out is None else out
        ldd = _require_matrix_out(dz, tokens, vocab, logits.dtype, dev) if out is not None else max(vocab, 1)
        loss = torch.empty(tokens, dtype=torch.float32, device=dev)
        lse = torch.empty(tokens, dtype=torch.float32, device=dev)
        ws, wsp, need = _distill_workspace(tokens, vocab, dev)
        _check(lib().nvfp4_distill_topk_step(*args, gp, loss.data_ptr(), lse.data_ptr(), dz.data_ptr(),
                                             ldd, wsp, need, _current_handle(dev)),
               "nvfp4_distill_topk_step")
    return loss, lse, dz
