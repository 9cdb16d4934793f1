"""The operators of a feed-forward block (``include/gemm_ffn.h``): root-mean-square norm with
the residual's addition, conversion to 8 bits (e4m3) with scales, the product of 8-bit matrices,
and the gated product with its gradients.

As in the rest of the binding, a plan class owns a C handle, its methods take torch tensors
(device memory) and a stream, and everything is computed by the library's CUDA kernels.  8-bit
matrices are ``torch.float8_e4m3fn`` tensors; their scales are fp32 matrices, one value for each
128 elements of a row ("row") or for each 128 x 128 elements ("square").  A tensor of another
shape, type or device than the call's raises ``GemmError`` before anything is queued.

    with RmsNormPlan(max_rows, cols, "bf16", weight="f32") as norm:
        norm.forward(x, gamma, y, rstd, residual=r, total=t)
        norm.backward(t, gamma, rstd, dy, dx, dgamma, dtotal=dt)
        norm.forward_fp8(x, gamma, q, scales, residual=r, total=t)
    fp8_quantize(w, wq, w_scales, block="square")
"""
from __future__ import annotations

import ctypes

from . import GemmError, _check, _stream, library
from .train import _INVALID_ARG, _UNSUPPORTED, GEMM_ELEM_F32, _elem, _elem_of, _matrix, _on_device, _Plan, _torch_types, _vector

__all__ = ["GEMM_SCALE_ROW", "GEMM_SCALE_SQUARE", "SCALES", "RmsNormPlan", "fp8_quantize"]

GEMM_SCALE_ROW, GEMM_SCALE_SQUARE = 0, 1
SCALES = {"row": GEMM_SCALE_ROW, "square": GEMM_SCALE_SQUARE}
GROUP = 128                 # elements that share a scale


def signatures():
    """(argument types, result type) of the C functions of gemm_ffn.h."""
    i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    vpp = ctypes.POINTER(ctypes.c_void_p)
    return {
        "gemm_rms_plan_create": ([i64, i64, i32, i32, vpp], i32),
        "gemm_rms_forward": ([vp, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, vp], i32),
        "gemm_rms_forward_fp8": ([vp, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp, vp], i32),
        "gemm_rms_backward": ([vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp], i32),
        "gemm_rms_plan_destroy": ([vp], i32),
        "gemm_fp8_quantize": ([i64, i64, i32, vp, i64, i32, i32, vp, i64, vp, i64, vp], i32),
    }


def _groups(n: int) -> int:
    return -(-n // GROUP)


def _scale_kind(kind) -> int:
    if isinstance(kind, str):
        if kind not in SCALES:
            raise GemmError(_UNSUPPORTED, "scales %r" % kind)
        return SCALES[kind]
    return int(kind)


def _bytes_matrix(t, rows, cols, what):
    """(address, row stride) of a rows x cols e4m3 matrix with contiguous rows."""
    import torch
    if t.dtype != torch.float8_e4m3fn:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    return _matrix(t, rows, cols, None, what)


def _optional(t, rows, cols, elem, what):
    return (None, 0) if t is None else _matrix(t, rows, cols, elem, what)


class RmsNormPlan(_Plan):
    """Root-mean-square norm over rows of `cols` elements, for up to `max_rows` rows a call."""

    _destroy = "gemm_rms_plan_destroy"

    def __init__(self, max_rows: int, cols: int, dtype="f16", weight=None):
        self.max_rows, self.cols = max_rows, cols
        self._elem = _elem(dtype)
        self._weight = self._elem if weight is None else _elem(weight)
        self._create("gemm_rms_plan_create", max_rows, cols, self._elem, self._weight)

    def _inputs(self, x, gamma, residual, total, eps):
        rows, cols = x.shape[0], self.cols
        return (rows, *_matrix(x, rows, cols, self._elem, "x"), *_optional(residual, rows, cols, self._elem, "residual"),
                _vector(gamma, cols, self._weight, "gamma", True), eps,
                *_optional(total, rows, cols, self._elem, "total"))

    def forward(self, x, gamma, y, rstd=None, residual=None, total=None, eps: float = 1e-5, stream=None) -> None:
        """y = t * rstd * gamma of t = x + residual; total and rstd (fp32) are kept for backward."""
        args = self._inputs(x, gamma, residual, total, eps)
        rows = args[0]
        _check(library().gemm_rms_forward(
            self.handle, *args, *_matrix(y, rows, self.cols, self._elem, "y"),
            _vector(rstd, rows, GEMM_ELEM_F32, "rstd", True), _stream(stream)), "gemm_rms_forward")

    def forward_fp8(self, x, gamma, q, scales, rstd=None, residual=None, total=None, eps: float = 1e-5,
                    stream=None) -> None:
        """As forward, with y as e4m3 numbers and their scales by rows."""
        args = self._inputs(x, gamma, residual, total, eps)
        rows = args[0]
        _check(library().gemm_rms_forward_fp8(
            self.handle, *args, *_bytes_matrix(q, rows, self.cols, "q"),
            *_matrix(scales, rows, _groups(self.cols), GEMM_ELEM_F32, "scales"),
            _vector(rstd, rows, GEMM_ELEM_F32, "rstd", True), _stream(stream)), "gemm_rms_forward_fp8")

    def backward(self, total, gamma, rstd, dy, dx=None, dgamma=None, dtotal=None, stream=None) -> None:
        """Gradients of x (and of the residual) and of gamma, each optional, from dy and from dtotal,
        the gradient that reaches the sum on its other way."""
        rows, cols = total.shape[0], self.cols
        _check(library().gemm_rms_backward(
            self.handle, rows, *_matrix(total, rows, cols, self._elem, "total"),
            _vector(gamma, cols, self._weight, "gamma", True), _vector(rstd, rows, GEMM_ELEM_F32, "rstd"),
            *_matrix(dy, rows, cols, self._elem, "dy"), *_optional(dtotal, rows, cols, self._elem, "dtotal"),
            *_optional(dx, rows, cols, self._elem, "dx"), _vector(dgamma, cols, self._weight, "dgamma", True),
            _stream(stream)), "gemm_rms_backward")


def fp8_quantize(x, q, scales, block="row", transpose: bool = False, stream=None) -> None:
    """x as e4m3 numbers `q` with fp32 `scales` for each 128 elements of a row ("row") or each
    128 x 128 elements ("square"); of its transpose where `transpose`."""
    _torch_types()
    kind = _scale_kind(block)
    if not _on_device(x) or x.dim() != 2:
        raise GemmError(_INVALID_ARG, "x: a matrix on the current device is needed")
    rows, cols = x.shape
    out = (cols, rows) if transpose else (rows, cols)
    px, ldx = _matrix(x, rows, cols, None, "x")
    pq, ldq = _bytes_matrix(q, *out, "q")
    ps, lds = _matrix(scales, _groups(out[0]) if kind == GEMM_SCALE_SQUARE else out[0], _groups(out[1]), GEMM_ELEM_F32,
                      "scales")
    _check(library().gemm_fp8_quantize(rows, cols, _elem_of(x, "x"), px, ldx, kind, 1 if transpose else 0, pq, ldq, ps, lds,
                                       _stream(stream)), "gemm_fp8_quantize")
