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
    with Fp8Plan(M, N, K, "bf16") as product:
        product.run(q, scales, wq, w_scales, c)
    with GatedPlan(M, F, K, "bf16", act="silu") as gated:           # w: 2F x K, the gate's rows first
        gated.forward(y, w, h, gate_up=gu)
        gated.backward(y, w, gu, dh, dgu, dy, dw)
"""
from __future__ import annotations

import ctypes

from . import ACTIVATIONS, GemmError, _check, _stream, library
from . import train
from .train import _INVALID_ARG, _UNSUPPORTED, GEMM_ELEM_F32, _elem, _elem_of, _on_device, _Plan, _torch_types, _vector

__all__ = ["GEMM_SCALE_ROW", "GEMM_SCALE_SQUARE", "SCALES", "RmsNormPlan", "fp8_quantize", "Fp8Plan", "GatedPlan"]

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
        "gemm_fp8_plan_create": ([i64, i64, i64, i32, i32, vpp], i32),
        "gemm_fp8_run": ([vp, vp, vp, vp, vp, vp, vp], i32),
        "gemm_gated_plan_create": ([i64, i64, i64, i32, i32, vpp], i32),
        "gemm_gated_forward": ([vp, vp, vp, vp, vp, vp], i32),
        "gemm_gated_backward": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        **{"gemm_%s_plan_%s" % (kind, call): ([vp, *more], i32) for kind in ("fp8", "gated")
           for call, more in (("set_timeout", [ctypes.c_uint64]), ("set_wait_test", [ctypes.c_uint32]), ("check", [vp]),
                              ("destroy", []))},
    }


# calls that the C entry points know, by their numbers there
_RMS_FORWARD, _RMS_FORWARD_FP8, _RMS_BACKWARD, _FP8_RUN, _GATED_FORWARD, _GATED_BACKWARD, _QUANTIZE = range(7, 14)


class _FfnPlan(_Plan):
    """A plan whose calls have C entry points (``_enter``), of which ``_drop`` forgets all."""

    def _enter(self, kind, name, elem, weight, cols, rows=0, *more):
        import torch
        return self._entry(kind, name, elem, weight, cols, rows, *more, extra_types=(torch.float8_e4m3fn,))

    def _drop(self):
        for name in [n for n in vars(self) if n.startswith("_enter_")]:
            setattr(self, name, None)


def _groups(n: int) -> int:
    return -(-n // GROUP)


def _scale_kind(kind) -> int:
    if isinstance(kind, str):
        if kind not in SCALES:
            raise GemmError(_UNSUPPORTED, "scales %r" % kind)
        return SCALES[kind]
    return int(kind)


def _needed(t, what):
    if t is None:
        raise GemmError(_INVALID_ARG, "%s: a tensor is needed" % what)
    return t


def _rows(t, what) -> int:
    """The rows of a call's first matrix."""
    if _needed(t, what).dim() != 2:
        raise GemmError(_INVALID_ARG, "%s: a matrix is needed" % what)
    return t.shape[0]


def _matrix(t, rows, cols, elem, what):
    return train._matrix(_needed(t, what), rows, cols, elem, what)


def _bytes_matrix(t, rows, cols, what):
    """(address, row stride) of a rows x cols e4m3 matrix with contiguous rows."""
    import torch
    if _needed(t, what).dtype != torch.float8_e4m3fn:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    return _matrix(t, rows, cols, None, what)


def _optional(t, rows, cols, elem, what):
    return (None, 0) if t is None else _matrix(t, rows, cols, elem, what)


def _whole(t, rows, cols, elem, what):
    """Address of a contiguous rows x cols matrix."""
    address, ld = _matrix(t, rows, cols, elem, what)
    if ld != cols and rows * cols > 0:
        raise GemmError(_INVALID_ARG, "%s: a contiguous matrix is needed" % what)
    return address


class _ProductPlan(_FfnPlan):
    """A plan of a product: its waits' limit, their test hook and their check (`_kind`: of its C functions)."""

    _kind = ""

    def _call(self, name, *args):
        name = "gemm_%s_plan_%s" % (self._kind, name)
        _check(getattr(library(), name)(self.handle, *args), name)

    def set_timeout(self, ns: int) -> None:
        """The limit of a wait in this plan's kernels, in nanoseconds (0: the default, 2e9)."""
        self._call("set_timeout", ns)

    def set_wait_test(self, extra_bytes: int) -> None:
        """Test hook: the ring's slots wait for bytes that do not come (0: off)."""
        self._call("set_wait_test", extra_bytes)

    def check(self, stream=None) -> None:
        """Synchronise `stream`; raise GemmError(GEMM_ERR_DEVICE_TIMEOUT) if a kernel gave up on a wait."""
        self._call("check", _stream(stream))


class RmsNormPlan(_FfnPlan):
    """Root-mean-square norm over rows of `cols` elements, for up to `max_rows` rows a call."""

    _destroy = "gemm_rms_plan_destroy"

    def __init__(self, max_rows: int, cols: int, dtype="f16", weight=None):
        self.max_rows, self.cols = max_rows, cols
        self._elem = _elem(dtype)
        self._weight = self._elem if weight is None else _elem(weight)
        self._create("gemm_rms_plan_create", max_rows, cols, self._elem, self._weight)
        self._enter_forward, self._enter_fp8, self._enter_backward = (
            self._enter(kind, name, self._elem, self._weight, cols)
            for kind, name in ((_RMS_FORWARD, "gemm_rms_forward"), (_RMS_FORWARD_FP8, "gemm_rms_forward_fp8"),
                               (_RMS_BACKWARD, "gemm_rms_backward")))

    def _inputs(self, x, gamma, residual, total, eps):
        rows, cols = _rows(x, "x"), self.cols
        return (rows, *_matrix(x, rows, cols, self._elem, "x"), *_optional(residual, rows, cols, self._elem, "residual"),
                _vector(gamma, cols, self._weight, "gamma", True), eps,
                *_optional(total, rows, cols, self._elem, "total"))

    def forward(self, x, gamma, y, rstd=None, residual=None, total=None, eps: float = 1e-5, stream=None) -> None:
        """y = t * rstd * gamma of t = x + residual; total and rstd (fp32) are kept for backward."""
        if self._taken(self._enter_forward, "gemm_rms_forward", (x, gamma, y, rstd, residual, total, eps, stream)):
            return
        args = self._inputs(x, gamma, residual, total, eps)
        rows = args[0]
        _check(library().gemm_rms_forward(
            self.handle, *args, *_matrix(y, rows, self.cols, self._elem, "y"),
            _vector(rstd, rows, GEMM_ELEM_F32, "rstd", True), _stream(stream)), "gemm_rms_forward")

    def forward_fp8(self, x, gamma, q, scales, rstd=None, residual=None, total=None, eps: float = 1e-5,
                    stream=None) -> None:
        """As forward, with y as e4m3 numbers and their scales by rows."""
        if self._taken(self._enter_fp8, "gemm_rms_forward_fp8",
                       (x, gamma, q, scales, rstd, residual, total, eps, stream)):
            return
        args = self._inputs(x, gamma, residual, total, eps)
        rows = args[0]
        _check(library().gemm_rms_forward_fp8(
            self.handle, *args, *_bytes_matrix(q, rows, self.cols, "q"),
            *_matrix(scales, rows, _groups(self.cols), GEMM_ELEM_F32, "scales"),
            _vector(rstd, rows, GEMM_ELEM_F32, "rstd", True), _stream(stream)), "gemm_rms_forward_fp8")

    def backward(self, total, gamma, rstd, dy, dx=None, dgamma=None, dtotal=None, stream=None) -> None:
        """Gradients of x (and of the residual) and of gamma, each optional, from dy and from dtotal,
        the gradient that reaches the sum on its other way."""
        if self._taken(self._enter_backward, "gemm_rms_backward", (total, gamma, rstd, dy, dx, dgamma, dtotal, stream)):
            return
        rows, cols = _rows(total, "total"), self.cols
        _check(library().gemm_rms_backward(
            self.handle, rows, *_matrix(total, rows, cols, self._elem, "total"),
            _vector(gamma, cols, self._weight, "gamma", True), _vector(rstd, rows, GEMM_ELEM_F32, "rstd"),
            *_matrix(dy, rows, cols, self._elem, "dy"), *_optional(dtotal, rows, cols, self._elem, "dtotal"),
            *_optional(dx, rows, cols, self._elem, "dx"), _vector(dgamma, cols, self._weight, "dgamma", True),
            _stream(stream)), "gemm_rms_backward")


_quantize = None            # the C entry point of fp8_quantize, where there is one device


def _quantize_entry():
    global _quantize
    if _quantize is None:
        import torch
        library()
        if not torch.cuda.is_available() or torch.cuda.device_count() != 1:
            return None
        call = _FfnPlan()
        call.handle = 0
        _quantize = call._enter(_QUANTIZE, "gemm_fp8_quantize", 0, 0, 0)
    return _quantize


def fp8_quantize(x, q, scales, block="row", transpose: bool = False, stream=None) -> None:
    """x as e4m3 numbers `q` with fp32 `scales` for each 128 elements of a row ("row") or each
    128 x 128 elements ("square"); of its transpose where `transpose`."""
    kind = _scale_kind(block)
    if _Plan._taken(_quantize_entry(), "gemm_fp8_quantize", (x, q, scales, kind, transpose, stream)):
        return
    _torch_types()
    if not _on_device(_needed(x, "x")) or x.dim() != 2:
        raise GemmError(_INVALID_ARG, "x: a matrix on the current device is needed")
    rows, cols = x.shape
    out = (cols, rows) if transpose else (rows, cols)
    px, ldx = _matrix(x, rows, cols, None, "x")
    pq, ldq = _bytes_matrix(q, *out, "q")
    ps, lds = _matrix(scales, _groups(out[0]) if kind == GEMM_SCALE_SQUARE else out[0], _groups(out[1]), GEMM_ELEM_F32,
                      "scales")
    _check(library().gemm_fp8_quantize(rows, cols, _elem_of(x, "x"), px, ldx, kind, 1 if transpose else 0, pq, ldq, ps, lds,
                                       _stream(stream)), "gemm_fp8_quantize")


class Fp8Plan(_ProductPlan):
    """C = A B^T of e4m3 matrices (A M x K, B N x K) with scales, C of `dtype` ("f16" or "bf16").  A's scales go
    by rows, B's by squares (`b_scales` "square") or by rows ("row").  K is a multiple of 16: a weight gradient over any
    other number of tokens takes matrices of the next one with zeros behind the tokens, q[:, :tokens] for fp8_quantize
    (their scales are as many)."""

    _destroy, _kind = "gemm_fp8_plan_destroy", "fp8"

    def __init__(self, M: int, N: int, K: int, dtype="bf16", b_scales="square"):
        self.M, self.N, self.K = M, N, K
        self._elem, self._scales = _elem(dtype), _scale_kind(b_scales)
        self._create("gemm_fp8_plan_create", M, N, K, self._elem, self._scales)
        self._enter_run = self._enter(_FP8_RUN, "gemm_fp8_run", self._elem, self._elem, N, M, K,
                                      self._scales == GEMM_SCALE_SQUARE)

    def run(self, A, a_scales, B, b_scales, C, stream=None) -> None:
        """C = A B^T.  All matrices contiguous."""
        if self._taken(self._enter_run, "gemm_fp8_run", (A, a_scales, B, b_scales, C, stream)):
            return
        M, N, K = self.M, self.N, self.K
        _bytes_matrix(A, M, K, "A")
        _bytes_matrix(B, N, K, "B")
        n = _groups(K)
        _check(library().gemm_fp8_run(
            self.handle, _whole(A, M, K, None, "A"), _whole(a_scales, M, n, GEMM_ELEM_F32, "a_scales"),
            _whole(B, N, K, None, "B"),
            _whole(b_scales, _groups(N) if self._scales == GEMM_SCALE_SQUARE else N, n, GEMM_ELEM_F32, "b_scales"),
            _whole(C, M, N, self._elem, "C"), _stream(stream)), "gemm_fp8_run")


class GatedPlan(_ProductPlan):
    """H = act(X Wg^T) * (X Wu^T) with X M x K, W = [Wg; Wu] 2F x K and H M x F, all of `dtype` ("f16" or "bf16");
    act: "silu", "gelu", "relu" or "none"."""

    _destroy, _kind = "gemm_gated_plan_destroy", "gated"

    def __init__(self, M: int, F: int, K: int, dtype="bf16", act="silu"):
        self.M, self.F, self.K = M, F, K
        self._elem = _elem(dtype)
        if isinstance(act, str) and act not in ACTIVATIONS:
            raise GemmError(_UNSUPPORTED, "activation %r" % act)
        self._create("gemm_gated_plan_create", M, F, K, self._elem, ACTIVATIONS[act] if isinstance(act, str) else int(act))
        self._enter_forward, self._enter_backward = (
            self._enter(kind, name, self._elem, self._elem, F, M, K)
            for kind, name in ((_GATED_FORWARD, "gemm_gated_forward"), (_GATED_BACKWARD, "gemm_gated_backward")))

    def _matrix(self, t, rows, cols, what, may_be_none=False):
        if t is None and may_be_none:
            return None
        return _whole(t, rows, cols, self._elem, what)

    def forward(self, X, W, H, gate_up=None, stream=None) -> None:
        """H; and both products side by side (M x 2F), for backward, where `gate_up` is given."""
        if self._taken(self._enter_forward, "gemm_gated_forward", (X, W, H, gate_up, stream)):
            return
        M, F, K, m = self.M, self.F, self.K, self._matrix
        _check(library().gemm_gated_forward(self.handle, m(X, M, K, "X"), m(W, 2 * F, K, "W"), m(H, M, F, "H"),
                                            m(gate_up, M, 2 * F, "gate_up", True), _stream(stream)), "gemm_gated_forward")

    def backward(self, X, W, gate_up, dH, dgate_up, dX=None, dW=None, stream=None) -> None:
        """dgate_up (which may be gate_up) from dH, and from it dX and dW, each optional (W and X may be None with them)."""
        if self._taken(self._enter_backward, "gemm_gated_backward", (X, W, gate_up, dH, dgate_up, dX, dW, stream)):
            return
        M, F, K, m = self.M, self.F, self.K, self._matrix
        _check(library().gemm_gated_backward(
            self.handle, m(X, M, K, "X", dW is None), m(W, 2 * F, K, "W", dX is None), m(gate_up, M, 2 * F, "gate_up"),
            m(dH, M, F, "dH"), m(dgate_up, M, 2 * F, "dgate_up"), m(dX, M, K, "dX", True), m(dW, 2 * F, K, "dW", True),
            _stream(stream)), "gemm_gated_backward")
