"""The operators around the products of a training step (``include/gemm_train.h``):
embedding lookup, layer norm and distillation from a teacher's top logits, each with
its gradient.

As in the rest of the binding, a plan class owns a C handle, its methods take torch
tensors (device memory) and a stream, and everything is computed by the library's
CUDA kernels.  Matrices are 2-D tensors with contiguous rows (any row stride).  A
tensor of another shape or type than the plan's raises ``GemmError``
(``GEMM_ERR_INVALID_ARG`` / ``GEMM_ERR_UNSUPPORTED``) before anything is queued.

    with NormPlan(max_rows, cols, "bf16", weight="f32") as norm:
        norm.forward(x, gamma, beta, y, mean, rstd)
        norm.backward(x, gamma, mean, rstd, dy, dx, dgamma, dbeta)
    with EmbedPlan(vocab, dim, max_tokens, "bf16", grad="f32") as embed:
        embed.forward(ids, table, out, scale=8.0, padding=0)
        embed.backward(ids, dout, dtable, scale=8.0, padding=0, accumulate=True)
        embed.check()                       # ids outside the table raise here
    with DistillPlan(max_rows, vocab, max_top, "bf16") as kd:
        kd.forward_backward(logits, ids, values, loss, lse, dlogits, temperature=2.0)
"""
from __future__ import annotations

import ctypes

import dense_gemm_hgemm_gb300 as _base   # (its C entry points are there once the library is loaded)

from . import GemmError, _check, _stream, library

__all__ = ["GEMM_ELEM_F16", "GEMM_ELEM_BF16", "GEMM_ELEM_F32", "GEMM_INDEX_I32", "GEMM_INDEX_I64",
           "ELEMS", "NormPlan", "EmbedPlan", "DistillPlan"]

GEMM_ELEM_F16, GEMM_ELEM_BF16, GEMM_ELEM_F32 = 0, 1, 2
GEMM_INDEX_I32, GEMM_INDEX_I64 = 0, 1
ELEMS = {"f16": GEMM_ELEM_F16, "bf16": GEMM_ELEM_BF16, "f32": GEMM_ELEM_F32}

_INVALID_ARG, _UNSUPPORTED = 1, 2


class gemm_teacher_t(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("values", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("top", ctypes.c_int64), ("ld_ids", ctypes.c_int64), ("ld_values", ctypes.c_int64),
                ("id_type", ctypes.c_int32), ("value_elem", ctypes.c_int32)]


def signatures():
    """(argument types, result type) of the C functions of gemm_train.h."""
    i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    u64, u32 = ctypes.c_uint64, ctypes.c_uint32
    vpp, teacher = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(gemm_teacher_t)
    return {
        "gemm_norm_plan_create": ([i64, i64, i32, i32, vpp], i32),
        "gemm_norm_forward": ([vp, i64, vp, i64, vp, vp, f32, vp, i64, vp, vp, vp], i32),
        "gemm_norm_backward": ([vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp], i32),
        "gemm_norm_plan_set_timeout": ([vp, u64], i32),
        "gemm_norm_plan_set_wait_test": ([vp, u32, u32], i32),
        "gemm_norm_plan_check": ([vp, vp], i32),
        "gemm_norm_plan_destroy": ([vp], i32),
        "gemm_embed_plan_create": ([i64, i64, i64, i32, i32, vpp], i32),
        "gemm_embed_forward": ([vp, i64, vp, i32, i64, vp, i64, f32, vp, i64, vp], i32),
        "gemm_embed_backward": ([vp, i64, vp, i32, i64, vp, i64, f32, vp, i64, i32, vp], i32),
        "gemm_embed_plan_check": ([vp, vp], i32),
        "gemm_embed_plan_destroy": ([vp], i32),
        "gemm_distill_plan_create": ([i64, i64, i64, i32, vpp], i32),
        "gemm_distill_forward": ([vp, i64, vp, i64, teacher, f32, vp, vp, vp], i32),
        "gemm_distill_backward": ([vp, i64, vp, i64, teacher, f32, vp, vp, vp, i64, vp], i32),
        "gemm_distill_forward_backward": ([vp, i64, vp, i64, teacher, f32, vp, vp, vp, vp, i64, vp],
                                          i32),
        "gemm_distill_plan_set_timeout": ([vp, u64], i32),
        "gemm_distill_plan_set_wait_test": ([vp, u32, u32], i32),
        "gemm_distill_plan_check": ([vp, vp], i32),
        "gemm_distill_plan_destroy": ([vp], i32),
    }


def _elem(e) -> int:
    if isinstance(e, str):
        if e not in ELEMS:
            raise GemmError(_UNSUPPORTED, "element type %r" % e)
        return ELEMS[e]
    return int(e)


_torch_elems = None     # torch dtype -> gemm_elem_t
_torch_indices = None   # torch dtype -> gemm_index_t


def _torch_types():
    global _torch_elems, _torch_indices
    if _torch_elems is None:
        import torch
        _torch_indices = {torch.int32: GEMM_INDEX_I32, torch.int64: GEMM_INDEX_I64}
        _torch_elems = {torch.float16: GEMM_ELEM_F16, torch.bfloat16: GEMM_ELEM_BF16,
                        torch.float32: GEMM_ELEM_F32}


def _elem_of(t, what):
    e = _torch_elems.get(t.dtype)
    if e is None:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    return e


def _index_of(t, what):
    i = _torch_indices.get(t.dtype)
    if i is None:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    return i


def _on_device(t) -> bool:
    """Whether a tensor is on the current device (the library refuses a plan of another one)."""
    import torch
    return t.is_cuda and t.get_device() == torch.cuda.current_device()


def _matrix(t, rows, cols, elem, what):
    """(address, row stride) of a rows x cols device matrix with contiguous rows
    (`elem` None: any type)."""
    if not _on_device(t) or t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise GemmError(_INVALID_ARG, "%s: a %d x %d matrix on the current device is needed"
                        % (what, rows, cols))
    if elem is not None and _torch_elems.get(t.dtype) != elem:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    if cols > 1 and t.stride(1) != 1:
        raise GemmError(_INVALID_ARG, "%s: rows have to be contiguous" % what)
    # the stride of a single row says nothing; rows may not overlap
    ld = t.stride(0) if rows > 1 else cols
    return t.data_ptr(), ld


def _vector(t, n, elem, what, may_be_none=False):
    """Address of a contiguous device vector of n values (`elem` None: any type)."""
    if t is None:
        if may_be_none:
            return None
        raise GemmError(_INVALID_ARG, "%s: a tensor is needed" % what)
    if not _on_device(t) or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise GemmError(_INVALID_ARG, "%s: a contiguous vector of %d values on the current device is needed"
                        % (what, n))
    if elem is not None and _torch_elems.get(t.dtype) != elem:
        raise GemmError(_UNSUPPORTED, "%s: %s" % (what, t.dtype))
    return t.data_ptr()


class _Plan:
    """Owner of a C plan handle (`_destroy`: the C function that frees it)."""

    _destroy = ""

    def _drop(self):
        """Forget the C entry points: they hold the plan's handle."""

    def _create(self, name, *args):
        _torch_types()
        self.handle = None
        h = ctypes.c_void_p()
        _check(getattr(library(), name)(*args, ctypes.byref(h)), name)
        self.handle = h.value

    def _entry(self, kind, name, elem, weight, cols, rows=0, *more, extra_types=()):
        """The C entry point of one call of this plan, which checks the arguments and
        marshals them (the general path below each method does the same in Python and
        says what is wrong); None where the C module could not be built."""
        call = getattr(_base._pycall, "TrainCall", None)
        if call is None:
            return None
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            raw = lambda device: torch.cuda.current_stream(device).cuda_stream  # noqa: E731
        kinds = (torch.float16, torch.bfloat16, torch.float32)
        return call(kind, ctypes.cast(getattr(library(), name), ctypes.c_void_p).value, self.handle, kinds[elem],
                    kinds[weight], (*kinds, torch.int32, torch.int64, *extra_types), cols, rows,
                    torch.cuda.current_device(), raw,
                    torch.cuda.current_device() if torch.cuda.device_count() > 1 else -1, *more)

    @staticmethod
    def _taken(entry, name, args) -> bool:
        """Whether the C entry point took the call."""
        if entry is None:
            return False
        status = entry(*args)
        if status > 0:
            raise GemmError(status, name)
        return status == 0

    def close(self) -> None:
        self._drop()
        handle, self.handle = getattr(self, "handle", None), None
        if handle:
            _check(getattr(library(), self._destroy)(handle), self._destroy)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class NormPlan(_Plan):
    """Layer norm over rows of `cols` elements, for up to `max_rows` rows a call."""

    _destroy = "gemm_norm_plan_destroy"

    def __init__(self, max_rows: int, cols: int, dtype="f16", weight=None):
        self.max_rows, self.cols = max_rows, cols
        self._elem = _elem(dtype)
        self._weight = self._elem if weight is None else _elem(weight)
        self._create("gemm_norm_plan_create", max_rows, cols, self._elem, self._weight)
        self._forward = self._entry(0, "gemm_norm_forward", self._elem, self._weight, cols)
        self._backward = self._entry(1, "gemm_norm_backward", self._elem, self._weight, cols)

    def _drop(self):
        self._forward = self._backward = None

    def forward(self, x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5,
                stream=None) -> None:
        """y = (x - mean) * rstd * gamma + beta; mean and rstd (fp32) are kept for backward."""
        if self._taken(self._forward, "gemm_norm_forward", (x, gamma, beta, y, mean, rstd, eps, stream)):
            return
        rows, cols = x.shape[0], self.cols
        px, ldx = _matrix(x, rows, cols, self._elem, "x")
        py, ldy = _matrix(y, rows, cols, self._elem, "y")
        _check(library().gemm_norm_forward(
            self.handle, rows, px, ldx, _vector(gamma, cols, self._weight, "gamma", True),
            _vector(beta, cols, self._weight, "beta", True), eps, py, ldy,
            _vector(mean, rows, GEMM_ELEM_F32, "mean", True),
            _vector(rstd, rows, GEMM_ELEM_F32, "rstd", True), _stream(stream)), "gemm_norm_forward")

    def backward(self, x, gamma, mean, rstd, dy, dx=None, dgamma=None, dbeta=None,
                 stream=None) -> None:
        """Gradients of x, gamma and beta (each optional) from dy."""
        if self._taken(self._backward, "gemm_norm_backward",
                       (x, gamma, mean, rstd, dy, dx, dgamma, dbeta, stream)):
            return
        rows, cols = x.shape[0], self.cols
        px, ldx = _matrix(x, rows, cols, self._elem, "x")
        pdy, lddy = _matrix(dy, rows, cols, self._elem, "dy")
        pdx, lddx = (None, 0) if dx is None else _matrix(dx, rows, cols, self._elem, "dx")
        _check(library().gemm_norm_backward(
            self.handle, rows, px, ldx, _vector(gamma, cols, self._weight, "gamma", True),
            _vector(mean, rows, GEMM_ELEM_F32, "mean"), _vector(rstd, rows, GEMM_ELEM_F32, "rstd"),
            pdy, lddy, pdx, lddx, _vector(dgamma, cols, self._weight, "dgamma", True),
            _vector(dbeta, cols, self._weight, "dbeta", True), _stream(stream)),
            "gemm_norm_backward")

    def set_timeout(self, ns: int) -> None:
        """The limit of a wait in this plan's kernels, in nanoseconds (0: the default, 2e9)."""
        _check(library().gemm_norm_plan_set_timeout(self.handle, ns), "gemm_norm_plan_set_timeout")

    def set_wait_test(self, extra_bytes: int, every: int = 1) -> None:
        """Test hook: the copies of every `every`-th block wait for bytes that do not come (0: off)."""
        _check(library().gemm_norm_plan_set_wait_test(self.handle, extra_bytes, every),
               "gemm_norm_plan_set_wait_test")

    def check(self, stream=None) -> None:
        """Synchronise `stream`; raise GemmError(GEMM_ERR_DEVICE_TIMEOUT) if a kernel gave up on a wait."""
        _check(library().gemm_norm_plan_check(self.handle, _stream(stream)), "gemm_norm_plan_check")


class EmbedPlan(_Plan):
    """Lookup in a table of `vocab` rows of `dim` elements, for up to `max_tokens` tokens a call."""

    _destroy = "gemm_embed_plan_destroy"

    def __init__(self, vocab: int, dim: int, max_tokens: int, dtype="f16", grad=None):
        self.vocab, self.dim, self.max_tokens = vocab, dim, max_tokens
        self._elem = _elem(dtype)
        self._grad = self._elem if grad is None else _elem(grad)
        self._create("gemm_embed_plan_create", vocab, dim, max_tokens, self._elem, self._grad)
        self._forward = self._entry(2, "gemm_embed_forward", self._elem, self._grad, dim, vocab)
        self._backward = self._entry(3, "gemm_embed_backward", self._elem, self._grad, dim, vocab)

    def _drop(self):
        self._forward = self._backward = None

    def forward(self, ids, table, out, scale: float = 1.0, padding: int = -1, stream=None) -> None:
        """out[t] = scale * table[ids[t]]; rows of padding tokens are zeros."""
        if self._taken(self._forward, "gemm_embed_forward", (ids, table, out, scale, padding, stream)):
            return
        n = ids.shape[0]
        pt, ldt = _matrix(table, self.vocab, self.dim, self._elem, "table")
        po, ldo = _matrix(out, n, self.dim, self._elem, "out")
        _check(library().gemm_embed_forward(
            self.handle, n, _vector(ids, n, None, "ids"), _index_of(ids, "ids"), padding, pt, ldt,
            scale, po, ldo, _stream(stream)), "gemm_embed_forward")

    def backward(self, ids, dout, dtable, scale: float = 1.0, padding: int = -1,
                 accumulate: bool = False, stream=None) -> None:
        """The table's gradient: written whole, or added to dtable where `accumulate`."""
        if self._taken(self._backward, "gemm_embed_backward",
                       (ids, dout, dtable, scale, padding, accumulate, stream)):
            return
        n = ids.shape[0]
        pd, ldo = _matrix(dout, n, self.dim, self._elem, "dout")
        pt, ldt = _matrix(dtable, self.vocab, self.dim, self._grad, "dtable")
        _check(library().gemm_embed_backward(
            self.handle, n, _vector(ids, n, None, "ids"), _index_of(ids, "ids"), padding, pd, ldo,
            scale, pt, ldt, 1 if accumulate else 0, _stream(stream)), "gemm_embed_backward")

    def check(self, stream=None) -> None:
        """Synchronise `stream`; raise GemmError(GEMM_ERR_INDEX) if an id was outside the table."""
        _check(library().gemm_embed_plan_check(self.handle, _stream(stream)),
               "gemm_embed_plan_check")


class DistillPlan(_Plan):
    """Distillation loss of up to `max_rows` rows of logits over `vocab` tokens against up to
    `max_top` teacher entries a row (token ids, negative = none, and logits)."""

    _destroy = "gemm_distill_plan_destroy"

    def __init__(self, max_rows: int, vocab: int, max_top: int, dtype="f16"):
        self.max_rows, self.vocab, self.max_top = max_rows, vocab, max_top
        self._elem = _elem(dtype)
        self._create("gemm_distill_plan_create", max_rows, vocab, max_top, self._elem)
        self._forward, self._backward, self._both = (
            self._entry(kind, name, self._elem, self._elem, vocab)
            for kind, name in ((4, "gemm_distill_forward"), (5, "gemm_distill_backward"),
                               (6, "gemm_distill_forward_backward")))

    def _drop(self):
        self._forward = self._backward = self._both = None

    def _teacher(self, rows, ids, values, lse):
        top = ids.shape[1]
        pi, ldi = _matrix(ids, rows, top, None, "ids")
        pv, ldv = _matrix(values, rows, top, None, "values")
        return gemm_teacher_t(pi, pv, _vector(lse, rows, GEMM_ELEM_F32, "teacher_lse", True), top,
                              ldi, ldv, _index_of(ids, "ids"), _elem_of(values, "values"))

    def forward(self, logits, ids, values, loss, lse, temperature: float = 1.0, teacher_lse=None,
                stream=None) -> None:
        """Each row's loss and the logits' log-sum-exp at the temperature (fp32)."""
        if self._taken(self._forward, "gemm_distill_forward",
                       (logits, ids, values, loss, lse, temperature, teacher_lse, stream)):
            return
        rows = logits.shape[0]
        pl, ldl = _matrix(logits, rows, self.vocab, self._elem, "logits")
        teacher = self._teacher(rows, ids, values, teacher_lse)
        _check(library().gemm_distill_forward(
            self.handle, rows, pl, ldl, ctypes.byref(teacher), temperature,
            _vector(loss, rows, GEMM_ELEM_F32, "loss"), _vector(lse, rows, GEMM_ELEM_F32, "lse"),
            _stream(stream)), "gemm_distill_forward")

    def backward(self, logits, ids, values, lse, dlogits, dloss=None, temperature: float = 1.0,
                 teacher_lse=None, stream=None) -> None:
        """The logits' gradient from forward's lse and each row's upstream gradient (None: ones)."""
        if self._taken(self._backward, "gemm_distill_backward",
                       (logits, ids, values, lse, dlogits, dloss, temperature, teacher_lse, stream)):
            return
        rows = logits.shape[0]
        pl, ldl = _matrix(logits, rows, self.vocab, self._elem, "logits")
        pd, ldd = _matrix(dlogits, rows, self.vocab, self._elem, "dlogits")
        teacher = self._teacher(rows, ids, values, teacher_lse)
        _check(library().gemm_distill_backward(
            self.handle, rows, pl, ldl, ctypes.byref(teacher), temperature,
            _vector(lse, rows, GEMM_ELEM_F32, "lse"),
            _vector(dloss, rows, GEMM_ELEM_F32, "dloss", True), pd, ldd, _stream(stream)),
            "gemm_distill_backward")

    def forward_backward(self, logits, ids, values, loss, lse, dlogits, dloss=None,
                         temperature: float = 1.0, teacher_lse=None, stream=None) -> None:
        """Loss, lse and gradient in one call."""
        if self._taken(self._both, "gemm_distill_forward_backward",
                       (logits, ids, values, loss, lse, dlogits, dloss, temperature, teacher_lse, stream)):
            return
        rows = logits.shape[0]
        pl, ldl = _matrix(logits, rows, self.vocab, self._elem, "logits")
        pd, ldd = _matrix(dlogits, rows, self.vocab, self._elem, "dlogits")
        teacher = self._teacher(rows, ids, values, teacher_lse)
        _check(library().gemm_distill_forward_backward(
            self.handle, rows, pl, ldl, ctypes.byref(teacher), temperature,
            _vector(dloss, rows, GEMM_ELEM_F32, "dloss", True),
            _vector(loss, rows, GEMM_ELEM_F32, "loss"), _vector(lse, rows, GEMM_ELEM_F32, "lse"),
            pd, ldd, _stream(stream)), "gemm_distill_forward_backward")

    def set_timeout(self, ns: int) -> None:
        """The limit of a wait in this plan's kernels, in nanoseconds (0: the default, 2e9)."""
        _check(library().gemm_distill_plan_set_timeout(self.handle, ns), "gemm_distill_plan_set_timeout")

    def set_wait_test(self, extra_bytes: int, every: int = 1) -> None:
        """Test hook: the copies of every `every`-th block wait for bytes that do not come (0: off)."""
        _check(library().gemm_distill_plan_set_wait_test(self.handle, extra_bytes, every),
               "gemm_distill_plan_set_wait_test")

    def check(self, stream=None) -> None:
        """Synchronise `stream`; raise GemmError(GEMM_ERR_INDEX) if a teacher id was too large,
        GemmError(GEMM_ERR_DEVICE_TIMEOUT) if a kernel gave up on a wait."""
        _check(library().gemm_distill_plan_check(self.handle, _stream(stream)),
               "gemm_distill_plan_check")
