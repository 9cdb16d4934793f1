"""Host side of the feed-forward block's operators (no GPU needed): exports, refusals of the C functions
before they touch a device, plan creation without one, and the oracle of their tests."""
import ctypes
import os
import re

import pytest
import torch

import ffn_oracle as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HAS_GPU = torch.cuda.is_available()


def test_every_declared_function_has_a_signature(gemm_lib):
    text = open(os.path.join(ROOT, "include", "gemm_ffn.h"), encoding="utf-8").read()
    names = set(re.findall(r"\b(gemm_[a-z_0-9]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(gemm_lib.ffn.signatures())
    for n in names:
        assert getattr(gemm_lib.library(), n).argtypes is not None


@pytest.mark.parametrize("name,args,expect", [
    ("gemm_rms_plan_create", (4, 8, 7, 2), 2),              # unknown type
    ("gemm_rms_plan_create", (4, 8, 0, 1), 2),              # bf16 weights of an fp16 norm
    ("gemm_rms_plan_create", (4, 0, 0, 0), 1),
    ("gemm_rms_plan_create", (-1, 8, 0, 0), 1),
    ("gemm_rms_plan_create", (2 ** 31, 8, 0, 0), 1),
    ("gemm_rms_plan_create", (4, 2 ** 30 + 1, 0, 0), 1),
    ("gemm_rms_plan_create", (4, 8, 0, 2), None),
    ("gemm_fp8_plan_create", (4, 8, 16, 2, 0), 2),          # fp32 results
    ("gemm_fp8_plan_create", (4, 8, 16, 0, 2), 2),          # kind of scales
    ("gemm_fp8_plan_create", (-4, 8, 16, 0, 0), 1),
    ("gemm_fp8_plan_create", (4, 8, 2 ** 31 - 16, 0, 0), 1),
    ("gemm_fp8_plan_create", (4, 12, 16, 0, 0), 3),
    ("gemm_fp8_plan_create", (4, 8, 24, 0, 0), 3),
    ("gemm_fp8_plan_create", (2 ** 30, 2 ** 30, 16, 0, 0), 1),
    ("gemm_fp8_plan_create", (4, 8, 16, 1, 1), None),
    ("gemm_gated_plan_create", (4, 8, 8, 2, 3), 2),         # fp32 elements
    ("gemm_gated_plan_create", (4, 8, 8, 0, 4), 2),         # unknown activation
    ("gemm_gated_plan_create", (4, -8, 8, 0, 3), 1),
    ("gemm_gated_plan_create", (4, 2 ** 30, 8, 0, 3), 1),
    ("gemm_gated_plan_create", (2 ** 28, 2 ** 20, 8, 0, 3), 1),
    ("gemm_gated_plan_create", (4, 12, 8, 0, 3), 3),
    ("gemm_gated_plan_create", (4, 8, 12, 0, 3), 3),
    ("gemm_gated_plan_create", (4, 8, 8, 1, 3), None),
])
def test_plan_creation_validates_first(gemm_lib, name, args, expect):
    h = ctypes.c_void_p()
    lib = gemm_lib.library()
    st = getattr(lib, name)(*args, ctypes.byref(h))
    assert st == (expect if expect is not None else 0 if HAS_GPU else 4)
    if st == 0:
        assert getattr(lib, name.replace("create", "destroy"))(h.value) == 0
    else:
        assert not h.value
    assert getattr(lib, name)(*args, None) == 1


def test_null_handles(gemm_lib):
    lib = gemm_lib.library()
    assert lib.gemm_rms_forward(None, 0, None, 0, None, 0, None, 0.0, None, 0, None, 0, None, None) == 1
    assert lib.gemm_rms_forward_fp8(None, 0, None, 0, None, 0, None, 0.0, None, 0, None, 0, None, 0, None, None) == 1
    assert lib.gemm_rms_backward(None, 0, None, 0, None, None, None, 0, None, 0, None, 0, None, None) == 1
    assert lib.gemm_rms_plan_destroy(None) == 0
    assert lib.gemm_fp8_run(None, None, None, None, None, None, None) == 1
    assert lib.gemm_gated_forward(None, None, None, None, None, None) == 1
    assert lib.gemm_gated_backward(None, None, None, None, None, None, None, None, None) == 1
    for kind in ("fp8", "gated"):
        assert getattr(lib, "gemm_%s_plan_set_timeout" % kind)(None, 1) == 1
        assert getattr(lib, "gemm_%s_plan_set_wait_test" % kind)(None, 16) == 1
        assert getattr(lib, "gemm_%s_plan_check" % kind)(None, None) == 1
        assert getattr(lib, "gemm_%s_plan_destroy" % kind)(None) == 0


@pytest.mark.parametrize("args,expect", [
    ((4, 8, 9, 4096, 8, 0, 0, 4096, 8, 4096, 1), 2),         # type
    ((4, 8, 0, 4096, 8, 2, 0, 4096, 8, 4096, 1), 2),         # kind of scales
    ((4, 8, 0, 4096, 8, 0, 2, 4096, 8, 4096, 1), 1),         # transpose
    ((-4, 8, 0, 4096, 8, 0, 0, 4096, 8, 4096, 1), 1),
    ((4, 2 ** 31, 0, 4096, 2 ** 31, 0, 0, 4096, 2 ** 31, 4096, 2 ** 24), 1),
    ((4, 8, 0, 4096, 7, 0, 0, 4096, 8, 4096, 1), 1),         # strides
    ((4, 8, 0, 4096, 8, 0, 0, 4096, 7, 4096, 1), 1),
    ((4, 8, 0, 4096, 8, 0, 1, 4096, 3, 4096, 1), 1),
    ((4, 200, 0, 4096, 200, 0, 0, 4096, 200, 4096, 1), 1),
    ((4, 8, 0, None, 8, 0, 0, 4096, 8, 4096, 1), 1),
    ((4, 8, 0, 4096, 8, 0, 0, 4096, 8, None, 1), 1),
    ((4, 8, 0, 4097, 8, 0, 0, 4096, 8, 4096, 1), 3),
    ((4, 8, 0, 4096, 8, 0, 0, 4096, 8, 4098, 1), 3),
])
def test_conversion_validates_first(gemm_lib, args, expect):
    assert gemm_lib.library().gemm_fp8_quantize(*args, None) == expect


@pytest.mark.skipif(HAS_GPU, reason="checks the no-device path")
def test_plans_without_a_gpu_raise(gemm_lib):
    for make, status in ((lambda: gemm_lib.RmsNormPlan(4, 8), 4), (lambda: gemm_lib.RmsNormPlan(4, 8, "i8"), 2),
                         (lambda: gemm_lib.Fp8Plan(4, 8, 16), 4), (lambda: gemm_lib.Fp8Plan(4, 8, 16, b_scales="column"), 2),
                         (lambda: gemm_lib.GatedPlan(4, 8, 8), 4), (lambda: gemm_lib.GatedPlan(4, 8, 8, act="tanh"), 2),
                         (lambda: gemm_lib.fp8_quantize(*[torch.zeros(4, 8)] * 3), 1)):
        with pytest.raises(gemm_lib.GemmError) as e:
            make()
        assert e.value.status == status


def test_oracle_gradients_agree_with_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    t, gamma, dy, dt, step = r(4, 9), r(9), r(4, 9), r(4, 9), 1e-5
    value = lambda t, gamma: ((ref.rms_forward(t, gamma, 1e-5)[0] * dy).sum() + (t * dt).sum())  # noqa: E731
    rstd = ref.rms_forward(t, gamma, 1e-5)[1]
    dx, dgamma = ref.rms_backward(t, gamma, rstd, dy, dt)
    for at in ((0, 0), (2, 5), (3, 8)):
        d = torch.zeros_like(t)
        d[at] = step
        assert abs((value(t + d, gamma) - value(t - d, gamma)) / (2 * step) - dx[at]) < 1e-7
        e = torch.zeros_like(gamma)
        e[at[1]] = step
        assert abs((value(t, gamma + e) - value(t, gamma - e)) / (2 * step) - dgamma[at[1]]) < 1e-7
    x = r(50)
    for kind in ("silu", "gelu", "relu", "none"):
        slope = (ref.act(x + step, kind)[0] - ref.act(x - step, kind)[0]) / (2 * step)
        assert (slope - ref.act(x, kind)[1]).abs().max() < 1e-7


def test_oracle_conversion():
    x = torch.tensor([[448.0, 1.0, -3.3, 2.0 ** -10]])
    q, s = ref.quantize(x, False)
    assert s.item() == 1.0 and q.float().tolist() == [[448.0, 1.0, -3.25, 0.0]]     # 2^-10 is half the smallest: even
    assert (ref.stands_for(q, s, False) - x.double()).abs().le(ref.conversion_bound(x.double(), s, False)).all()


class _Tensor:
    """A stand-in for a device tensor."""
    is_cuda = True

    def __init__(self, address, shape, ld, dtype):
        self.address, self.shape, self.dtype = address, tuple(shape), dtype
        self._stride = (ld, 1) if len(self.shape) == 2 else (1,)

    def data_ptr(self):
        return self.address

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return len(self.shape) == 1 or self._stride[0] == self.shape[1]


def test_entry_points_marshal_what_they_take(gemm_lib):
    """The C entry points hand the C functions the arguments' addresses, sizes and strides, and take nothing
    that does not fit; a fake function stands in for the library's."""
    gemm_lib.library()
    pc = gemm_lib._pycall
    if pc is None or not hasattr(pc, "TrainCall"):
        pytest.skip("CPython entry points not built")
    seen = []
    bf, f32, f8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    kinds = (torch.float16, bf, f32, torch.int32, torch.int64, f8)

    def fake(kind, name, *sizes, plan=4096):
        args, res = gemm_lib.ffn.signatures()[name]
        fn = ctypes.CFUNCTYPE(res, *args)(lambda *a: seen.append(a) or 0)
        cols, rows, *more = sizes
        return pc.TrainCall(kind, ctypes.cast(fn, ctypes.c_void_p).value, plan, bf, f32, kinds, cols, rows, 0,
                            lambda device: 77 + device, -1, *more), fn
    m = lambda at, rows=6, cols=200, ld=None, dtype=bf: _Tensor(at, (rows, cols), cols if ld is None else ld, dtype)  # noqa: E731
    v = lambda at, n, dtype=f32: _Tensor(at, (n,), 1, dtype)  # noqa: E731

    call, keep = fake(7, "gemm_rms_forward", 200, 0)
    assert call(m(0x100, ld=208), v(0x200, 200), m(0x300), v(0x400, 6), None, m(0x600, ld=224), 0.5, None) == 0
    assert seen[-1] == (4096, 6, 0x100, 208, None, 0, 0x200, 0.5, 0x600, 224, 0x300, 200, 0x400, 77)
    n = len(seen)
    for i, bad in ((0, m(0x100, dtype=f32)), (0, None), (1, v(0x200, 199)), (2, m(0x300, rows=5)), (2, m(0x300, dtype=f8)),
                   (3, v(0x400, 5)), (4, m(0x500, cols=100)), (5, m(0x600, dtype=f32)), (6, "eps")):
        args = [m(0x100), v(0x200, 200), m(0x300), None, None, None, 0.5, None]
        args[i] = bad
        assert call(*args) == -1
    assert len(seen) == n
    call, keep = fake(8, "gemm_rms_forward_fp8", 200, 0)
    assert call(m(0x100), None, m(0x300, dtype=f8, ld=256), m(0x700, cols=2, ld=4, dtype=f32), None, m(0x500, ld=201), None, 0.5, 9) == 0
    assert seen[-1] == (4096, 6, 0x100, 200, 0x500, 201, None, 0.5, None, 0, 0x300, 256, 0x700, 4, None, 9)
    assert call(m(0x100), None, m(0x300), m(0x700, cols=2, dtype=f32), None, None, None, 0.5, 9) == -1
    assert call(m(0x100), None, m(0x300, dtype=f8), m(0x700, cols=1, dtype=f32), None, None, None, 0.5, 9) == -1
    assert call(m(0x100), None, m(0x300, dtype=f8), None, None, None, None, 0.5, 9) == -1
    call, keep = fake(9, "gemm_rms_backward", 200, 0)
    assert call(m(0x100, ld=201), v(0x200, 200), v(0x300, 6), m(0x400, ld=202), m(0x500, ld=203), v(0x600, 200), m(0x700, ld=204), 9) == 0
    assert seen[-1] == (4096, 6, 0x100, 201, 0x200, 0x300, 0x400, 202, 0x700, 204, 0x500, 203, 0x600, 9)
    assert call(m(0x100), None, v(0x300, 6), m(0x400), None, None, None, 9) == 0
    assert seen[-1] == (4096, 6, 0x100, 200, None, 0x300, 0x400, 200, None, 0, None, 0, None, 9)
    assert call(m(0x100), None, None, m(0x400), None, None, None, 9) == -1

    q = lambda at, rows, cols, ld=None: m(at, rows, cols, ld, f8)  # noqa: E731
    s = lambda at, rows, cols, ld=None: m(at, rows, cols, ld, f32)  # noqa: E731
    for square, down in ((True, 3), (False, 264)):
        call, keep = fake(10, "gemm_fp8_run", 264, 6, 144, square)
        args = [q(0x100, 6, 144), s(0x200, 6, 2), q(0x300, 264, 144), s(0x400, down, 2), m(0x500, 6, 264), None]
        assert call(*args) == 0
        assert seen[-1] == (4096, 0x100, 0x200, 0x300, 0x400, 0x500, 77)
        for i, bad in ((0, q(0x100, 6, 144, 160)), (0, m(0x100, 6, 144)), (1, s(0x200, 6, 1)), (2, q(0x300, 6, 144)),
                       (3, s(0x400, 2, 2)), (4, m(0x500, 6, 264, dtype=f32)), (4, None)):
            assert call(*args[:i], bad, *args[i + 1:]) == -1
    call, keep = fake(11, "gemm_gated_forward", 40, 6, 200)
    assert call(m(0x100), m(0x200, 80), m(0x300, 6, 40), None, 9) == 0
    assert seen[-1] == (4096, 0x100, 0x200, 0x300, None, 9)
    assert call(m(0x100), m(0x200, 80), m(0x300, 6, 40), m(0x400, 6, 80), 9) == 0 and seen[-1][4] == 0x400
    assert call(m(0x100), m(0x200, 40), m(0x300, 6, 40), None, 9) == -1
    assert call(m(0x100, ld=208), m(0x200, 80), m(0x300, 6, 40), None, 9) == -1
    call, keep = fake(12, "gemm_gated_backward", 40, 6, 200)
    assert call(m(0x100), m(0x200, 80), m(0x300, 6, 80), m(0x400, 6, 40), m(0x500, 6, 80), m(0x600), m(0x700, 80), 9) == 0
    assert seen[-1] == (4096, 0x100, 0x200, 0x300, 0x400, 0x500, 0x600, 0x700, 9)
    assert call(None, None, m(0x300, 6, 80), m(0x400, 6, 40), m(0x500, 6, 80), None, None, 9) == 0
    assert call(None, m(0x200, 80), m(0x300, 6, 80), m(0x400, 6, 40), m(0x500, 6, 80), None, m(0x700, 80), 9) == -1
    assert call(m(0x100), None, m(0x300, 6, 80), m(0x400, 6, 40), m(0x500, 6, 80), m(0x600), None, 9) == -1

    call, keep = fake(13, "gemm_fp8_quantize", 0, 0, plan=0)
    assert call(m(0x100, ld=208), q(0x200, 6, 200, 256), s(0x300, 6, 2, 5), 0, False, 9) == 0
    assert seen[-1] == (6, 200, 1, 0x100, 208, 0, 0, 0x200, 256, 0x300, 5, 9)
    assert call(m(0x100), q(0x200, 200, 6), s(0x300, 200, 1), 0, True, 9) == 0
    assert seen[-1] == (6, 200, 1, 0x100, 200, 0, 1, 0x200, 6, 0x300, 1, 9)
    assert call(m(0x100), q(0x200, 200, 6), s(0x300, 2, 1), 1, True, 9) == 0
    assert call(m(0x100), q(0x200, 6, 200), s(0x300, 6, 2), 1, False, 9) == -1
    assert call(m(0x100), q(0x200, 6, 200), s(0x300, 6, 2), 0, True, 9) == -1
    assert call(m(0x100, dtype=f8), q(0x200, 6, 200), s(0x300, 6, 2), 0, False, 9) == -1
    for kind, plan, types in ((14, 1, kinds), (7, 0, kinds), (7, 1, kinds[:5]), (6, 1, kinds)):
        with pytest.raises(ValueError):
            pc.TrainCall(kind, 1, plan, bf, bf, types, 1, 1, 0, len)


def test_entry_points_take_the_plans_device_only(gemm_lib):
    gemm_lib.library()
    pc = gemm_lib._pycall
    if pc is None or not hasattr(pc, "TrainCall"):
        pytest.skip("CPython entry points not built")
    args, res = gemm_lib.ffn.signatures()["gemm_gated_forward"]
    fn = ctypes.CFUNCTYPE(res, *args)(lambda *a: 0)
    kinds = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn)
    call = pc.TrainCall(11, ctypes.cast(fn, ctypes.c_void_p).value, 4096, torch.bfloat16, torch.bfloat16, kinds, 40, 6, 1,
                        lambda device: 0, 1, 200)

    def at(device, rows, cols):
        t = _Tensor(4096, (rows, cols), cols, torch.bfloat16)
        t.get_device = lambda: device
        return t
    for x, w, h, want in ((1, 1, 1, 0), (0, 1, 1, -1), (1, 0, 1, -1), (1, 1, 0, -1)):
        assert call(at(x, 6, 200), at(w, 80, 200), at(h, 6, 40), None, 9) == want
