"""Host side of the operators around a training step's products (no GPU needed): exports,
refusals of the C functions before they touch a device, and plan creation without one."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HAS_GPU = torch.cuda.is_available()


def test_every_declared_function_has_a_signature(gemm_lib):
    text = open(os.path.join(ROOT, "include", "gemm_train.h"), encoding="utf-8").read()
    names = set(re.findall(r"\b(gemm_[a-z_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(gemm_lib.train.signatures())
    for n in names:
        assert getattr(gemm_lib.library(), n).argtypes is not None


@pytest.mark.parametrize("name,args,expect", [
    ("gemm_norm_plan_create", (4, 8, 7, 2), 2),             # unknown type
    ("gemm_norm_plan_create", (4, 8, 0, 1), 2),             # bf16 weights of an fp16 norm
    ("gemm_norm_plan_create", (4, 0, 0, 0), 1),
    ("gemm_norm_plan_create", (-1, 8, 0, 0), 1),
    ("gemm_norm_plan_create", (4, 2 ** 31, 0, 0), 1),
    ("gemm_norm_plan_create", (4, 2 ** 30 + 1, 0, 0), 1),
    ("gemm_norm_plan_create", (4, 8, 0, 2), None),
    ("gemm_embed_plan_create", (0, 8, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 0, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 8, -4, 0, 0), 1),
    ("gemm_embed_plan_create", (2 ** 31, 8, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 2 ** 30 + 1, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 8, 4, 1, 0), 2),
    ("gemm_embed_plan_create", (8, 8, 4, 1, 2), None),
    ("gemm_distill_plan_create", (4, 0, 4, 0), 1),
    ("gemm_distill_plan_create", (4, 2 ** 30 + 1, 4, 0), 1),
    ("gemm_distill_plan_create", (4, 8, 1025, 0), 1),
    ("gemm_distill_plan_create", (4, 8, -1, 0), 1),
    ("gemm_distill_plan_create", (4, 8, 4, 3), 2),
    ("gemm_distill_plan_create", (4, 8, 4, 2), None),
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
    t = gemm_lib.train.gemm_teacher_t()
    assert lib.gemm_norm_forward(None, 0, None, 0, None, None, 0.0, None, 0, None, None, None) == 1
    assert lib.gemm_norm_backward(None, 0, None, 0, None, None, None, None, 0, None, 0, None, None, None) == 1
    assert lib.gemm_embed_forward(None, 0, None, 0, 0, None, 0, 1.0, None, 0, None) == 1
    assert lib.gemm_embed_backward(None, 0, None, 0, 0, None, 0, 1.0, None, 0, 0, None) == 1
    assert lib.gemm_distill_forward(None, 0, None, 0, ctypes.byref(t), 1.0, None, None, None) == 1
    assert lib.gemm_distill_backward(None, 0, None, 0, ctypes.byref(t), 1.0, None, None, None, 0, None) == 1
    assert lib.gemm_distill_forward_backward(None, 0, None, 0, ctypes.byref(t), 1.0, None, None, None, None, 0, None) == 1
    for kind in ("norm", "embed", "distill"):
        assert getattr(lib, "gemm_%s_plan_destroy" % kind)(None) == 0
    assert lib.gemm_embed_plan_check(None, None) == 1 and lib.gemm_distill_plan_check(None, None) == 1


@pytest.mark.skipif(HAS_GPU, reason="checks the no-device path")
def test_plans_without_a_gpu_raise(gemm_lib):
    for make in (lambda: gemm_lib.NormPlan(4, 8), lambda: gemm_lib.EmbedPlan(8, 8, 4),
                 lambda: gemm_lib.DistillPlan(4, 8, 2)):
        with pytest.raises(gemm_lib.GemmError) as e:
            make()
        assert e.value.status == 4
    with pytest.raises(gemm_lib.GemmError) as e:
        gemm_lib.NormPlan(4, 8, "i8")
    assert e.value.status == 2


class _Tensor:
    """What the C entry points ask of a tensor."""

    is_cuda = True

    def __init__(self, address, shape, stride, dtype):
        self.address, self.shape, self._stride, self.dtype = address, tuple(shape), tuple(stride), dtype

    def data_ptr(self):
        return self.address

    def stride(self):
        return self._stride

    def is_contiguous(self):
        want = 1
        for n, at in zip(reversed(self.shape), reversed(self._stride)):
            if at != want:
                return False
            want *= n
        return True


def test_entry_points_marshal_what_they_take(gemm_lib):
    """The C entry points hand the C functions the arguments' addresses, sizes and strides, and take nothing
    that does not fit; a fake function stands in for the library's."""
    gemm_lib.library()
    pc = gemm_lib._pycall
    if pc is None or not hasattr(pc, "TrainCall"):
        pytest.skip("CPython entry points not built")
    seen = []

    def fake(kind, name):
        args, res = gemm_lib.train.signatures()[name]
        args = [ctypes.c_void_p if hasattr(a, "_type_") and not isinstance(a._type_, str) else a for a in args]

        def called(*a):
            teacher = None
            if "distill" in name:
                t = gemm_lib.train.gemm_teacher_t.from_address(a[4])
                teacher = {f: getattr(t, f) for f, _ in t._fields_}
            seen.append((a, teacher))
            return 0
        fn = ctypes.CFUNCTYPE(res, *args)(called)
        kinds = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64)
        call = pc.TrainCall(kind, ctypes.cast(fn, ctypes.c_void_p).value, 4096, torch.bfloat16, torch.float32, kinds,
                            24, 100, 0, lambda device: 77 + device)
        return call, fn

    bf, f32 = torch.bfloat16, torch.float32
    m = lambda at, rows=6, cols=24, ld=32, dtype=bf: _Tensor(at, (rows, cols), (ld, 1), dtype)  # noqa: E731
    v = lambda at, n=24, dtype=f32: _Tensor(at, (n,), (1,), dtype)  # noqa: E731

    call, keep = fake(0, "gemm_norm_forward")
    assert call(m(0x100), v(0x200), None, m(0x300, ld=40), v(0x400, 6), None, 0.5, None) == 0
    assert seen[-1][0] == (4096, 6, 0x100, 32, 0x200, None, 0.5, 0x300, 40, 0x400, None, 77)
    n = len(seen)
    for bad in ([m(0x100, cols=23)], [m(0x100, dtype=f32)], [v(0x100)], [None], [3], ["x"]):
        assert call(bad[0], v(0x200), None, m(0x300), v(0x400, 6), None, 0.5, None) == -1
    assert call(m(0x100), v(0x200, 23), None, m(0x300), None, None, 0.5, None) == -1
    assert call(m(0x100), v(0x200), None, m(0x300, rows=5), None, None, 0.5, None) == -1
    assert call(m(0x100), v(0x200), None, m(0x300), None, None, "eps", None) == -1
    assert call(m(0x100), v(0x200), None, m(0x300), None, None, 0.5) == -1
    host = m(0x100)
    host.is_cuda = False
    assert call(host, v(0x200), None, m(0x300), None, None, 0.5, None) == -1
    assert len(seen) == n

    call, keep = fake(1, "gemm_norm_backward")
    assert call(m(0x100), None, v(0x200, 6), v(0x300, 6), m(0x400), None, v(0x500), None, 5) == 0
    assert seen[-1][0] == (4096, 6, 0x100, 32, None, 0x200, 0x300, 0x400, 32, None, 0, 0x500, None, 5)
    assert call(m(0x100), None, None, v(0x300, 6), m(0x400), None, v(0x500), None, 5) == -1

    ids = _Tensor(0x700, (6,), (1,), torch.int64)
    table = lambda dtype: m(0x800, rows=100, ld=24, dtype=dtype)  # noqa: E731
    call, keep = fake(2, "gemm_embed_forward")
    assert call(ids, table(bf), m(0x900), 2.0, -1, 9) == 0
    assert seen[-1][0] == (4096, 6, 0x700, 1, -1, 0x800, 24, 2.0, 0x900, 32, 9)
    assert call(ids, m(0x800, rows=99), m(0x900), 2.0, -1, 9) == -1
    call, keep = fake(3, "gemm_embed_backward")
    assert call(ids, m(0x900), table(f32), 2.0, 3, True, 9) == 0
    assert seen[-1][0] == (4096, 6, 0x700, 1, 3, 0x900, 32, 2.0, 0x800, 24, 1, 9)
    assert call(ids, m(0x900), table(bf), 2.0, 3, True, 9) == -1

    entry = _Tensor(0xa00, (6, 3), (4, 1), torch.int32)
    value = _Tensor(0xb00, (6, 3), (3, 1), torch.float16)
    want = {"ids": 0xa00, "values": 0xb00, "lse": None, "top": 3, "ld_ids": 4, "ld_values": 3, "id_type": 0, "value_elem": 0}
    call, keep = fake(4, "gemm_distill_forward")
    assert call(m(0x100), entry, value, v(0x200, 6), v(0x300, 6), 1.5, None, 9) == 0
    a, t = seen[-1]
    assert a[:4] + a[5:] == (4096, 6, 0x100, 32, 1.5, 0x200, 0x300, 9) and t == want
    assert call(m(0x100), entry, _Tensor(0xb00, (6, 2), (3, 1), f32), v(0x200, 6), v(0x300, 6), 1.5, None, 9) == -1
    call, keep = fake(5, "gemm_distill_backward")
    assert call(m(0x100), entry, value, v(0x300, 6), m(0x400), None, 1.5, v(0x500, 6), 9) == 0
    a, t = seen[-1]
    assert a[:4] + a[5:] == (4096, 6, 0x100, 32, 1.5, 0x300, None, 0x400, 32, 9) and t == dict(want, lse=0x500)
    call, keep = fake(6, "gemm_distill_forward_backward")
    assert call(m(0x100), entry, value, v(0x200, 6), v(0x300, 6), m(0x400), v(0x600, 6), 1.5, None, 9) == 0
    a, t = seen[-1]
    assert a[:4] + a[5:] == (4096, 6, 0x100, 32, 1.5, 0x600, 0x200, 0x300, 0x400, 32, 9) and t == want
    with pytest.raises(TypeError):
        call(m(0x100), stream=None)
    for bad in ((9, 1), (0, 0)):
        with pytest.raises(ValueError):
            pc.TrainCall(bad[0], bad[1], 1, bf, bf, (1, 2, 3, 4, 5), 1, 1, 0, len)
