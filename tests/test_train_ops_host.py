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
    ("gemm_norm_plan_create", (4, 8, 0, 2), None),
    ("gemm_embed_plan_create", (0, 8, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 0, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 8, -4, 0, 0), 1),
    ("gemm_embed_plan_create", (2 ** 31, 8, 4, 0, 0), 1),
    ("gemm_embed_plan_create", (8, 8, 4, 1, 0), 2),
    ("gemm_embed_plan_create", (8, 8, 4, 1, 2), None),
    ("gemm_distill_plan_create", (4, 0, 4, 0), 1),
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
