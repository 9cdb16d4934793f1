"""Tensors of another GPU than the plan's are refused (no GPU needed: stand-ins for tensors)."""
import ctypes

import pytest
import torch


class _Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_index = tuple(shape), dtype, device

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device_index

    def dim(self):
        return len(self.shape)

    def stride(self, at=None):
        strides = (self.shape[1], 1) if len(self.shape) == 2 else (1,)
        return strides if at is None else strides[at]

    def is_contiguous(self):
        return True


def test_entry_points_take_the_plans_device_only(gemm_lib):
    gemm_lib.library()
    pc = gemm_lib._pycall
    if pc is None or not hasattr(pc, "TrainCall"):
        pytest.skip("CPython entry points not built")
    args, res = gemm_lib.train.signatures()["gemm_embed_forward"]
    fn = ctypes.CFUNCTYPE(res, *args)(lambda *a: 0)
    kinds = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64)
    call = pc.TrainCall(2, ctypes.cast(fn, ctypes.c_void_p).value, 4096, torch.float32, torch.float32, kinds, 24, 100, 1,
                        lambda device: 0, 1)
    for ids, table, out, want in ((1, 1, 1, 0), (0, 1, 1, -1), (1, 0, 1, -1), (1, 1, 0, -1)):
        assert call(_Tensor((6,), torch.int64, ids), _Tensor((100, 24), torch.float32, table),
                    _Tensor((6, 24), torch.float32, out), 1.0, -1, 9) == want


def test_general_path_takes_the_current_device_only(gemm_lib, monkeypatch):
    train = gemm_lib.train
    train._torch_types()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert train._matrix(_Tensor((6, 24), torch.float32, 1), 6, 24, 2, "x") == (4096, 24)
    assert train._vector(_Tensor((6,), torch.float32, 1), 6, 2, "mean") == 4096
    for call in (lambda: train._matrix(_Tensor((6, 24), torch.float32, 0), 6, 24, 2, "x"),
                 lambda: train._vector(_Tensor((6,), torch.float32, 0), 6, 2, "mean")):
        with pytest.raises(gemm_lib.GemmError) as e:
            call()
        assert e.value.status == 1
