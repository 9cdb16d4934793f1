"""How the operators' kernels are launched, as a captured graph has it."""
import ctypes

import pytest
import torch

import test_train_ops_gpu as ops

pytestmark = pytest.mark.gpu


class _KernelNode(ctypes.Structure):      # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _grids(call):
    """Blocks of each kernel that the call launches, the largest first (the graph's nodes have no order)."""
    cuda = ctypes.CDLL("libcuda.so.1")
    stream, graph, n = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()
    assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 1) == 0
    try:
        call(stream)
    finally:
        status = cuda.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
    assert status == 0 and cuda.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    grids = []
    for node in nodes:
        p = _KernelNode()
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        grids.append((p.block[0], p.grid[0]))
    assert cuda.cuGraphDestroy(graph) == 0
    return [g for _, g in sorted(grids, reverse=True)]


@pytest.mark.parametrize("rows,cols,elem,groups", [
    (2500, 125, "f32", 16), (2500, 121, "f32", 16), (5000, 127, "f32", 16), (2500, 256, "f32", 16), (2500, 253, "bf16", 16),
    (2500, 512, "f16", 16), (1300, 4096, "bf16", 2), (400, 12000, "bf16", 1)])
def test_norm_gradient_has_enough_blocks(gemm_lib, rows, cols, elem, groups):
    """Where a block has `groups` of warps with a row each: two rows a group, or a block on every multiprocessor."""
    c = ops._norm_case(rows, cols, elem, "f32", 0, 0)
    with gemm_lib.NormPlan(rows, cols, elem, weight="f32") as plan:
        plan.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"])

        def call(stream):
            plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"], c["dbeta"], stream=stream)
        # the rows' kernel, and the one of fewer threads a block that joins the weights' gradients
        blocks, sms = _grids(call)[0], torch.cuda.get_device_properties(0).multi_processor_count
        assert blocks <= sms and (blocks == sms or blocks * groups * 2 >= rows), blocks
        call(None)
        torch.cuda.synchronize()
        ops._check_norm(c, elem, "f32")
        plan.check()
