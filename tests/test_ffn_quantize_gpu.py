"""Conversion to 8 bits: the same bits as the definition's fp32 arithmetic, every element."""
import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
T = ref.TYPES
FP8 = torch.float8_e4m3fn


def _run(lib, x, block, transpose, pad=0, pad_q=0):
    rows, cols = x.shape
    held = torch.zeros(rows, cols + pad, dtype=x.dtype, device="cuda")
    held[:, :cols] = x.cuda()
    out = (cols, rows) if transpose else (rows, cols)
    q = torch.full((out[0] + 1, out[1] + pad_q), 0x55, dtype=torch.uint8, device="cuda").view(FP8)
    n = ref.groups(out[0]) if block == "square" else out[0]
    s = torch.full((n + 1, ref.groups(out[1]) + 1), 7.0, device="cuda")
    lib.fp8_quantize(held[:, :cols], q[:out[0], :out[1]], s[:n, :-1], block=block, transpose=transpose)
    torch.cuda.synchronize()
    bits = q.view(torch.uint8).cpu()
    assert (bits[out[0]:] == 0x55).all() and (bits[:, out[1]:] == 0x55).all()
    assert (s[n:] == 7).all() and (s[:, -1] == 7).all()
    return bits[:out[0], :out[1]], s[:n, :-1].cpu()


def _same(got, want):
    """Equal bits, any NaN like any other."""
    q, s = got
    wq, ws = want
    nan = wq.float().isnan()
    bits = q.contiguous().view(FP8)
    assert torch.equal(bits.float().isnan(), nan)
    assert torch.equal(q[~nan], wq.contiguous().view(torch.uint8)[~nan])
    assert torch.equal(s, ws)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (127, 5), (128, 128), (129, 257), (1000, 64), (17, 4096),
                                       (300, 1000)])
@pytest.mark.parametrize("elem", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("transpose", [False, True])
def test_bits(gemm_lib, rows, cols, elem, block, transpose):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(T[elem])
    for pad, pad_q in ((0, 0), (3, 5), (8, 8)):
        v = x.float().t() if transpose else x.float()
        _same(_run(gemm_lib, x, block, transpose, pad, pad_q), ref.quantize(v.contiguous(), block == "square"))


@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("transpose", [False, True])
def test_special_values(gemm_lib, block, transpose):
    x = torch.zeros(600, 300)
    x[0, :5] = torch.tensor([float("nan"), 1.0, -2.0, 448.0, 1e-3])
    x[130, 0], x[131, 1] = float("inf"), 3.0                      # a group with an infinity: zeros, NaN in its place
    x[260, 0], x[261, 3] = 1e-40, -1e-45                          # below the smallest scale
    x[400, 200] = 3.4e38
    x[513] = torch.linspace(-1, 1, 300)
    v = x.t().contiguous() if transpose else x
    _same(_run(gemm_lib, x, block, transpose), ref.quantize(v, block == "square"))


def test_nothing_to_convert(gemm_lib):
    for shape in ((0, 64), (64, 0)):
        x = torch.zeros(shape, device="cuda")
        gemm_lib.fp8_quantize(x, torch.zeros(shape, dtype=FP8, device="cuda"),
                              torch.zeros(shape[0], ref.groups(shape[1]), device="cuda"))


def test_refusals(gemm_lib):
    x, q, s = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, dtype=FP8, device="cuda"), torch.zeros(4, 1, device="cuda")

    def refused(status, *args, **more):
        with pytest.raises(gemm_lib.GemmError) as e:
            gemm_lib.fp8_quantize(*args, **more)
        assert e.value.status == status
    refused(2, x, q.view(torch.uint8), s)
    refused(2, x, q, s.half())
    refused(2, x.double(), q, s)
    refused(2, x, q, s, block="column")
    refused(1, x, q, s, transpose=True)
    refused(1, x, q, s, block="square")
    refused(1, x.cpu(), q, s)
    refused(1, x[0], q, s)
    refused(1, x.t(), q, s)
    refused(1, x, q[:3], s)
