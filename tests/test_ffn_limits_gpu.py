"""The conversion of as many rows and as many columns as it takes."""
import torch
import pytest

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
N, PART = 2 ** 31 - 1, 2 ** 20 + 128          # the values repeat after PART, a number of whole groups


def _repeats(got, part):
    """Whether a long vector is `part` again and again."""
    whole = got.numel() // part.numel() * part.numel()
    return bool((got[:whole].view(-1, part.numel()) == part).all()) and torch.equal(got[whole:], part[:got.numel() - whole])


def test_conversion_of_2_31_rows_and_columns(gemm_lib):
    part = torch.randn(PART, generator=torch.Generator().manual_seed(1)).bfloat16()
    x = part.cuda().repeat(N // PART + 1)[:N].clone()
    last = N % 128                             # of the last group
    for shape in ((1, N), (N, 1)):
        q, s = torch.empty(1, N, dtype=FP8, device="cuda"), torch.empty(1, ref.groups(N), device="cuda")
        gemm_lib.fp8_quantize(x.view(shape), q, s, transpose=shape[0] == N)
        want, scales = ref.quantize(part.float().view(1, -1), False)
        end_q, end_s = ref.quantize(x[N - last:].float().cpu().view(1, -1), False)
        assert _repeats(q.view(torch.uint8)[0, :N - last], want.view(torch.uint8)[0].cuda())
        assert torch.equal(q.view(torch.uint8)[0, N - last:].cpu(), end_q.view(torch.uint8)[0])
        assert _repeats(s[0, :-1], scales[0].cuda()) and torch.equal(s[0, -1:].cpu(), end_s[0])
    del q, s
    q, s = torch.empty(N, 1, dtype=FP8, device="cuda"), torch.empty(N, 1, device="cuda")
    gemm_lib.fp8_quantize(x.view(N, 1), q, s)
    want, scales = ref.quantize(part.float().view(-1, 1), False)
    assert _repeats(q.view(torch.uint8)[:, 0], want.view(torch.uint8)[:, 0].cuda()) and _repeats(s[:, 0], scales[:, 0].cuda())
