"""Sizes at the limits that gemm_ffn.h names (no GPU needed)."""
import pytest
import torch

HAS_GPU = torch.cuda.is_available()


@pytest.mark.parametrize("rows,cols,transpose,expect", [
    (2 ** 31 - 1, 0, 0, 0), (0, 2 ** 31 - 1, 0, 0), (2 ** 31 - 1, 0, 1, 0), (2 ** 31 - 128, 0, 0, 0),
    (2 ** 31, 0, 0, 1), (0, 2 ** 31, 1, 1),
    (2 ** 31 - 1, 32 * 128 + 1, 0, 1), (32 * 128 + 1, 2 ** 31 - 1, 1, 1),      # more than 2^29 squares
])
@pytest.mark.parametrize("kind", [0, 1])
def test_conversion_takes_up_to_2_31_rows_and_columns(gemm_lib, rows, cols, transpose, expect, kind):
    out = rows if transpose else cols
    st = gemm_lib.library().gemm_fp8_quantize(rows, cols, 1, 4096, max(cols, 1), kind, transpose, 4096, max(out, 1), 4096,
                                              max(1, -(-out // 128)), None)
    assert st == (expect if expect or HAS_GPU else 4)
