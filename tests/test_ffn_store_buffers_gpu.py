"""The 8-bit product's store buffers where a tile's last columns fill one of a warp's two: the next tile of the same
pair of SMs may not write to it before the copy out of it has read it."""
import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


# Tiles of 256 columns, several to each pair with more behind a ragged one: N mod 256 in 8 .. 64 (the first warps' second
# half is missing) and in 136 .. 192 (the other warps').  One and two k-blocks: the next tile's sums follow at once.
@pytest.mark.parametrize("M,N", [(8192, 2112), (4096, 2112), (8000, 4264), (4096, 4904), (2560, 10000)])
@pytest.mark.parametrize("K", [128, 256])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_ragged_last_columns_before_further_tiles(gemm_lib, M, N, K, out):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b = (torch.randn(r, K, generator=g, device="cuda").to(FP8) for r in (M, N))
    sa, sb = (torch.rand(r, ref.groups(K), generator=g, device="cuda") + 0.5 for r in (M, ref.groups(N)))
    want, bound = ref.fp8_product(a, sa, b, sb, True)
    bound = bound + ref.rounded(want, out) * 1.01
    first = None
    with gemm_lib.Fp8Plan(M, N, K, out) as plan:
        for _ in range(20):
            C = torch.full((M, N), 7.0, dtype=ref.TYPES[out], device="cuda")
            plan.run(a, sa, b, sb, C)
            if first is None:
                first = C
                assert ((C.double() - want).abs() <= bound).all()
            assert torch.equal(C, first)
        plan.check()
