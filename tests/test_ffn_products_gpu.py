"""The 8-bit and the gated product against their 64-bit definitions (tests/ffn_oracle.py has the bounds)."""
import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
T = ref.TYPES
FP8 = torch.float8_e4m3fn

# one tile and less, ragged edges in each direction, one k-block and several, more tiles than one wave
FP8_SIZES = [(1, 8, 16), (1, 128, 128), (3, 136, 272), (16, 1024, 1040), (31, 392, 4096), (33, 256, 640), (64, 2056, 512),
             (127, 264, 1152), (128, 128, 2064), (129, 256, 128), (256, 256, 256), (300, 520, 656), (513, 1032, 1040),
             (2000, 2560, 384)]


def _fp8_operands(M, N, K, square, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = r(M, K) * torch.exp(r(M, 1))
    a[:, : K // 3] *= 20
    if M > 2:
        a[1] = 0
    b = r(N, K) * torch.exp(0.5 * r(N, 1))
    return (*ref.quantize(a, False), *ref.quantize(b, square))


@pytest.mark.parametrize("M,N,K", FP8_SIZES)
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_fp8_product(gemm_lib, M, N, K, square, out):
    a, sa, b, sb = _fp8_operands(M, N, K, square, M + N + K)
    if out == "f16":
        sa = sa / 64                                          # within fp16's range
    want, bound = (v.cpu() for v in ref.fp8_product(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), square))
    whole = torch.full((M + 1, N), 7.0, dtype=T[out], device="cuda")
    C = whole[:M]
    with gemm_lib.Fp8Plan(M, N, K, out, b_scales="square" if square else "row") as plan:
        args = (a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
        plan.run(*args, C)
        plan.check()
        first = C.clone()
        plan.run(*args, C)
        plan.check()
    assert torch.equal(first, C) and (whole[M:] == 7).all()
    assert ((C.cpu().double() - want).abs() <= bound + ref.rounded(want, out) * 1.01).all()


def test_fp8_scales_at_odd_addresses_and_nan(gemm_lib):
    M, N, K = 130, 256, 512
    a, sa, b, sb = _fp8_operands(M, N, K, True, 5)
    bits = a.view(torch.uint8).clone()
    bits[5, 7] = 0x7F                                        # NaN: its row and no other
    a = bits.view(FP8)
    for rows in (M, 17):
        shifted = [torch.empty(v.numel() + 1, device="cuda")[1:].view(v.shape).copy_(v) for v in (sa[:rows].contiguous(), sb)]
        C = torch.empty(rows, N, dtype=T["bf16"], device="cuda")
        with gemm_lib.Fp8Plan(rows, N, K) as plan:
            plan.run(a[:rows].cuda(), shifted[0], b.cuda(), shifted[1], C)
            plan.check()
        keep = torch.arange(rows) != 5
        want, bound = ref.fp8_product(bits[:rows][keep].view(FP8), sa[:rows][keep], b, sb, True)
        assert C[5].isnan().all()
        assert ((C.cpu()[keep].double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()


GATED_SIZES = [(1, 8, 8), (1, 64, 64), (1, 1024, 1096), (3, 72, 200), (17, 200, 4096), (32, 264, 640), (33, 128, 72), (64, 2056, 512),
               (128, 264, 1152), (129, 128, 64), (256, 128, 256), (300, 520, 656), (513, 1032, 264), (1500, 1288, 1024)]


def _gated_operands(M, F, K, elem, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return r(M, K).to(T[elem]).cuda(), (2 * r(2 * F, K) / K ** 0.5).to(T[elem]).cuda()


@pytest.mark.parametrize("M,F,K", GATED_SIZES)
@pytest.mark.parametrize("elem", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_gated_forward(gemm_lib, M, F, K, elem, act):
    X, W = _gated_operands(M, F, K, elem, M + F + K)
    want, bound, gate_up, off = ref.gated_forward(X, W, act)
    whole, kept_whole = (torch.full((M + 1, n), 7.0, dtype=T[elem], device="cuda") for n in (F, 2 * F))
    H, kept = whole[:M], kept_whole[:M]
    with gemm_lib.GatedPlan(M, F, K, elem, act=act) as plan:
        plan.forward(X, W, H)
        plan.check()
        first = H.clone()
        H.zero_()
        plan.forward(X, W, H, gate_up=kept)
        plan.check()
    assert torch.equal(first, H) and (whole[M:] == 7).all() and (kept_whole[M:] == 7).all()
    assert ((H.double() - want).abs() <= bound + ref.rounded(want, elem) * 1.01).all()
    assert ((kept.double() - gate_up).abs() <= off + ref.rounded(gate_up, elem) * 1.01).all()


@pytest.mark.parametrize("M,F,K", GATED_SIZES)
@pytest.mark.parametrize("elem", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_gated_backward(gemm_lib, M, F, K, elem, act):
    X, W = _gated_operands(M, F, K, elem, M + F + K + 1)
    g = torch.Generator().manual_seed(M)
    gate_up = (3 * torch.randn(M, 2 * F, generator=g)).to(T[elem]).cuda()
    gate_up[0, :4] = torch.tensor([0.0, -0.0, 30.0, -30.0], dtype=T[elem])
    dh = torch.randn(M, F, generator=g).to(T[elem]).cuda()
    dgu, dX, dW = torch.empty_like(gate_up), torch.empty_like(X), torch.empty_like(W)
    with gemm_lib.GatedPlan(M, F, K, elem, act=act) as plan:
        plan.backward(X, W, gate_up, dh, dgu, dX, dW)
        plan.check()
        inside, dX2, dW2 = gate_up.clone(), torch.empty_like(X), torch.empty_like(W)
        plan.backward(None, W, inside, dh, inside, dX=dX2)
        plan.backward(X, None, gate_up, dh, torch.empty_like(dgu), dW=dW2)
        plan.check()
    assert torch.equal(inside, dgu) and torch.equal(dX, dX2) and torch.equal(dW, dW2)
    want, bound = ref.gate_gradient(gate_up, dh, act)
    assert ((dgu.double() - want).abs() <= bound + ref.rounded(want, elem) * 1.01).all()
    d = dgu.double()                                         # as it was rounded: the products' operand
    for got, a, b in ((dX, d, W.double()), (dW, d.t(), X.double())):
        value, off = a @ b, ref.mma_error(a.shape[1], 16) * (a.abs() @ b.abs())
        assert ((got.double() - value).abs() <= off + ref.rounded(value, elem) * 1.01).all()


def test_empty_products(gemm_lib):
    new = lambda *s: torch.full(s, 7.0, dtype=T["bf16"], device="cuda")  # noqa: E731
    with gemm_lib.GatedPlan(3, 16, 0) as plan:
        H, gu, dX, dW = new(3, 16), new(3, 32), new(3, 0), new(32, 0)
        plan.forward(new(3, 0), new(32, 0), H, gate_up=gu)
        assert (H == 0).all() and (gu == 0).all()
        plan.backward(new(3, 0), new(32, 0), gu, H, gu, dX, dW)
    with gemm_lib.GatedPlan(0, 16, 24) as plan:
        dW = new(32, 24)
        plan.forward(new(0, 24), new(32, 24), new(0, 16))
        plan.backward(new(0, 24), new(32, 24), new(0, 32), new(0, 16), new(0, 32), new(0, 24), dW)
        assert (dW == 0).all()
    with gemm_lib.GatedPlan(3, 0, 24) as plan:
        dX = new(3, 24)
        plan.backward(new(3, 24), new(0, 24), new(3, 0), new(3, 0), new(3, 0), dX, new(0, 24))
        assert (dX == 0).all()
    with gemm_lib.Fp8Plan(3, 16, 0) as plan:
        C = new(3, 16)
        none = torch.empty(3, 0, device="cuda")
        plan.run(none.to(FP8), none, torch.empty(16, 0, device="cuda").to(FP8), torch.empty(1, 0, device="cuda"), C)
        assert (C == 0).all()


def test_streams_and_graphs(gemm_lib):
    M, F, K = 200, 264, 512
    X, W = _gated_operands(M, F, K, "bf16", 3)
    a, sa, b, sb = (v.cuda() for v in _fp8_operands(M, F, K, True, 4))
    new = lambda *s: torch.zeros(s, dtype=T["bf16"], device="cuda")  # noqa: E731
    outs = H, gu, dgu, dX, dW, C = new(M, F), new(M, 2 * F), new(M, 2 * F), new(M, K), new(2 * F, K), new(M, F)
    side = torch.cuda.Stream()
    with gemm_lib.GatedPlan(M, F, K) as gated, gemm_lib.Fp8Plan(M, F, K) as product:
        def step(stream=None):
            gated.forward(X, W, H, gate_up=gu, stream=stream)
            gated.backward(X, W, gu, H, dgu, dX, dW, stream=stream)
            product.run(a, sa, b, sb, C, stream=stream)
        torch.cuda.synchronize()
        step(side)
        side.synchronize()
        want = [v.clone() for v in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip(outs, want):
            assert torch.equal(v, w)
        gated.check()
        product.check()


@pytest.mark.parametrize("M", [5, 100, 300])
@pytest.mark.parametrize("kind", ["gated", "square", "row"])
def test_a_wait_that_runs_out_is_reported(gemm_lib, M, kind):
    F, K = 520, 2048
    if kind == "gated":
        X, W = _gated_operands(M, F, K, "bf16", 3)
        plan, args = gemm_lib.GatedPlan(M, F, K), (X, W, torch.empty(M, F, dtype=T["bf16"], device="cuda"))
        call = plan.forward
    else:
        ops = [v.cuda() for v in _fp8_operands(M, F, K, kind == "square", 4)]
        plan, args = gemm_lib.Fp8Plan(M, F, K, b_scales=kind), (*ops, torch.empty(M, F, dtype=T["bf16"], device="cuda"))
        call = plan.run
    with plan:
        call(*args)
        plan.check()
        want = args[-1].clone()
        plan.set_timeout(20_000_000)
        plan.set_wait_test(16)
        call(*args)
        with pytest.raises(gemm_lib.GemmError) as e:
            plan.check()
        assert e.value.status == 9
        plan.set_wait_test(0)
        plan.set_timeout(0)
        plan.check()
        call(*args)
        plan.check()
        assert torch.equal(args[-1], want)


def test_refusals(gemm_lib):
    new = lambda *s, dtype=T["bf16"]: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731

    def refused(status, call, *args, **more):
        with pytest.raises(gemm_lib.GemmError) as e:
            call(*args, **more)
        assert e.value.status == status
    X, W, H = new(4, 64), new(32, 64), new(4, 16)
    with gemm_lib.GatedPlan(4, 16, 64) as plan:
        refused(2, plan.forward, X.half(), W, H)
        refused(1, plan.forward, new(4, 72)[:, :64], W, H)
        refused(1, plan.forward, X, new(31, 64), H)
        refused(1, plan.forward, X, W, H, gate_up=new(4, 16))
        refused(1, plan.forward, X.cpu(), W, H)
        refused(3, plan.forward, new(4 * 64 + 1)[1:].view(4, 64), W, H)
        refused(1, plan.backward, None, W, new(4, 32), H, new(4, 32), None, W)
        refused(1, plan.backward, X, None, new(4, 32), H, new(4, 32), X, None)
        refused(1, plan.backward, X, W, None, H, new(4, 32))
        refused(1, plan.set_wait_test, 8)
    q, s = new(4, 64, dtype=FP8), new(4, 1, dtype=torch.float32)
    b, sb = new(16, 64, dtype=FP8), new(1, 1, dtype=torch.float32)
    with gemm_lib.Fp8Plan(4, 16, 64) as plan:
        refused(2, plan.run, q.view(torch.uint8), s, b, sb, H)
        refused(2, plan.run, q, s.half(), b, sb, H)
        refused(2, plan.run, q, s, b, sb, H.half())
        refused(1, plan.run, q, s, b, new(16, 1, dtype=torch.float32), H)
        refused(1, plan.run, q[:3], s, b, sb, H)
        refused(1, plan.run, q, s, b, sb, new(4, 24)[:, :16])
        refused(3, plan.run, new(4 * 64 + 8, dtype=FP8)[8:].view(4, 64), s, b, sb, H)
