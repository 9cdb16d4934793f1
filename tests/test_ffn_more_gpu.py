"""The feed-forward block's operators where they could go wrong: offsets past 32 bits, several streams and plans at
once, first calls within a capture, one matrix in two roles, the limits between the kernels' paths."""
import os
import subprocess
import sys

import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
T = ref.TYPES
FP8 = torch.float8_e4m3fn
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _randn(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _room(rows, cols, ld, dtype):
    """A matrix whose rows stand `ld` elements apart, in a buffer of that size."""
    return torch.empty((rows - 1) * ld + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1))


FAR = 2 ** 31 + 16       # elements: the second row lies past 2^32 bytes, the third past 2^32 elements


def test_norm_of_rows_far_apart(gemm_lib):
    rows, cols = 3, 1000
    x, r, dy = (_randn(rows, cols, seed=s) for s in range(3))
    gamma = _randn(cols, seed=4, dtype=torch.float32) + 2
    far = _room(rows, cols, FAR, torch.bfloat16)
    q, s = _room(rows, cols, 2 * FAR, FP8), torch.empty(rows, 8, device="cuda")
    near, total, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    dx, dgamma, dgamma2 = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    q2, s2 = torch.empty(rows, cols, dtype=FP8, device="cuda"), torch.empty_like(s)
    with gemm_lib.RmsNormPlan(rows, cols, "bf16", weight="f32") as plan:
        plan.forward(x, gamma, near, rstd, residual=r, total=total)
        far.copy_(x)
        plan.forward(far, gamma, far, residual=r)                 # y is x
        assert torch.equal(far, near)
        plan.forward_fp8(x, gamma, q2, s2, residual=r)
        far.copy_(r)
        plan.forward_fp8(x, gamma, q, s, residual=far, total=far)
        assert torch.equal(far, total) and torch.equal(s, s2)
        assert torch.equal(q.contiguous().view(torch.uint8), q2.view(torch.uint8))
        plan.backward(total, gamma, rstd, dy, dx, dgamma, dtotal=r)
        plan.backward(far, gamma, rstd, dy, far, dgamma2, dtotal=r)
        assert torch.equal(far, dx) and torch.equal(dgamma, dgamma2)


@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("transpose", [False, True])
def test_conversion_of_rows_far_apart(gemm_lib, block, transpose):
    x = _randn(3, 200, seed=1)
    far = _room(3, 200, FAR, torch.bfloat16)
    far.copy_(x)
    shape = (200, 3) if transpose else (3, 200)
    n = ref.groups(shape[0]) if block == "square" else shape[0]
    results = []
    for source in (x, far):
        q, s = torch.empty(shape, dtype=FP8, device="cuda"), torch.empty(n, ref.groups(shape[1]), device="cuda")
        if source is far and not transpose:
            q = _room(*shape, 2 * FAR, FP8)
        gemm_lib.fp8_quantize(source, q, s, block=block, transpose=transpose)
        results.append((q.contiguous().view(torch.uint8), s))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


def test_products_of_more_than_2_32_elements(gemm_lib):
    """Rows from both ends of operands and results past 2^32 elements, against 64 bits."""
    at = [0, 1, 127, 128, 40000, 65535, 65536, 69998, 69999]
    M, N, K = 70000, 24, 65536 + 16
    a = _randn(M // 10, K, seed=2, dtype=torch.float32).to(FP8).view(torch.uint8).repeat(10, 1).view(FP8)
    b = _randn(N, K, seed=3, dtype=torch.float32).to(FP8)
    sa = torch.rand(M, ref.groups(K), device="cuda") + 0.5
    for kind in ("square", "row"):
        sb = torch.rand(1 if kind == "square" else N, ref.groups(K), device="cuda") + 0.5
        C = torch.empty(M, N, dtype=T["bf16"], device="cuda")
        with gemm_lib.Fp8Plan(M, N, K, b_scales=kind) as plan:
            plan.run(a, sa, b, sb, C)
            plan.check()
        part = a.view(torch.uint8)[at].view(FP8)
        want, bound = ref.fp8_product(part, sa[at], b, sb, kind == "square")
        assert ((C[at].double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()
    del a, sa, C
    M, F, K = 300000, 8192, 16
    at = [0, 5, 131072, 262143, 262144, 299999]
    X, W = _randn(M, K, seed=4), _randn(2 * F, K, seed=5, scale=0.5)
    H, kept = torch.empty(M, F, dtype=T["bf16"], device="cuda"), torch.empty(M, 2 * F, dtype=T["bf16"], device="cuda")
    with gemm_lib.GatedPlan(M, F, K) as plan:
        plan.forward(X, W, H, gate_up=kept)
        plan.check()
        want, bound, gate_up, off = ref.gated_forward(X[at], W, "silu")
        assert ((H[at].double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()
        assert ((kept[at].double() - gate_up).abs() <= off + ref.rounded(gate_up, "bf16") * 1.01).all()
        before = kept[at].clone()
        plan.backward(None, None, kept, H, kept)                 # in place
        plan.check()
    want, bound = ref.gate_gradient(before, H[at], "silu")
    assert ((kept[at].double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()


@pytest.mark.parametrize("M,F,K", [(32, 512, 2048), (33, 512, 2048), (128, 512, 2048), (129, 512, 2048), (256, 64, 4096),
                                   (257, 128, 8192), (400, 4096, 64), (640, 320, 1088), (40, 8, 64 * 9), (40, 8, 64 * 5)])
def test_between_the_kernels_of_few_and_many_rows(gemm_lib, M, F, K):
    """Both sides of the sizes where the kernel or the slices of K change, slices without a k-block among them."""
    X, W = _randn(M, K, seed=M), _randn(2 * F, K, seed=F, scale=2 * K ** -0.5)
    want, bound, gate_up, off = ref.gated_forward(X, W, "gelu")
    H, kept = torch.empty(M, F, dtype=T["bf16"], device="cuda"), torch.empty(M, 2 * F, dtype=T["bf16"], device="cuda")
    with gemm_lib.GatedPlan(M, F, K, act="gelu") as plan:
        plan.forward(X, W, H, gate_up=kept)
        plan.check()
    assert ((H.double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()
    assert ((kept.double() - gate_up).abs() <= off + ref.rounded(gate_up, "bf16") * 1.01).all()
    for square in (True, False):
        a, sa = (v.cuda() for v in ref.quantize(X.float().cpu(), False))
        b, sb = (v.cuda() for v in ref.quantize(W.float().cpu(), square))
        C = torch.empty(M, 2 * F, dtype=T["bf16"], device="cuda")
        want, bound = ref.fp8_product(a, sa, b, sb, square)
        with gemm_lib.Fp8Plan(M, 2 * F, K, b_scales="square" if square else "row") as plan:
            plan.run(a, sa, b, sb, C)
            plan.check()
        assert ((C.double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()


def test_plans_on_two_streams_at_once(gemm_lib):
    """Two plans of each kind, each on its own stream, again and again without a wait between."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    M, F, K = 96, 1024, 2048
    work = []
    for n in range(2):
        X, W, r = _randn(M, K, seed=10 + n), _randn(2 * F, K, seed=20 + n, scale=K ** -0.5), _randn(M, K, seed=30 + n)
        gamma = _randn(K, seed=40 + n)
        q, s = torch.empty(M, K, dtype=FP8, device="cuda"), torch.empty(M, K // 128, device="cuda")
        wq, ws = torch.empty(2 * F, K, dtype=FP8, device="cuda"), torch.empty(2 * F // 128, K // 128, device="cuda")
        new = lambda *shape: torch.zeros(*shape, dtype=T["bf16"], device="cuda")  # noqa: E731
        outs = [new(M, K), new(M, F), new(M, 2 * F), new(M, 2 * F), new(M, K), new(2 * F, K), new(M, K), new(K)]
        plans = (gemm_lib.RmsNormPlan(M, K, "bf16"), gemm_lib.GatedPlan(M, F, K), gemm_lib.Fp8Plan(M, 2 * F, K))

        def step(stream, X=X, W=W, r=r, gamma=gamma, q=q, s=s, wq=wq, ws=ws, outs=outs, plans=plans,
                 rstd=torch.empty(M, device="cuda")):
            y, h, kept, c, dy, dw, dx, dgamma = outs
            norm, gated, product = plans
            norm.forward(X, gamma, y, rstd, residual=r, stream=stream)
            gated.forward(y, W, h, gate_up=kept, stream=stream)
            gated.backward(y, W, kept, h, kept, dy, dw, stream=stream)
            norm.backward(X, gamma, rstd, dy, dx, dgamma, dtotal=r, stream=stream)
            norm.forward_fp8(X, gamma, q, s, residual=r, stream=stream)
            gemm_lib.fp8_quantize(W, wq, ws, block="square", stream=stream)
            product.run(q, s, wq, ws, c, stream=stream)
        work.append((step, outs, plans))
    torch.cuda.synchronize()
    want = []
    for (step, outs, _), stream in zip(work, streams):
        step(stream)
        torch.cuda.synchronize()
        want.append([v.clone() for v in outs])
    for _ in range(20):
        for (step, _, _), stream in zip(work, streams):
            step(stream)
    torch.cuda.synchronize()
    for (_, outs, plans), kept in zip(work, want):
        assert all(torch.equal(v, w) for v, w in zip(outs, kept))
        for plan in plans[1:]:
            plan.check()
        for plan in plans:
            plan.close()


def test_first_calls_within_a_capture(gemm_lib):
    """A fresh process whose first call of every kernel is captured; the replay's results are those of plain calls."""
    code = """
import torch, dense_gemm_hgemm_gb300 as g
B, F8 = torch.bfloat16, torch.float8_e4m3fn
x, r, w = (torch.randn(s, 512, device='cuda').to(B) for s in (300, 300, 512))
gamma = torch.rand(512, device='cuda').to(B)
new = lambda *s, dtype=B: torch.zeros(s, dtype=dtype, device='cuda')
q, s, wq, ws = new(300, 512, dtype=F8), new(300, 4, dtype=torch.float32), new(512, 512, dtype=F8), new(4, 4, dtype=torch.float32)
tq, ts = new(512, 300, dtype=F8), new(512, 3, dtype=torch.float32)
y, rstd, h, gu, dgu, dx, dw, c, dg = new(300, 512), new(300, dtype=torch.float32), new(300, 256), new(300, 512), new(300, 512), new(300, 512), new(512, 512), new(300, 512), new(512)
norm, gated, product = g.RmsNormPlan(300, 512, 'bf16'), g.GatedPlan(300, 256, 512), g.Fp8Plan(300, 512, 512)
few = g.GatedPlan(16, 256, 512)
def step():
    norm.forward(x, gamma, y, rstd, residual=r)
    gated.forward(y, w, h, gate_up=gu)
    gated.backward(y, w, gu, h, dgu, dx, dw)
    norm.backward(x, gamma, rstd, dx, dx, dg)
    norm.forward_fp8(x, gamma, q, s)
    g.fp8_quantize(w, wq, ws, block='square')
    g.fp8_quantize(x, tq, ts, transpose=True)
    product.run(q, s, wq, ws, c)
    few.forward(y[:16], w, h[:16])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (y, h, gu, dgu, dx, dw, dg, c, ts)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (y, h, gu, dgu, dx, dw, dg, c, ts)))
assert all(float(v.float().abs().sum()) > 0 for v in got)
print('captured')
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


def test_conversion_and_product_without_a_plan_before(gemm_lib):
    """fp8_quantize as the first call of a process."""
    code = """
import torch, dense_gemm_hgemm_gb300 as g
x = torch.randn(200, 256, device='cuda')
q, s = torch.empty(200, 256, dtype=torch.float8_e4m3fn, device='cuda'), torch.empty(200, 2, device='cuda')
g.fp8_quantize(x, q, s)
assert ((q.float() * s.repeat_interleave(128, 1) - x).abs() <= x.abs() / 16 + s.repeat_interleave(128, 1) / 1024).all()
print('converted')
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "converted" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("cols", [128, 4096, 16384, 20000])
def test_norm_of_extreme_rows(gemm_lib, cols):
    """Rows of zeros, tiny and large elements, fp32 and bf16: the formula's values, and scales at their floor."""
    sizes = torch.tensor([0.0, 1e-30, 1e-18, 1e-5, 1.0, 1e10, 1e17])
    for elem in ("f32", "bf16"):
        x = (torch.randn(7, cols, generator=torch.Generator().manual_seed(1)) * sizes[:, None]).to(T[elem])
        gamma = torch.ones(cols, dtype=T[elem])
        y, rstd = torch.empty(7, cols, dtype=T[elem], device="cuda"), torch.empty(7, device="cuda")
        q, s = torch.empty(7, cols, dtype=FP8, device="cuda"), torch.empty(7, ref.groups(cols), device="cuda")
        with gemm_lib.RmsNormPlan(7, cols, elem) as plan:
            plan.forward(x.cuda(), gamma.cuda(), y, rstd)
            plan.forward_fp8(x.cuda(), gamma.cuda(), q, s)
        want, want_rstd = ref.rms_forward(x, gamma, 1e-5)
        e = ref.rms_error(cols)
        # (squares below the smallest normal number, of elements below 1e-19, vanish beside eps)
        assert ((rstd.cpu().double() - want_rstd).abs() <= e * want_rstd).all()
        assert ((y.cpu().double() - want).abs() <= 1.01 * (e + 3 * ref.U) * want.abs() + ref.rounded(want, elem) + 2.0 ** -126).all()
        far = (ref.stands_for(q.cpu(), s.cpu(), False) - want).abs()
        assert (far <= ref.conversion_bound(want, s.cpu(), False) * (1 + 1e-6) + 2 * (e + 6 * ref.U) * want.abs() + 2.0 ** -126).all()
        assert (s[0] == 2.0 ** -126).all() and (q[0].view(torch.uint8) & 0x7f).eq(0).all()


def _off(values, first, pad):
    """A device matrix of `values` whose first element lies `first` elements behind a boundary and whose rows stand
    `pad` elements apart, and the whole of its buffer, filled with 7 elsewhere."""
    rows, cols = values.shape
    whole = torch.full((first + rows * (cols + pad) + 8,), 7.0, dtype=values.dtype, device="cuda")
    m = whole.as_strided((rows, cols), (cols + pad, 1), first)
    m.copy_(values)
    return m, whole


def _only_in(m, whole):
    m.fill_(7.0)
    return bool((whole == 7).all())


@pytest.mark.parametrize("cols", [1, 2, 7, 9, 121, 249, 250, 255, 505, 506, 1001, 1024, 2041, 2048, 4089, 4090, 8185, 8186, 8192,
                                  16377, 16378])
@pytest.mark.parametrize("elem,weight", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_norm_of_rows_off_the_boundaries(gemm_lib, cols, elem, weight):
    """Inputs at one distance from the boundaries or at several, results at the same or at another: the same numbers
    wherever the results go, and nothing written beside them."""
    rows = 37 if cols < 4000 else 5
    x, r, dy, dt = (_randn(rows, cols, seed=s + cols, dtype=T[elem]) for s in range(4))
    gamma = (1 + 0.2 * _randn(cols, seed=9)).to(T[weight])
    total = ref.rms_total(x, r)
    want, want_rstd = ref.rms_forward(total, gamma, 1e-5)
    e = ref.rms_error(cols)
    zeros = torch.zeros_like(x)
    with gemm_lib.RmsNormPlan(rows, cols, elem, weight=weight) as plan:
        for first, pad, other in ((1, 0, 1), (3, 5, 3), (7, 8, 7), (0, 1, 0), (2, 3, 5)):
            (a, _), (b, _), (d, _), (m, _) = (_off(v, at, pad) for v, at in ((x, first), (r, other), (dy, first), (dt, other)))
            (y, y_all), (t, t_all), (far, far_all), (t2, _) = (
                _off(zeros, *at) for at in ((first, pad), (first, pad), (first + 1, pad + 2), (0, 0)))
            rstd = torch.empty(rows, device="cuda")
            plan.forward(a, gamma, y, rstd, residual=b, total=t)
            plan.forward(a, gamma, far, residual=b, total=t2)
            assert torch.equal(y, far) and torch.equal(t, t2) and torch.equal(t, total)
            assert ((rstd.double() - want_rstd).abs() <= e * want_rstd).all()
            assert ((y.double() - want).abs() <= 1.01 * (e + 3 * ref.U) * want.abs() + ref.rounded(want, elem)).all()
            assert all(_only_in(*v) for v in ((y, y_all), (t, t_all), (far, far_all)))
            (q, q_all), (s, s_all) = _off(torch.zeros(rows, cols, device="cuda").to(torch.uint8), first, 1), _off(
                torch.zeros(rows, ref.groups(cols), device="cuda"), 0, 1)
            plan.forward_fp8(a, gamma, q.view(FP8), s, residual=b)
            off = (ref.stands_for(q.view(FP8), s, False) - want).abs()
            assert (off <= ref.conversion_bound(want, s, False) * (1 + 1e-6) + 2 * (e + 6 * ref.U) * want.abs() + 2.0 ** -126).all()
            largest = ref.quantize(want.float().cpu(), False)[1].double().cuda()
            assert ((s.double() - largest).abs() <= (e + 6 * ref.U) * largest).all()
            assert _only_in(q, q_all) and _only_in(s, s_all)
            rstd = want_rstd.float()
            (dx, dx_all), (far, far_all) = _off(zeros, first, pad), _off(zeros, first + 1, pad + 2)
            t.copy_(total)
            dgamma, again = torch.empty_like(gamma), torch.empty_like(gamma)
            plan.backward(t, gamma, rstd, d, dx, dgamma, dtotal=m)
            plan.backward(t, gamma, rstd, d, far, dtotal=m)
            plan.backward(t, gamma, rstd, d, None, again)
            grad, grad_gamma = ref.rms_backward(total, gamma, rstd, dy, dt)
            bound, bound_gamma = ref.rms_backward_bounds(total, gamma, rstd, dy, dt, elem, weight)
            assert torch.equal(dx, far)
            for got in (dgamma, again):
                assert ((got.double() - grad_gamma).abs() <= bound_gamma).all()
            assert ((dx.double() - grad).abs() <= bound).all()
            plan.backward(t, gamma, rstd, d, d, dtotal=m)
            assert torch.equal(d, dx)
            assert _only_in(dx, dx_all) and _only_in(far, far_all)


@pytest.mark.parametrize("M,N,K", [(400, 4096, 1040), (400, 4104, 512), (300, 9728, 144), (512, 9736, 640), (768, 8192, 272)])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_8_bit_tiles_of_each_width(gemm_lib, M, N, K, out):
    """Two and three rows of tiles by squares, of 128 columns where all run at once, else of 256."""
    a, b = (torch.randn(r, K, generator=torch.Generator().manual_seed(r + K)).to(FP8) for r in (M, N))
    sa, sb = (torch.rand(r, ref.groups(K), generator=torch.Generator().manual_seed(r)) + 0.5 for r in (M, ref.groups(N)))
    whole = torch.full((M + 1, N), 7.0, dtype=T[out], device="cuda")
    with gemm_lib.Fp8Plan(M, N, K, out) as plan:
        plan.run(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), whole[:M])
        plan.check()
    want, bound = ref.fp8_product(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), True)
    assert (whole[M:] == 7).all()
    assert ((whole[:M].double() - want).abs() <= bound + ref.rounded(want, out) * 1.01).all()


@pytest.mark.parametrize("F", [3000, 4096, 4872, 5992, 6008, 7200, 7208, 8400, 8416, 9728])
@pytest.mark.parametrize("elem,act", [("bf16", "silu"), ("f16", "none")])
def test_gated_tiles_of_each_width(gemm_lib, F, elem, act):
    """250 rows are one row of tiles: from 75 tiles of 64 columns to 76 of 128, whole and ragged at the end."""
    M, K = 250, 1032
    X, W = _randn(M, K, seed=F, dtype=T[elem]), _randn(2 * F, K, seed=F + 1, dtype=T[elem], scale=2 * K ** -0.5)
    want, bound, gate_up, off = ref.gated_forward(X, W, act)
    whole, kept_whole = (torch.full((M + 1, n), 7.0, dtype=T[elem], device="cuda") for n in (F, 2 * F))
    with gemm_lib.GatedPlan(M, F, K, elem, act=act) as plan:
        plan.forward(X, W, whole[:M], gate_up=kept_whole[:M])
        plan.check()
        alone = torch.empty(M, F, dtype=T[elem], device="cuda")
        plan.forward(X, W, alone)
        plan.check()
    H, kept = whole[:M], kept_whole[:M]
    assert torch.equal(alone, H) and (whole[M:] == 7).all() and (kept_whole[M:] == 7).all()
    assert ((H.double() - want).abs() <= bound + ref.rounded(want, elem) * 1.01).all()
    assert ((kept.double() - gate_up).abs() <= off + ref.rounded(gate_up, elem) * 1.01).all()
