"""RMS norm with the residual's addition against its 64-bit definition (tests/ffn_oracle.py has the bounds)."""
import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
T = ref.TYPES
FP8 = torch.float8_e4m3fn

SIZES = [(1, 1), (1, 8), (2, 16), (3, 127), (5, 128), (4, 129), (33, 250), (1000, 64), (300, 256), (7, 520), (700, 1000),
         (1, 4096), (160, 4096), (3, 8192), (2, 8200), (2, 16384), (2, 16385), (3, 20001)]
KINDS = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]


def _padded(values, pad, fill=7.0):
    """A device matrix of `values` whose rows stand `pad` elements apart (filled), and the whole of it."""
    rows, cols = values.shape
    whole = torch.full((rows + 1, cols + pad), fill, dtype=values.dtype)
    whole[:rows, :cols] = values
    whole = whole.cuda()
    return whole[:rows, :cols], whole


def _untouched(whole, rows, cols, fill=7.0):
    w = whole.cpu().float()
    assert (w[rows:] == fill).all() and (w[:, cols:] == fill).all()


def _inputs(rows, cols, elem, weight, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(rows, cols).to(T[elem])
    return x, (2 * r(rows, cols)).to(T[elem]) if residual else None, (1 + 0.2 * r(cols)).to(T[weight])


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("elem,weight", KINDS)
def test_forward(gemm_lib, rows, cols, elem, weight):
    for pad, residual in ((0, True), (3, False), (8, True)):
        x, r, gamma = _inputs(rows, cols, elem, weight, rows + cols + pad, residual)
        dx, dr = _padded(x, pad)[0], _padded(r, pad)[0] if residual else None
        y, y_whole = _padded(torch.zeros(rows, cols, dtype=T[elem]), pad)
        t, t_whole = _padded(torch.zeros(rows, cols, dtype=T[elem]), pad)
        rstd = torch.full((rows + 1,), 7.0, device="cuda")
        with gemm_lib.RmsNormPlan(rows + 2, cols, elem, weight=weight) as plan:
            plan.forward(dx, gamma.cuda(), y, rstd[:rows], residual=dr, total=t)
            torch.cuda.synchronize()
        total = ref.rms_total(x, r)
        assert torch.equal(t.cpu(), total)
        want, want_rstd = ref.rms_forward(total, gamma, 1e-5)
        e = ref.rms_error(cols)
        assert ((y.cpu().double() - want).abs() <= 1.01 * (e + 3 * ref.U) * want.abs() + ref.rounded(want, elem)).all()
        assert ((rstd[:rows].cpu().double() - want_rstd).abs() <= e * want_rstd).all()
        assert rstd[rows] == 7
        for w in (y_whole, t_whole):
            _untouched(w, rows, cols)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("elem,weight", KINDS)
def test_forward_fp8(gemm_lib, rows, cols, elem, weight):
    for pad, residual in ((0, True), (3, False), (8, True)):
        x, r, gamma = _inputs(rows, cols, elem, weight, 2 * rows + cols + pad, residual)
        n = ref.groups(cols)
        q, q_whole = _padded(torch.zeros(rows, cols).to(FP8), pad)
        s, s_whole = _padded(torch.zeros(rows, n), 1)
        rstd = torch.empty(rows, device="cuda")
        with gemm_lib.RmsNormPlan(rows, cols, elem, weight=weight) as plan:
            plan.forward_fp8(_padded(x, pad)[0], gamma.cuda(), q, s, rstd, residual=_padded(r, pad)[0] if residual else None)
            torch.cuda.synchronize()
        want, want_rstd = ref.rms_forward(ref.rms_total(x, r), gamma, 1e-5)
        e = ref.rms_error(cols)
        assert ((rstd.cpu().double() - want_rstd).abs() <= e * want_rstd).all()
        scales = s.cpu()
        want_scales = ref.quantize(want.float(), False)[1].double()
        assert ((scales.double() - want_scales).abs() <= (e + 6 * ref.U) * want_scales).all()
        far = (ref.stands_for(q.cpu(), scales, False) - want).abs()
        # y itself is off by e + 3 U, and two more operations lie before the rounding
        assert (far <= ref.conversion_bound(want, scales, False) * (1 + 1e-6) + 2 * (e + 6 * ref.U) * want.abs()).all()
        _untouched(q_whole, rows, cols)
        _untouched(s_whole, rows, n)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("elem,weight", KINDS)
def test_backward(gemm_lib, rows, cols, elem, weight):
    for pad, more in ((0, True), (3, False), (8, True)):
        t, dt, gamma = _inputs(rows, cols, elem, weight, 3 * rows + cols + pad, more)
        g = torch.Generator().manual_seed(rows)
        dy = torch.randn(rows, cols, generator=g).to(T[elem])
        rstd = ref.rms_forward(t, gamma, 1e-5)[1].float()
        dx, dx_whole = _padded(torch.zeros(rows, cols, dtype=T[elem]), pad)
        dgamma = torch.full((cols + 1,), 7.0, dtype=T[weight], device="cuda")
        with gemm_lib.RmsNormPlan(rows, cols, elem, weight=weight) as plan:
            args = (_padded(t, pad)[0], gamma.cuda(), rstd.cuda(), _padded(dy, pad)[0])
            dtotal = _padded(dt, pad)[0] if more else None
            plan.backward(*args, dx, dgamma[:cols], dtotal=dtotal)
            alone = torch.empty_like(dx)
            plan.backward(*args, alone, None, dtotal=dtotal)
            weights = torch.empty_like(dgamma[:cols])
            plan.backward(*args, None, weights)
            torch.cuda.synchronize()
        want, want_dgamma = ref.rms_backward(t, gamma, rstd, dy, dt)
        bound, bound_dgamma = ref.rms_backward_bounds(t, gamma, rstd, dy, dt, elem, weight)
        assert ((dx.cpu().double() - want).abs() <= bound).all()
        assert ((dgamma[:cols].cpu().double() - want_dgamma).abs() <= bound_dgamma).all()
        assert torch.equal(alone, dx) and torch.equal(weights, dgamma[:cols]) and dgamma[cols] == 7
        _untouched(dx_whole, rows, cols)


def test_without_gamma_and_no_rows(gemm_lib):
    x, r, _ = _inputs(5, 200, "bf16", "bf16", 1)
    ones = torch.ones(200)
    with gemm_lib.RmsNormPlan(8, 200, "bf16", weight="f32") as plan:
        y, one = torch.empty(5, 200, dtype=T["bf16"], device="cuda"), torch.empty(5, 200, dtype=T["bf16"], device="cuda")
        plan.forward(x.cuda(), None, y, residual=r.cuda())
        plan.forward(x.cuda(), ones.cuda(), one, residual=r.cuda())
        assert torch.equal(y, one)
        rstd = torch.ones(5, device="cuda")
        plan.backward(x.cuda(), None, rstd, r.cuda(), y)
        plan.backward(x.cuda(), ones.cuda(), rstd, r.cuda(), one)
        assert torch.equal(y, one)
        none, dgamma = torch.empty(0, 200, dtype=T["bf16"], device="cuda"), torch.full((200,), 7.0, device="cuda")
        plan.forward(none, ones.cuda(), none)
        plan.backward(none, ones.cuda(), rstd[:0], none, none, dgamma)
        assert (dgamma == 0).all()


@pytest.mark.parametrize("cols", [192, 4096, 4100, 20000])
def test_in_place(gemm_lib, cols):
    x, r, gamma = (v.cuda() for v in _inputs(37, cols, "bf16", "bf16", cols))
    new = lambda: torch.empty_like(x)  # noqa: E731
    with gemm_lib.RmsNormPlan(37, cols, "bf16") as plan:
        y, t, rstd, dx, dgamma = new(), new(), torch.empty(37, device="cuda"), new(), torch.empty_like(gamma)
        plan.forward(x, gamma, y, rstd, residual=r, total=t)
        for total_is_x in (True, False):
            a, b = x.clone(), r.clone()
            total, out = (a, b) if total_is_x else (b, a)
            plan.forward(a, gamma, out, rstd, residual=b, total=total)
            assert torch.equal(total, t) and torch.equal(out, y)
        q, s, q2, s2 = (v for _ in range(2) for v in (torch.empty(37, cols, dtype=FP8, device="cuda"),
                                                      torch.empty(37, ref.groups(cols), device="cuda")))
        plan.forward_fp8(x, gamma, q, s, residual=r, total=new())
        a, b = x.clone(), r.clone()
        plan.forward_fp8(a, gamma, q2, s2, residual=b, total=b)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
        dy, dt = x * 0.5, r * 0.25
        plan.backward(t, gamma, rstd, dy, dx, dgamma, dtotal=dt)
        for which in range(3):
            args, again = [t.clone(), dy.clone(), dt.clone()], torch.empty_like(gamma)
            plan.backward(args[0], gamma, rstd, args[1], args[which], again, dtotal=args[2])
            assert torch.equal(args[which], dx) and torch.equal(again, dgamma)


def test_another_stream_and_a_graph(gemm_lib):
    x, r, gamma = (v.cuda() for v in _inputs(50, 1000, "f16", "f32", 3))
    new = lambda: torch.empty_like(x)  # noqa: E731
    y, t, rstd, dx, dgamma, q = new(), new(), torch.empty(50, device="cuda"), new(), torch.empty_like(gamma), None
    q, s = torch.empty(50, 1000, dtype=FP8, device="cuda"), torch.empty(50, 8, device="cuda")
    side = torch.cuda.Stream()
    with gemm_lib.RmsNormPlan(50, 1000, "f16", weight="f32") as plan:
        def step(stream):
            plan.forward(x, gamma, y, rstd, residual=r, total=t, stream=stream)
            plan.forward_fp8(x, gamma, q, s, residual=r, total=t, stream=stream)
            plan.backward(t, gamma, rstd, y, dx, dgamma, stream=stream)
        torch.cuda.synchronize()
        step(side)
        side.synchronize()
        want = [v.clone() for v in (y, t, rstd, dx, dgamma, s)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(None)
        for v in (y, t, rstd, dx, dgamma, s):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip((y, t, rstd, dx, dgamma, s), want):
            assert torch.equal(v, w)


def test_nan_and_infinity_stay_in_their_rows(gemm_lib):
    x, _, gamma = _inputs(6, 300, "f32", "f32", 4, False)
    x[1, 5], x[2, 7], x[3] = float("nan"), float("inf"), 0
    y = torch.empty(6, 300, device="cuda")
    with gemm_lib.RmsNormPlan(6, 300, "f32") as plan:
        plan.forward(x.cuda(), gamma.cuda(), y)
    y = y.cpu()
    assert y[1].isnan().all() and y[2, 7].isnan() and (y[2, :7] == 0).all() and (y[3] == 0).all()
    want = ref.rms_forward(x[[0, 4, 5]], gamma, 1e-5)[0]
    assert ((y[[0, 4, 5]].double() - want).abs() <= 1.01 * (ref.rms_error(300) + 4 * ref.U) * want.abs()).all()


def test_refusals(gemm_lib):
    x = torch.zeros(4, 64, dtype=T["bf16"], device="cuda")
    gamma, q, s = torch.ones(64, dtype=T["bf16"], device="cuda"), torch.zeros(4, 64, dtype=FP8, device="cuda"), torch.ones(4, 1, device="cuda")
    rstd = torch.ones(4, device="cuda")
    with gemm_lib.RmsNormPlan(4, 64, "bf16") as plan:
        def refused(call, status):
            with pytest.raises(gemm_lib.GemmError) as e:
                call()
            assert e.value.status == status
        refused(lambda: plan.forward(x.float(), gamma, x), 2)
        refused(lambda: plan.forward(x, gamma.float(), x), 2)
        refused(lambda: plan.forward(x, gamma, x.t()), 1)
        refused(lambda: plan.forward(x[:, :63], gamma, x), 1)
        refused(lambda: plan.forward(x, gamma[:63], x), 1)
        refused(lambda: plan.forward(x.cpu(), gamma, x), 1)
        refused(lambda: plan.forward(x, gamma, x, residual=x[:3]), 1)
        refused(lambda: plan.forward(x, gamma, x, total=x), 1)                 # y and total are one matrix
        refused(lambda: plan.forward(x, gamma, x, eps=-1.0), 1)
        refused(lambda: plan.forward(x, gamma, x, eps=float("nan")), 1)
        refused(lambda: plan.forward(x, gamma, x, rstd[:3]), 1)
        refused(lambda: plan.forward_fp8(x, gamma, q.view(torch.uint8), s), 2)
        refused(lambda: plan.forward_fp8(x, gamma, q[:, :32], s), 1)
        refused(lambda: plan.forward_fp8(x, gamma, q, s[:3]), 1)
        refused(lambda: plan.forward_fp8(x, gamma, q, s.half()), 2)
        refused(lambda: plan.backward(x, gamma, None, x, x), 1)
        refused(lambda: plan.backward(x, gamma, rstd, x[:, :60], x), 1)
        refused(lambda: plan.backward(x, gamma, rstd, x, x, gamma.float()), 2)
        big = torch.zeros(5, 64, dtype=T["bf16"], device="cuda")
        refused(lambda: plan.forward(big, gamma, big), 1)
        overlap = x.as_strided((4, 64), (60, 1))
        refused(lambda: plan.forward(overlap, gamma, x), 1)
