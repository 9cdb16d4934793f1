"""Embedding, layer norm and distillation on the GPU against their 64-bit definitions
(train_oracle.py, whose bounds are derived there), at the sizes, strides and masks where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

import train_oracle as to

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, want, bound, what):
    got = _f64(got) if isinstance(got, torch.Tensor) else got
    with np.errstate(invalid="ignore"):
        err = np.abs(got - want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))     # infinities and NaN where they belong
    bad = ~(same | (err <= bound))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside the bound; first at %s: %r, wanted %r +- %r"
                             % (what, bad.sum(), bad.size, i, got[i], want[i], np.broadcast_to(bound, got.shape)[i]))


def _rows(value, elem, pad=0, offset=0):
    """A device matrix of the type with rows `pad` elements further apart, starting `offset`
    elements into its memory; the rest of the memory holds a canary."""
    rows, cols = value.shape
    flat = torch.full((offset + rows * (cols + pad) + 8,), 99.0, dtype=TYPES[elem], device="cuda")
    m = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.as_tensor(value))
    m.flat = flat
    return m


def _canary_whole(m):
    flat, keep = m.flat.clone(), torch.ones_like(m.flat, dtype=torch.bool)
    rows, cols = m.shape
    off = (m.data_ptr() - m.flat.data_ptr()) // m.element_size()
    idx = off + torch.arange(rows, device="cuda")[:, None] * m.stride(0) + torch.arange(cols, device="cuda")
    keep[idx.reshape(-1)] = False
    assert bool((flat[keep] == 99.0).all()), "memory outside the matrix was written"


# ---------------------------------------------------------------- layer norm

NORM_SIZES = [(1, 1), (1, 2), (3, 7), (5, 8), (2, 31), (33, 32), (7, 100), (4, 250), (17, 256), (9, 511), (300, 96),
              (5, 1000), (3, 1024), (700, 72), (2, 1031), (6, 2048), (3, 2056), (4, 4096), (310, 1024), (2, 4100),
              (5, 5000), (3, 8192), (2, 8200), (3, 16384), (2, 16385), (2, 20000), (1, 40001),
              (10000, 256), (5200, 1000), (2500, 1032), (1300, 4096), (700, 8192), (650, 12000), (320, 16384)]


def _norm_case(rows, cols, elem, weight, pad, offset, seed=0):
    rng = np.random.default_rng(rows * 100003 + cols + seed)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=cols)) + rng.normal()
    if rows > 2:
        x[1] = 0.75                                          # a row without variance
    return {"x": _rows(x, elem, pad, offset), "dy": _rows(rng.normal(size=(rows, cols)), elem, pad, offset),
            "gamma": torch.as_tensor(rng.normal(size=cols) + 1).to("cuda", TYPES[weight]),
            "beta": torch.as_tensor(rng.normal(size=cols)).to("cuda", TYPES[weight]),
            "y": _rows(np.zeros((rows, cols)), elem, pad, offset),
            "dx": _rows(np.zeros((rows, cols)), elem, pad, offset),
            "mean": torch.full((rows,), 7.0, device="cuda"), "rstd": torch.full((rows,), 7.0, device="cuda"),
            "dgamma": torch.full((cols,), 7.0, dtype=TYPES[weight], device="cuda"),
            "dbeta": torch.full((cols,), 7.0, dtype=TYPES[weight], device="cuda")}


def _check_norm(c, elem, weight, eps=1e-5):
    x, gamma, beta = _f64(c["x"]), _f64(c["gamma"]), _f64(c["beta"])
    y, mean, rstd = to.norm_forward(x, gamma, beta, eps)
    by, bm, br = to.norm_forward_bounds(x, gamma, beta, eps, elem)
    _within(c["mean"], mean, bm, "mean")
    _within(c["rstd"], rstd, br, "rstd")
    _within(c["y"], y, by, "y")
    mean, rstd, dy = _f64(c["mean"]), _f64(c["rstd"]), _f64(c["dy"])
    want = to.norm_backward(x, gamma, mean, rstd, dy)
    bound = to.norm_backward_bounds(x, gamma, mean, rstd, dy, elem, weight)
    for k, name in enumerate(("dx", "dgamma", "dbeta")):
        _within(c[name], want[k], bound[k], name)


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("elem,weight,pad,offset", [("bf16", "bf16", 0, 0), ("f16", "f32", 3, 1), ("f32", "f32", 4, 0),
                                                    ("bf16", "f32", 8, 8), ("f16", "f16", 0, 1), ("f32", "f32", 1, 3)])
def test_norm(gemm_lib, rows, cols, elem, weight, pad, offset):
    c = _norm_case(rows, cols, elem, weight, pad, offset)
    with gemm_lib.NormPlan(rows + 3, cols, elem, weight=weight) as plan:
        plan.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"])
        plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"], c["dbeta"])
        torch.cuda.synchronize()
        _check_norm(c, elem, weight)
        _canary_whole(c["y"])
        _canary_whole(c["dx"])
        # the same inputs give the same bits
        first = [c[k].clone() for k in ("y", "dx", "dgamma", "dbeta")]
        plan.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"])
        plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"], c["dbeta"])
        assert all(torch.equal(a, c[k]) for a, k in zip(first, ("y", "dx", "dgamma", "dbeta")))


@pytest.mark.parametrize("rows,cols", [(10003, 259), (5003, 1003), (2511, 2049), (1301, 4090), (661, 8185), (331, 16377),
                                       (1300, 1003), (320, 4099), (165, 8190)])
@pytest.mark.parametrize("elem,weight", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_norm_rows_off_boundaries(gemm_lib, rows, cols, elem, weight):
    """Contiguous rows of odd lengths, each of which begins inside its neighbour's last 16 bytes."""
    c = _norm_case(rows, cols, elem, weight, 0, 0, seed=3)
    with gemm_lib.NormPlan(rows, cols, elem, weight=weight) as plan:
        def run(x, dy, y, dx):
            plan.forward(x, c["gamma"], c["beta"], y, c["mean"], c["rstd"])
            plan.backward(x, c["gamma"], c["mean"], c["rstd"], dy, dx, c["dgamma"], c["dbeta"])
        run(c["x"], c["dy"], c["y"], c["dx"])
        torch.cuda.synchronize()
        _check_norm(c, elem, weight)
        _canary_whole(c["y"])
        _canary_whole(c["dx"])
        y, dx = c["y"].clone(), c["dx"].clone()
        # in place, the same bits
        over = c["x"].clone()
        plan.forward(over, c["gamma"], c["beta"], over)
        assert torch.equal(over, y)
        over = c["dy"].clone()
        plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], over, over)
        assert torch.equal(over, dx)
        # results at other offsets than the inputs': right as well
        c["y"], c["dx"] = (_rows(np.zeros((rows, cols)), elem, 2, 1) for _ in range(2))
        run(c["x"], c["dy"], c["y"], c["dx"])
        torch.cuda.synchronize()
        _check_norm(c, elem, weight)
        # a row's bad values at its ends stay out of its neighbours
        bad = [0, 7, 160, rows - 1]
        clean = torch.ones(rows, dtype=torch.bool, device="cuda")
        clean[bad] = False
        for r, at in zip(bad, (-1, 0, -1, 0)):
            c["x"][r, at] = math.nan
        c["dy"][7, -1] = math.inf
        run(c["x"], c["dy"], y, dx)
        for name, t in (("y", y), ("dx", dx)):
            assert bool(torch.isfinite(t[clean]).all()), name
            assert not bool(torch.isfinite(t[~clean]).any(dim=1).any()), name


@pytest.mark.parametrize("rows,cols", [(5, 64), (37, 1000), (3, 4096), (2, 16400)])
def test_norm_parts(gemm_lib, rows, cols):
    """Without gamma, beta or statistics; each gradient alone; results in place."""
    c = _norm_case(rows, cols, "bf16", "f32", 0, 0, seed=1)
    ones, zeros = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    with gemm_lib.NormPlan(rows, cols, "bf16", weight="f32") as plan:
        want = torch.empty_like(c["y"])
        plan.forward(c["x"], ones, zeros, want, c["mean"], c["rstd"])
        plan.forward(c["x"], None, None, c["y"])
        assert torch.equal(c["y"], want)
        same = c["x"].clone()
        plan.forward(same, ones, zeros, same)
        assert torch.equal(same, want)
        args = (c["x"], c["gamma"], c["mean"], c["rstd"])
        plan.backward(*args, c["dy"], c["dx"], c["dgamma"], c["dbeta"])
        alone = {"dx": torch.empty_like(c["dx"]), "dgamma": torch.empty_like(c["dgamma"]),
                 "dbeta": torch.empty_like(c["dbeta"])}
        for name, t in alone.items():
            plan.backward(*args, c["dy"], **{name: t})
            assert torch.equal(t, c[name]), name
        for src in ("dy", "x"):
            over = {"dy": c["dy"].clone(), "x": c["x"].clone()}
            dg, db = torch.empty_like(c["dgamma"]), torch.empty_like(c["dbeta"])
            plan.backward(over["x"], c["gamma"], c["mean"], c["rstd"], over["dy"], over[src], dg, db)
            assert torch.equal(over[src], c["dx"]) and torch.equal(dg, c["dgamma"]) and torch.equal(db, c["dbeta"])
        plan.backward(c["x"][:0], c["gamma"], c["mean"][:0], c["rstd"][:0], c["dy"][:0], c["dx"][:0], c["dgamma"],
                      c["dbeta"])
        assert not c["dgamma"].any() and not c["dbeta"].any()
        plan.forward(c["x"][:0], None, None, c["y"][:0])


@pytest.mark.parametrize("cols", [40, 1000, 4096, 17000])
def test_norm_bad_values_stay_in_their_row(gemm_lib, cols):
    rows = 40
    c = _norm_case(rows, cols, "bf16", "bf16", 0, 0, seed=2)
    c["x"][3, 5], c["x"][17, 0], c["dy"][29, 39] = math.nan, math.inf, math.nan
    with gemm_lib.NormPlan(rows, cols, "bf16") as plan:
        plan.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"])
        plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"])
    bad = {"y": [3, 17], "dx": [3, 17, 29]}
    for name, rows_bad in bad.items():
        clean = torch.ones(rows, dtype=torch.bool, device="cuda")
        clean[rows_bad] = False
        assert bool(torch.isfinite(c[name][clean]).all()), name
        for r in rows_bad:
            assert not bool(torch.isfinite(c[name][r]).all()), (name, r)


def test_norm_large_mean(gemm_lib):
    """Rows far from zero: the variance is taken about the mean, not from the squares' sum."""
    rng = np.random.default_rng(6)
    x = torch.as_tensor(rng.normal(size=(6, 4096)) + 1000).float().cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    with gemm_lib.NormPlan(6, 4096, "f32") as plan:
        plan.forward(x, None, None, y, mean, rstd)
    one, zero = np.ones(4096), np.zeros(4096)
    want = to.norm_forward(_f64(x), one, zero, 1e-5)
    bound = to.norm_forward_bounds(_f64(x), one, zero, 1e-5, "f32")
    for got, w, b, name in zip((y, mean, rstd), want, bound, ("y", "mean", "rstd")):
        _within(got, w, b, name)


def test_norm_gradient_against_differences(gemm_lib):
    """sum(dy * y) of the kernel's fp32 forward, moved along random directions, against dx, dgamma and dbeta.
    Rounding: the forward is within its bound of the exact one, so a difference over 2h is off by at most
    sum(|dy| bound) / h; the exact curve's third derivative adds about h^2 (h = 2^-7, values near 1)."""
    rng = np.random.default_rng(7)
    rows, cols, h = 5, 200, 2.0 ** -7
    x, dy = rng.normal(size=(rows, cols)).astype(np.float32), rng.normal(size=(rows, cols)).astype(np.float32)
    gamma, beta = (rng.normal(size=cols).astype(np.float32) for _ in range(2))
    t = lambda v: torch.as_tensor(v, dtype=torch.float32).cuda()  # noqa: E731
    with gemm_lib.NormPlan(rows, cols, "f32") as plan:
        def f(xx, gg, bb):
            y = torch.empty(rows, cols, device="cuda")
            plan.forward(t(xx), t(gg), t(bb), y, mean, rstd)
            return (_f64(y) * dy).sum()
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        f(x, gamma, beta)
        dx, dg, db = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        plan.backward(t(x), t(gamma), mean, rstd, t(dy), dx, dg, db)
        noise = (np.abs(dy) * to.norm_forward_bounds(x.astype(float), gamma, beta, 1e-5, "f32")[0]).sum() / h
        for _ in range(3):
            u, w, v = rng.choice([-1.0, 1.0], size=x.shape), rng.choice([-1.0, 1.0], size=cols), rng.choice([-1.0, 1.0], size=cols)
            for diff, want, size in (
                    ((f(x + h * u, gamma, beta) - f(x - h * u, gamma, beta)) / (2 * h), (_f64(dx) * u).sum(), np.abs(_f64(dx)).sum()),
                    ((f(x, gamma + h * w, beta) - f(x, gamma - h * w, beta)) / (2 * h), (_f64(dg) * w).sum(), np.abs(_f64(dg)).sum()),
                    ((f(x, gamma, beta + h * v) - f(x, gamma, beta - h * v)) / (2 * h), (_f64(db) * v).sum(), np.abs(_f64(db)).sum())):
                # x +- h u rounds to fp32 (2^-24 of x over h of it), and the curve bends by up to ~ size * h^2 * 8
                assert abs(diff - want) <= 2 * noise + size * (8 * h * h + 2.0 ** -22 / h)


# ---------------------------------------------------------------- embedding

EMBED_SIZES = [(1, 1, 1), (1, 5, 8), (3, 2, 7), (40, 3, 33), (64, 1000, 64), (257, 16, 100), (1000, 50, 256),
               (1025, 5000, 24), (33, 70000, 40), (2048, 1, 72), (2500, 300, 1032), (100, 100, 4100), (5000, 40, 16),
               (9000, 30011, 8)]


def _embed_case(n, vocab, dim, elem, grad, index, pad, offset):
    rng = np.random.default_rng(n * 1009 + vocab * 7 + dim)
    ids = np.minimum((vocab + 1) ** rng.random(n) - 1, vocab - 1).astype(np.int64)
    if n > 4:
        ids[rng.random(n) < 0.1] = -1
    return {"ids": torch.as_tensor(ids).to("cuda", torch.int32 if index == "i32" else torch.int64),
            "table": _rows(rng.normal(size=(vocab, dim)), elem, pad, offset),
            "out": _rows(np.zeros((n, dim)), elem, pad, offset),
            "dout": _rows(rng.normal(size=(n, dim)), elem, pad, offset),
            "dtable": _rows(rng.normal(size=(vocab, dim)), grad, pad, offset)}


@pytest.mark.parametrize("elem,n,dim", [("bf16", 4865, 8200), ("f16", 4866, 4104), ("f32", 4867, 4100), ("f32", 9731, 1500),
                                        ("bf16", 38915, 300), ("bf16", 155651, 128), ("f16", 19459, 97),
                                        ("bf16", 9730, 2080), ("f32", 77826, 60)])
def test_lookup_of_many_tokens(gemm_lib, elem, n, dim):
    """Token counts that leave the last group of tokens incomplete, rows of several steps: every element."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randn(700, dim, generator=gen, device="cuda").to(TYPES[elem])
    ids = torch.randint(0, 700, (n,), generator=gen, device="cuda")
    out = torch.full((n + 1, dim), 99.0, dtype=TYPES[elem], device="cuda")
    with gemm_lib.EmbedPlan(700, dim, n, elem) as plan:
        plan.forward(ids, table, out[:n], scale=2.0)
    assert torch.equal(out[:n], 2 * table[ids])
    assert bool((out[n] == 99).all())


@pytest.mark.parametrize("n,vocab,dim", EMBED_SIZES)
@pytest.mark.parametrize("elem,grad,index,pad,offset", [("bf16", "bf16", "i64", 0, 0), ("f16", "f32", "i32", 3, 1),
                                                        ("f32", "f32", "i32", 0, 0), ("bf16", "f32", "i64", 8, 8),
                                                        ("f16", "f16", "i32", 1, 0)])
def test_embedding(gemm_lib, n, vocab, dim, elem, grad, index, pad, offset):
    c = _embed_case(n, vocab, dim, elem, grad, index, pad, offset)
    ids, scale = c["ids"].cpu().numpy(), float(np.float32(math.sqrt(dim) / 3))
    start = _f64(c["dtable"])
    with gemm_lib.EmbedPlan(vocab, dim, n + 5, elem, grad=grad) as plan:
        plan.forward(c["ids"], c["table"], c["out"], scale=scale)
        want = to.embed_forward(ids, -1, _f64(c["table"]), scale)
        _within(c["out"], want, to.rounded(want, elem) + to.U * np.abs(want), "out")
        for accumulate in (True, False):
            plan.backward(c["ids"], c["dout"], c["dtable"], scale=scale, accumulate=accumulate)
            want, bound = to.embed_backward(ids, -1, _f64(c["dout"]), scale, vocab, start if accumulate else None)
            _within(c["dtable"], want, bound + to.rounded(want, grad), "dtable %s" % accumulate)
        first = c["dtable"].clone()
        plan.backward(c["ids"], c["dout"], c["dtable"], scale=scale)
        assert torch.equal(first, c["dtable"])
        for name in ("out", "dtable"):
            _canary_whole(c[name])
        plan.check()


def test_embedding_untouched_rows(gemm_lib):
    """Accumulation leaves rows without a token as they are, NaN and infinities too."""
    vocab, dim = 500, 136
    dtable = torch.full((vocab, dim), math.nan, device="cuda")
    ids = torch.tensor([3, 77, 3, 499], device="cuda")
    dtable[[3, 77, 499]] = 1.0
    dout = torch.ones(4, dim, dtype=torch.bfloat16, device="cuda")
    with gemm_lib.EmbedPlan(vocab, dim, 4, "bf16", grad="f32") as plan:
        plan.backward(ids, dout, dtable, accumulate=True)
    want = torch.full((vocab, dim), math.nan, device="cuda")
    want[3], want[77], want[499] = 3.0, 2.0, 2.0
    assert torch.equal(torch.nan_to_num(want, 5.0), torch.nan_to_num(dtable, 5.0))


@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_without_tokens(gemm_lib, accumulate):
    dtable = torch.full((70, 24), 3.0, dtype=torch.float16, device="cuda")
    with gemm_lib.EmbedPlan(70, 24, 40, "f16") as plan:
        none = torch.empty(0, 24, dtype=torch.float16, device="cuda")
        plan.forward(torch.empty(0, dtype=torch.int64, device="cuda"), dtable, none)
        plan.backward(torch.empty(0, dtype=torch.int64, device="cuda"), none, dtable, accumulate=accumulate)
        assert bool((dtable == (3.0 if accumulate else 0.0)).all())
        dtable.fill_(3.0)      # nothing but padding
        plan.backward(torch.full((40,), 9, device="cuda"), torch.ones(40, 24, dtype=torch.float16, device="cuda"),
                      dtable, padding=9, accumulate=accumulate)
        assert bool((dtable == (3.0 if accumulate else 0.0)).all())
        plan.check()


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_embedding_ids_outside_the_table(gemm_lib, index):
    vocab, dim = 100, 64
    ids = torch.tensor([5, 100, -2, 7, -1, 5], device="cuda").to(index)
    if index == torch.int64:
        ids[1] = (1 << 32) + 3           # would be 3 in 32 bits
    table = torch.randn(vocab, dim, device="cuda")
    out, dtable = torch.full((6, dim), 9.0, device="cuda"), torch.empty(vocab, dim, device="cuda")
    with gemm_lib.EmbedPlan(vocab, dim, 6, "f32") as plan:
        for call in (lambda: plan.forward(ids, table, out), lambda: plan.backward(ids, table[:6], dtable)):
            call()
            with pytest.raises(gemm_lib.GemmError) as e:
                plan.check()
            assert e.value.status == 12
            plan.check()                 # reported once
    want = torch.zeros(6, dim, device="cuda")
    want[[0, 3, 5]] = table[[5, 7, 5]]
    assert torch.equal(out, want)
    grad = torch.zeros(vocab, dim, device="cuda")
    grad[5], grad[7] = table[0] + table[5], table[3]
    assert torch.equal(grad, dtable)


def test_embedding_one_token_many_times(gemm_lib):
    """A whole batch of the same token, and two tokens in turn: long sums, exact in small integers."""
    n, dim = 20000, 24
    dout = (torch.arange(n, device="cuda")[:, None] % 7 - 3).float().repeat(1, dim).contiguous()
    with gemm_lib.EmbedPlan(300, dim, n, "f32") as plan:
        dtable = torch.empty(300, dim, device="cuda")
        for ids in (torch.full((n,), 123, device="cuda"), 123 + (torch.arange(n, device="cuda") % 2)):
            plan.backward(ids, dout, dtable)
            want = torch.zeros(300, dim, device="cuda").index_add_(0, ids, dout)
            assert torch.equal(dtable, want)


@pytest.mark.parametrize("dim,scale_up", [(8, 1), (4096, 1), (8192, 1), (8192, 2), (4095, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_runs_of_every_length(gemm_lib, dim, scale_up, accumulate):
    """Tokens that come 1 to 70 times each, in several orders of the lengths (so that runs of every length begin and
    end at every place of the kernels' chunks, whose size depends on tokens and columns), exact in small integers."""
    lengths = np.concatenate([np.arange(1, 35), np.arange(70, 1, -3), [8, 8, 16, 7, 9, 32, 31, 33, 1, 1, 64, 65, 2]])
    lengths = np.tile(lengths, scale_up)
    vocab = len(lengths) + 2
    rng = np.random.default_rng(dim + scale_up)
    with gemm_lib.EmbedPlan(vocab, dim, int(lengths.sum()) + 5, "bf16", grad="f32") as plan:
        for _ in range(3):
            ids = np.concatenate([np.repeat(np.arange(len(lengths)) + 1, lengths), [-1] * 5])
            rng.shuffle(ids)
            rng.shuffle(lengths)
            ids = torch.as_tensor(ids).cuda()
            dout = torch.randint(-2, 3, (len(ids), dim), device="cuda").bfloat16()
            dtable = torch.randint(-2, 3, (vocab, dim), device="cuda").float()
            want = dtable.clone() if accumulate else torch.zeros_like(dtable)
            there = ids >= 0
            want.index_add_(0, ids[there], dout[there].float())
            plan.backward(ids, dout, dtable, accumulate=accumulate)
            assert torch.equal(dtable, want)


@pytest.mark.parametrize("n", [1000, 4097, 9000, 33000, 70001])
def test_embedding_sorts_any_number_of_tokens(gemm_lib, n):
    """From one sorting block to several tiles of a cluster's blocks; 1 to 4 passes over the ids' digits."""
    for vocab in (300, 70000, 1 << 20):
        gen = torch.Generator(device="cuda").manual_seed(n)
        ids = torch.randint(vocab, (n,), generator=gen, device="cuda")
        dout = torch.randint(-2, 3, (n, 8), generator=gen, device="cuda").float()
        dtable = torch.full((vocab, 8), 7.0, device="cuda")
        with gemm_lib.EmbedPlan(vocab, 8, n, "f32") as plan:
            plan.backward(ids, dout, dtable)
        assert torch.equal(dtable, torch.zeros_like(dtable).index_add_(0, ids, dout))


# ---------------------------------------------------------------- distillation

DISTILL_SIZES = [(1, 1, 1), (1, 8, 3), (3, 7, 7), (5, 100, 1), (2, 1000, 64), (40, 333, 20), (3, 4096, 200), (2, 8200, 33),
                 (7, 20011, 16), (2, 50021, 1024), (1, 131072, 64), (400, 136, 5), (2, 300000, 8),
                 (1, 850000, 4), (1000, 333, 20), (600, 4500, 7), (480, 20011, 9), (160, 66000, 64)]


def _distill_case(rows, vocab, top, elem, value, index, pad, offset, given, tau, mask=True):
    rng = np.random.default_rng(rows * 17 + vocab * 3 + top)
    top = min(top, vocab)
    ids = np.stack([rng.permutation(vocab)[:top] for _ in range(rows)]) if vocab <= 60000 else \
        (rng.integers(vocab, size=(rows, 1)) + np.arange(top) * (vocab // top)) % vocab
    logits = rng.normal(size=(rows, vocab)) * 2
    values = rng.normal(size=(rows, top)) + 3
    if rows > 2 and mask:
        ids[1] = -1                                     # a row without entries
        ids[2, top // 2:] = -1                          # a row with fewer
    if vocab > 50 and mask:
        free = np.ones(vocab, bool)
        free[ids[ids >= 0]] = False
        logits[:, np.flatnonzero(free)[::7]] = -np.inf  # masked tokens
    c = {"logits": _rows(logits, elem, pad, offset), "values": _rows(values, value, 1, 1),
         "ids": torch.as_tensor(ids).to("cuda", torch.int32 if index == "i32" else torch.int64),
         "dlogits": _rows(np.zeros((rows, vocab)), elem, pad, offset), "given": None,
         "loss": torch.full((rows,), 7.0, device="cuda"), "lse": torch.full((rows,), 7.0, device="cuda"),
         "dloss": torch.as_tensor(rng.uniform(0.5, 2, size=rows)).float().cuda()}
    if given:
        c["given"] = torch.as_tensor(np.log(np.exp(values / tau).sum(1)) + rng.uniform(0, 0.3, size=rows)).float().cuda()
    return c


def _check_distill(c, elem, tau, dloss=True, what=""):
    args = (_f64(c["logits"]), c["ids"].cpu().numpy().astype(np.int64), _f64(c["values"]), tau)
    more = {"teacher_lse": None if c["given"] is None else _f64(c["given"]), "dloss": _f64(c["dloss"]) if dloss else None}
    want = to.distill(*args, **more)
    bound = to.distill_bounds(*args, elem, **more)
    for k, name in enumerate(("loss", "lse", "dlogits")):
        _within(c[name], want[k], bound[k], what + name)


@pytest.mark.parametrize("rows,vocab,top", DISTILL_SIZES)
@pytest.mark.parametrize("elem,value,index,pad,offset,given,tau", [
    ("bf16", "f32", "i64", 0, 0, False, 1.0), ("f16", "f16", "i32", 3, 1, True, 2.0), ("f32", "f32", "i32", 0, 0, True, 0.7),
    ("bf16", "bf16", "i64", 8, 8, True, 1.0), ("f32", "bf16", "i64", 5, 3, False, 4.0)])
def test_distillation(gemm_lib, rows, vocab, top, elem, value, index, pad, offset, given, tau):
    c = _distill_case(rows, vocab, top, elem, value, index, pad, offset, given, tau)
    more = {"temperature": tau, "teacher_lse": c["given"]}
    tau = float(np.float32(tau))
    with gemm_lib.DistillPlan(rows + 2, vocab, c["ids"].shape[1], elem) as plan:
        plan.forward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], **more)
        plan.backward(c["logits"], c["ids"], c["values"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
        _check_distill(c, elem, tau)
        _canary_whole(c["dlogits"])
        first = {k: c[k].clone() for k in ("loss", "lse", "dlogits")}
        for k in first:
            c[k].fill_(5.0)
        plan.forward_backward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
        _check_distill(c, elem, tau, what="both: ")
        _canary_whole(c["dlogits"])
        again = {k: c[k].clone() for k in first}
        plan.forward_backward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
        assert all(torch.equal(again[k], c[k]) for k in again)
        plan.check()


@pytest.mark.parametrize("rows,vocab", [(6, 24), (6, 1000), (6, 50000), (6, 150001), (700, 1000), (500, 9001), (160, 70000)])
@pytest.mark.parametrize("call", ["backward", "forward_backward"])
def test_distillation_in_place_and_without_dloss(gemm_lib, rows, vocab, call):
    c = _distill_case(rows, vocab, 9, "bf16", "f32", "i32", 0, 0, False, 1.5)
    with gemm_lib.DistillPlan(rows, vocab, 9, "bf16") as plan:
        over = c["logits"].clone()
        if call == "backward":
            plan.forward(over, c["ids"], c["values"], c["loss"], c["lse"], temperature=1.5)
            plan.backward(over, c["ids"], c["values"], c["lse"], over, temperature=1.5)
        else:
            plan.forward_backward(over, c["ids"], c["values"], c["loss"], c["lse"], over, temperature=1.5)
        c["dlogits"] = over
        _check_distill(c, "bf16", 1.5, dloss=False)


@pytest.mark.parametrize("vocab,times", [(40, 1), (3000, 1), (70000, 1), (40, 100), (1003, 60), (17000, 30)])
def test_distillation_odd_rows(gemm_lib, vocab, times):
    """Rows whose masks leave nothing, infinities and NaN, equal ids: each stays in its row."""
    c = _distill_case(9, vocab, 6, "f32", "f32", "i64", 0, 0, False, 1.0, mask=False)
    ids, values, logits = c["ids"], c["values"], c["logits"]
    logits[0] = -math.inf                  # no token at all
    values[1] = -math.inf                  # no teacher mass
    ids[2] = -1                            # no entries
    logits[2, 3] = math.nan                # ... whose logits do not matter
    logits[3] = -math.inf
    logits[3, ids[3, 0]] = 2.0             # one token left: probability one
    ids[3, 1:] = -1
    ids[4, 3] = ids[4, 0]                  # equal ids add
    ids[4, 5] = ids[4, 0]
    values[5, 2] = -math.inf               # an entry without probability
    logits[5, ids[5, 2]] = -math.inf
    logits[6, 1] = math.nan
    logits[7, :] = torch.finfo(torch.float32).min
    logits[7, ids[7, 0]] = 0.0             # a mask of the type's lowest value
    ids[7, 1:] = -1
    for k in ("loss", "lse", "dlogits", "logits", "ids", "values", "dloss"):     # the same rows many times
        c[k] = c[k].repeat(times, *[1] * (c[k].dim() - 1))
    ids, values, logits = c["ids"], c["values"], c["logits"]
    with gemm_lib.DistillPlan(9 * times, vocab, 6, "f32") as plan:
        for both in (False, True):
            for k in ("loss", "lse", "dlogits"):
                c[k].fill_(5.0)
            if both:
                plan.forward_backward(logits, ids, values, c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"])
            else:
                plan.forward(logits, ids, values, c["loss"], c["lse"])
                plan.backward(logits, ids, values, c["lse"], c["dlogits"], dloss=c["dloss"])
            loss, lse, grad = (c[k].clone() for k in ("loss", "lse", "dlogits"))
            for r in (0, 1, 2):
                assert not bool(loss[r::9].any()) and bool((lse[r::9] == -math.inf).all()) and not bool(grad[r::9].any()), r
            for r in (3, 7):
                assert bool((loss[r::9].abs() < 1e-6).all()) and not bool((grad[r::9].abs() > 1e-6).any()), r
            assert all(bool(torch.isnan(t[6::9]).all()) for t in (loss, lse, grad))
            some = torch.tensor([r for r in range(9 * times) if r % 9 in (4, 5, 8)], device="cuda")
            part = {k: c[k][some] for k in ("logits", "ids", "values", "dloss", "loss", "lse", "dlogits")}
            part["given"] = None
            _check_distill(part, "f32", 1.0, what="both %s: " % both)


def test_distillation_masked_token_with_teacher_mass(gemm_lib):
    """A token the teacher wants and the student masks: infinite loss, finite gradient."""
    logits = torch.tensor([[0.0, -math.inf, 1.0, 2.0]], device="cuda")
    ids, values = torch.tensor([[1, 3]], device="cuda"), torch.tensor([[1.0, 1.0]], device="cuda")
    loss, lse, grad = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
    with gemm_lib.DistillPlan(1, 4, 2, "f32") as plan:
        plan.forward_backward(logits, ids, values, loss, lse, grad)
    q = torch.softmax(logits, 1)
    assert loss.item() == math.inf
    want = q - torch.tensor([[0.0, 0.5, 0.0, 0.5]], device="cuda")
    assert bool(((grad - want).abs() < 1e-6).all())


def test_distillation_without_entries(gemm_lib):
    logits = torch.randn(3, 50, device="cuda").half()
    out = torch.full((3, 50), 5.0, dtype=torch.float16, device="cuda")
    loss, lse = torch.ones(3, device="cuda"), torch.ones(3, device="cuda")
    none = torch.empty(3, 0, dtype=torch.int64, device="cuda"), torch.empty(3, 0, device="cuda")
    with gemm_lib.DistillPlan(3, 50, 4, "f16") as plan:
        plan.forward_backward(logits, *none, loss, lse, out)
        assert not bool(out.any()) and not bool(loss.any()) and bool((lse == -math.inf).all())
        plan.forward(logits[:0], none[0][:0], none[1][:0], loss[:0], lse[:0])


def test_distillation_ids_too_large(gemm_lib):
    logits, values = torch.randn(2, 50, device="cuda"), torch.randn(2, 3, device="cuda")
    ids = torch.tensor([[1, 50, 2], [4, 5, (1 << 32) + 4]], device="cuda")
    with gemm_lib.DistillPlan(2, 50, 3, "f32") as plan:
        res = []
        for i in (ids, torch.where(ids < 50, ids, -1)):
            loss, lse, grad = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, 50, device="cuda")
            plan.forward_backward(logits, i, values, loss, lse, grad)
            res.append((loss, lse, grad))
            if not res[1:]:
                with pytest.raises(gemm_lib.GemmError) as e:
                    plan.check()
                assert e.value.status == 12
        plan.check()
        assert all(torch.equal(a, b) for a, b in zip(*res))


def test_distillation_gradient_against_differences(gemm_lib):
    """The kernel's fp32 loss, moved along random directions, against its gradient: a difference over 2h is off
    by the loss' bound over h and by the curve's bend (h^2)."""
    rng = np.random.default_rng(8)
    rows, vocab, tau, h = 4, 30, 2.0, 2.0 ** -6
    c = _distill_case(rows, vocab, 5, "f32", "f32", "i64", 0, 0, True, tau)
    base = _f64(c["logits"])
    with gemm_lib.DistillPlan(rows, vocab, 5, "f32") as plan:
        def f(s):
            t = torch.as_tensor(s, dtype=torch.float32).cuda()
            plan.forward(t, c["ids"], c["values"], c["loss"], c["lse"], temperature=tau, teacher_lse=c["given"])
            return (_f64(c["loss"]) * _f64(c["dloss"])).sum()
        f(base)
        plan.backward(c["logits"], c["ids"], c["values"], c["lse"], c["dlogits"], dloss=c["dloss"], temperature=tau,
                      teacher_lse=c["given"])
        noise = (to.distill_bounds(base, c["ids"].cpu().numpy(), _f64(c["values"]), tau, "f32",
                                   _f64(c["given"]))[0] * _f64(c["dloss"])).sum() / h
        grad = _f64(c["dlogits"])
        for _ in range(4):
            u = rng.choice([-1.0, 1.0], size=base.shape)
            diff = (f(base + h * u) - f(base - h * u)) / (2 * h)
            # third derivative of a log-sum-exp along u: at most 2 (per temperature); tau^2 / tau^3 of it, a sixth, over rows
            assert abs(diff - (grad * u).sum()) <= 2 * noise + _f64(c["dloss"]).sum() * h * h + np.abs(grad).sum() * 2.0 ** -20 / h


# ---------------------------------------------------------------- all of them

def test_offsets_beyond_32_bits(gemm_lib):
    """Matrices of more than 2^32 elements: rows at both ends."""
    rng = torch.Generator(device="cuda").manual_seed(3)
    rows, cols = 262150, 16400                                  # 4.3e9 elements
    big = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 131000, rows - 2, rows - 1]
    big.zero_()
    big[at] = torch.randn(len(at), cols, generator=rng, device="cuda").bfloat16()
    few, want = big[at].contiguous(), torch.empty(len(at), cols, dtype=torch.bfloat16, device="cuda")
    with gemm_lib.NormPlan(rows, cols, "bf16", weight="f32") as plan:
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        plan.forward(big, None, None, out, mean, rstd)
        m, r = torch.empty(len(at), device="cuda"), torch.empty(len(at), device="cuda")
        plan.forward(few, None, None, want, m, r)
        assert torch.equal(out[at], want) and torch.equal(mean[at], m)
        plan.backward(big, None, mean, rstd, big, out)
        plan.backward(few, None, m, r, few, want)
        assert torch.equal(out[at], want)
    ids = torch.tensor([rows - 1, 0, 131000, rows - 1], device="cuda")
    with gemm_lib.EmbedPlan(rows, cols, 4, "bf16") as plan:
        got = torch.empty(4, cols, dtype=torch.bfloat16, device="cuda")
        plan.forward(ids, big, got)
        assert torch.equal(got, big[ids])
        plan.backward(ids, got, out)
        assert torch.equal(out[rows - 1], (2 * got[0].float()).bfloat16()) and torch.equal(out[131000], got[2])
        assert not bool(out[rows - 2].any())
    with gemm_lib.DistillPlan(rows, cols, 2, "bf16") as plan:
        entry = torch.full((rows, 2), -1, device="cuda")
        entry[at, 0], entry[at, 1] = 3, cols - 1
        values = torch.ones(rows, 2, device="cuda")
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        plan.forward_backward(big, entry, values, loss, lse, out)
        l2, e2 = torch.empty(len(at), device="cuda"), torch.empty(len(at), device="cuda")
        plan.forward_backward(few, entry[at].contiguous(), values[at].contiguous(), l2, e2, want)
        tol = 1e-5                                              # the rows may be split otherwise when there are few
        assert bool(((loss[at] - l2).abs() < tol).all()) and bool(((lse[at] - e2).abs() < tol).all())
        assert bool(((out[at].float() - want.float()).abs() <= 2.0 ** -8 * want.float().abs() + 1e-9).all())
        assert not bool(out[2].any())


def test_other_streams_and_graphs(gemm_lib):
    """Each call on a stream of its own, and captured into a graph that runs on new inputs."""
    c = _norm_case(64, 1024, "bf16", "f32", 0, 0)
    e = _embed_case(500, 900, 256, "bf16", "f32", "i64", 0, 0)
    d = _distill_case(12, 3000, 10, "bf16", "f32", "i64", 0, 0, False, 1.0)
    norm, embed = gemm_lib.NormPlan(64, 1024, "bf16", weight="f32"), gemm_lib.EmbedPlan(900, 256, 500, "bf16", grad="f32")
    kd = gemm_lib.DistillPlan(12, 3000, 10, "bf16")

    def calls(stream):
        norm.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"], stream=stream)
        norm.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"], c["dbeta"], stream=stream)
        embed.forward(e["ids"], e["table"], e["out"], stream=stream)
        embed.backward(e["ids"], e["dout"], e["dtable"], stream=stream)
        kd.forward(d["logits"], d["ids"], d["values"], d["loss"], d["lse"], stream=stream)
        kd.backward(d["logits"], d["ids"], d["values"], d["lse"], d["dlogits"], dloss=d["dloss"], stream=stream)
        kd.forward_backward(d["logits"], d["ids"], d["values"], d["loss"], d["lse"], d["dlogits"], dloss=d["dloss"],
                            stream=stream)

    def check():
        torch.cuda.synchronize()
        _check_norm(c, "bf16", "f32")
        ids = e["ids"].cpu().numpy()
        want = to.embed_forward(ids, -1, _f64(e["table"]), 1.0)
        _within(e["out"], want, to.rounded(want, "bf16"), "out")
        want, bound = to.embed_backward(ids, -1, _f64(e["dout"]), 1.0, 900)
        _within(e["dtable"], want, bound + to.rounded(want, "f32"), "dtable")
        _check_distill(d, "bf16", 1.0)

    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    calls(stream)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls(stream)
    c["x"].mul_(0.5)
    e["ids"].copy_(torch.flip(e["ids"], [0]))
    d["logits"].mul_(0.25)
    d["logits"][5] = 1.0
    for t in (c["y"], c["dx"], e["dtable"], d["dlogits"]):
        t.fill_(3.0)
    graph.replay()
    check()
    for p in (norm, embed, kd):
        p.close()
        p.close()


def test_refusals(gemm_lib):
    """Arguments that do not fit are refused before anything is queued."""
    g = gemm_lib
    x = torch.zeros(4, 64, device="cuda")
    v, w = torch.zeros(64, device="cuda"), torch.zeros(4, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    norm, embed, kd = g.NormPlan(4, 64, "f32"), g.EmbedPlan(4, 64, 4, "f32"), g.DistillPlan(4, 64, 3, "f32")
    ent, val = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.zeros(4, 3, device="cuda")
    wide = torch.zeros(5, 64, device="cuda")
    bad = [
        (1, lambda: norm.forward(wide, v, v, wide)),                               # more rows than the plan's
        (1, lambda: norm.forward(x[:, :32], v, v, x[:, :32])),                     # other columns
        (1, lambda: norm.forward(x.t().contiguous().t(), v, v, x)),                # columns contiguous
        (1, lambda: norm.forward(x[:1].expand(4, 64), v, v, x)),                   # overlapping rows
        (2, lambda: norm.forward(x.half(), v, v, x)),                              # another type
        (1, lambda: norm.forward(x, v, v, x, eps=-1.0)),
        (1, lambda: norm.forward(x, v, v, x, eps=math.nan)),
        (1, lambda: norm.forward(x.cpu(), v, v, x)),                               # host memory
        (1, lambda: norm.forward(x, v[:32], v, x)),
        (1, lambda: norm.backward(x, v, w, w[:3], x, x)),
        (1, lambda: norm.backward(x, v, None, w, x, x)),
        (2, lambda: norm.backward(x, v, w.double(), w, x, x)),
        (1, lambda: embed.forward(ids, x, x[:3])),
        (2, lambda: embed.forward(ids.to(torch.int16), x, x)),
        (1, lambda: embed.forward(torch.zeros(5, dtype=torch.int64, device="cuda"), x, wide)),
        (1, lambda: embed.backward(ids, x, x[:3])),
        (2, lambda: embed.backward(ids, x, x.half())),
        (1, lambda: kd.forward(x, ent, val, w, w, temperature=0.0)),
        (1, lambda: kd.forward(x, ent, val, w, w, temperature=math.nan)),
        (1, lambda: kd.forward(x, torch.zeros(4, 4, dtype=torch.int64, device="cuda"), torch.zeros(4, 4, device="cuda"), w, w)),
        (1, lambda: kd.forward(x, ent, val[:3], w, w)),
        (2, lambda: kd.forward(x, ent, val.double(), w, w)),
        (2, lambda: kd.forward(x, ent.short(), val, w, w)),
        (1, lambda: kd.forward(x[:, :60], ent, val, w, w)),
        (1, lambda: kd.backward(x, ent, val, w, x[:3])),
        (2, lambda: kd.backward(x, ent, val, w, x.half())),
        (1, lambda: kd.forward_backward(x, ent, val, w, w, x, dloss=w[:3])),
        (1, lambda: kd.forward_backward(x, ent, val, w, w, x, teacher_lse=w[:3])),
    ]
    for k, (status, call) in enumerate(bad):
        with pytest.raises(g.GemmError) as e:
            call()
        assert e.value.status == status, (k, e.value)
    torch.cuda.synchronize()
    assert not bool(x.any()) and not bool(w.any())
    for args in ((g.NormPlan, 4, 8, "f16", "bf16"), (g.EmbedPlan, 4, 8, 4, "bf16", "f16")):
        with pytest.raises(g.GemmError) as e:
            args[0](*args[1:])
        assert e.value.status == 2
    norm.close()
    with pytest.raises(g.GemmError) as e:                     # a closed plan
        norm.forward(x, v, v, x)
    assert e.value.status == 1
