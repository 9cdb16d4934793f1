"""The operators where their kernels change paths: limits of the sort, plans with many teacher
entries, matrices beyond 2^32 elements at usual widths, streams of their own, first calls in a graph."""
import os
import subprocess
import sys

import pytest
import torch

import test_train_ops_gpu as ops
import train_oracle as to

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8192, 16384, 16385, 20000])
@pytest.mark.parametrize("vocab", [511, 512, 2 ** 18 - 1, 2 ** 18])
def test_embedding_sort_at_its_limits(gemm_lib, n, vocab):
    """Pairs that fit the cluster's shared memory, one more; ids whose largest key takes one more bit or pass."""
    gen = torch.Generator(device="cuda").manual_seed(n + vocab)
    ids = torch.randint(vocab, (n,), generator=gen, device="cuda")
    ids[0], ids[1], ids[2] = vocab - 1, 0, vocab - 1
    dout = torch.randint(-2, 3, (n, 8), generator=gen, device="cuda").float()
    dtable = torch.full((vocab, 8), 7.0, device="cuda")
    with gemm_lib.EmbedPlan(vocab, 8, n, "f32") as plan:
        plan.backward(ids, dout, dtable)
        plan.check()
    assert torch.equal(dtable, torch.zeros_like(dtable).index_add_(0, ids, dout))


@pytest.mark.parametrize("rows,vocab,top,elem", [(500, 9001, 137, "bf16"), (500, 9001, 1024, "f16"), (400, 20011, 300, "f32"),
                                                 (200, 66000, 1000, "bf16")])
@pytest.mark.parametrize("given", [False, True])
def test_distillation_of_many_rows_and_entries(gemm_lib, rows, vocab, top, elem, given):
    """Plans for more entries than six of a block's slots hold."""
    c = ops._distill_case(rows, vocab, top, elem, "f32", "i32", 0, 0, given, 1.0)
    c["ids"][5, top - 1] = c["ids"][5, 0]            # equal ids, far apart
    c["ids"][6, ::2] = -1
    more = {"teacher_lse": c["given"]}
    with gemm_lib.DistillPlan(rows, vocab, top, elem) as plan:
        plan.forward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], **more)
        plan.backward(c["logits"], c["ids"], c["values"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
        ops._check_distill(c, elem, 1.0)
        for k in ("loss", "lse", "dlogits"):
            c[k].fill_(5.0)
        plan.forward_backward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
        ops._check_distill(c, elem, 1.0, what="both: ")
        plan.check()


@pytest.mark.parametrize("cols", [4096, 4099, 12000, 16376])
def test_norm_rows_beyond_32_bits(gemm_lib, cols):
    """More than 2^32 elements in rows that go through rings: rows at both ends and in the middle, by the formula."""
    rows = 2 ** 32 // cols + 1000
    gen = torch.Generator(device="cuda").manual_seed(cols)
    at = [0, 1, 2 ** 31 // cols, 2 ** 31 // cols + 1, rows - 200, rows - 2, rows - 1]
    x, out = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[at] = torch.randn(len(at), cols, generator=gen, device="cuda").bfloat16()
    gamma = torch.randn(cols, generator=gen, device="cuda") + 1
    beta = torch.randn(cols, generator=gen, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    few = ops._f64(x[at])
    with gemm_lib.NormPlan(rows, cols, "bf16", weight="f32") as plan:
        plan.forward(x, gamma, beta, out, mean, rstd)
        args = (few, ops._f64(gamma), ops._f64(beta), 1e-5)
        want, bound = to.norm_forward(*args), to.norm_forward_bounds(*args, "bf16")
        for got, w, b, name in zip((out[at], mean[at], rstd[at]), want, bound, ("y", "mean", "rstd")):
            ops._within(got, w, b, name)
        dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        plan.backward(x, gamma, mean, rstd, x, out, dgamma, dbeta)         # (dy is x: zero but at those rows)
        args = (few, ops._f64(gamma), ops._f64(mean[at]), ops._f64(rstd[at]), few)
        want, bound = to.norm_backward(*args), to.norm_backward_bounds(*args, "bf16", "f32")
        ops._within(out[at], want[0], bound[0], "dx")
        ops._within(dgamma, want[1], bound[1], "dgamma")
        ops._within(dbeta, want[2], bound[2], "dbeta")
        plan.check()


def test_operators_on_streams_of_their_own(gemm_lib):
    """Each operator on a stream that is not the tensors', with events between what depends on one another."""
    rows, dim, vocab = 600, 1024, 5000
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(vocab, dim, generator=gen, device="cuda").bfloat16()
    ids = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    x, y, dx = (torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    mean, rstd, loss, lse = (torch.zeros(rows, device="cuda") for _ in range(4))
    entries = torch.randint(dim, (rows, 4), generator=gen, device="cuda")
    values, dlogits = torch.randn(rows, 4, generator=gen, device="cuda"), torch.zeros_like(y)
    dtable = torch.zeros(vocab, dim, device="cuda")
    with gemm_lib.EmbedPlan(vocab, dim, rows, "bf16", grad="f32") as embed, \
            gemm_lib.NormPlan(rows, dim, "bf16", weight="f32") as norm, gemm_lib.DistillPlan(rows, dim, 4, "bf16") as kd:
        def step(s):
            def after(this, before):
                if this is not None:
                    this.wait_stream(before)
            embed.forward(ids, table, x, stream=s[0])
            after(s[1], s[0])
            norm.forward(x, None, None, y, mean, rstd, stream=s[1])
            after(s[2], s[1])
            kd.forward_backward(y, entries, values, loss, lse, dlogits, stream=s[2])
            after(s[1], s[2])
            norm.backward(x, None, mean, rstd, dlogits, dx, stream=s[1])
            after(s[0], s[1])
            embed.backward(ids, dx, dtable, stream=s[0])
            torch.cuda.synchronize()
            return [t.clone() for t in (x, y, mean, rstd, loss, lse, dlogits, dx, dtable)]

        torch.cuda.synchronize()
        want = step([None, None, None])
        for t in (x, y, mean, rstd, loss, lse, dlogits, dx, dtable):
            t.fill_(3.0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, step([torch.cuda.Stream() for _ in range(3)])))
        for plan in (embed, norm, kd):
            plan.check()


COLD = """
import torch
import dense_gemm_hgemm_gb300 as g
x = torch.randn(2000, 4096, device="cuda").bfloat16()
y, dx = torch.zeros_like(x), torch.zeros_like(x)
w, dw, db = torch.ones(4096, device="cuda"), torch.empty(4096, device="cuda"), torch.empty(4096, device="cuda")
m, r, loss, lse = (torch.empty(2000, device="cuda") for _ in range(4))
ids = torch.randint(0, 500, (300,), device="cuda")
table, out = torch.randn(500, 256, device="cuda").bfloat16(), torch.empty(300, 256, device="cuda").bfloat16()
grad, e, v = torch.empty(500, 256, device="cuda"), torch.randint(0, 4096, (2000, 8), device="cuda"), torch.randn(2000, 8, device="cuda")
n, em, kd = g.NormPlan(2000, 4096, "bf16", weight="f32"), g.EmbedPlan(500, 256, 300, "bf16", grad="f32"), g.DistillPlan(2000, 4096, 8, "bf16")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    n.forward(x, w, w, y, m, r)
    n.backward(x, w, m, r, y, dx, dw, db)
    em.forward(ids, table, out)
    em.backward(ids, out, grad)
    kd.forward(x, e, v, loss, lse)
    kd.backward(x, e, v, lse, dx)
    kd.forward_backward(x, e, v, loss, lse, dx)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, out, grad, loss, lse, dx)]
n.forward(x, w, w, y, m, r)
em.forward(ids, table, out)
em.backward(ids, out, grad)
kd.forward_backward(x, e, v, loss, lse, dx)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (y, out, grad, loss, lse, dx)))
for p in (n, em, kd):
    p.check()
print("captured cold")
"""


def test_first_calls_of_fresh_plans_can_be_captured(gemm_lib):
    """In a process that has launched none of the kernels."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(ops.__file__)))
    done = subprocess.run([sys.executable, "-c", COLD], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured cold" in done.stdout, done.stderr[-2000:]
