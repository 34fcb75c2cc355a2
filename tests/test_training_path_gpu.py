"""The operators of a training step run together: tokens sorted by expert,
through the experts' two products with their gradients, a norm, and the loss
over the vocabulary with its gradient, from labels or from a teacher.

Each step is held to its own formula in 64 bits on the values the step before
left on the device, with the bounds of that operator's own tests.
"""
import pytest
import torch

import dense_gemm_05_amd as g5
import test_grouped_gpu as grouped
import test_linear_loss_gpu as loss
import test_norm_gpu as norm

pytestmark = pytest.mark.gpu

EPS = 1e-5


class _Step:
    """T tokens of width H, E experts of inner width I with k each, V words; topk 0: labels."""

    def __init__(self, T, H, E, I, k, V, topk):
        self.g = norm._gen(21, T, H, E, I, k, V, topk)
        self.k, self.E = k, E
        self.c = loss.Case(T, V, H, topk, seed=3)
        self.x, self.w = self._bf(T, H), self._bf(H)
        self.router = self._bf(E, H, scale=H ** -0.5)
        self.up, self.down = self._bf(E, 2 * I, H, scale=H ** -0.5), self._bf(E, H, I, scale=I ** -0.5)
        self.head, self.ids, self.dloss = self.c.w.cuda(), self.c.ids.cuda(), self.c.dloss.cuda()
        self.t = self.c.t.cuda() if topk else None

    def _bf(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g) * scale).bfloat16().cuda()

    def run(self, ws):
        r, I = {}, self.down.shape[2]
        logits = g5.gemm_bf16_nt(self.x, self.router, out_dtype=torch.float32, workspace=ws)
        gates, experts = logits.softmax(1).topk(self.k, dim=1)
        flat = experts.reshape(-1)
        order = flat.argsort(stable=True)
        # where each expert's rows start among the sorted ones
        starts = torch.searchsorted(flat[order], torch.arange(self.E + 1, device="cuda"))
        r["offsets"], token = starts.to(torch.int32), order // self.k
        gate = gates.reshape(-1)[order, None]
        r["rows"] = self.x[token]
        r["gu"] = g5.gemm_bf16_grouped_nt(r["rows"], self.up, r["offsets"], workspace=ws)
        r["z"] = g5.act_swiglu(r["gu"][:, :I].contiguous(), r["gu"][:, I:].contiguous())
        r["y"] = g5.gemm_bf16_grouped_nt(r["z"], self.down, r["offsets"], workspace=ws)
        back = torch.empty_like(order)
        back[order] = torch.arange(order.numel(), device="cuda")
        m = ((r["y"].float() * gate)[back].reshape(-1, self.k, self.x.shape[1]).sum(1)).bfloat16()
        r["rstd"] = torch.empty((self.x.shape[0],), device="cuda")
        r["n"], r["h"] = g5.rms_norm(m, self.w, residual=self.x, eps=EPS, rstd=r["rstd"])
        if self.t is None:
            r["loss"], r["lse"] = g5.linear_cross_entropy(r["n"], self.head, self.ids, workspace=ws)
            r["dn"], r["dhead"] = g5.linear_cross_entropy_backward(self.dloss, r["n"], self.head, self.ids, r["lse"], workspace=ws)
        else:
            r["loss"], r["lse"] = g5.linear_distill(r["n"], self.head, self.ids, self.t, workspace=ws)
            r["dn"], r["dhead"] = g5.linear_distill_backward(self.dloss, r["n"], self.head, self.ids, self.t, r["lse"], workspace=ws)
        r["dh"], r["dw"] = g5.rms_norm_backward(r["dn"], r["h"], self.w, r["rstd"], workspace=ws)
        r["dy"] = (r["dh"].float()[token] * gate).bfloat16()
        r["dz"] = g5.gemm_bf16_grouped(r["dy"], self.down, r["offsets"], workspace=ws)
        r["ddown"] = g5.gemm_bf16_grouped_tn(r["dy"], r["z"], r["offsets"], workspace=ws)
        return r

    def check(self, r):
        v = {k: t.cpu() for k, t in r.items()}
        o = v["offsets"].tolist()
        assert o[0] == 0 and o[-1] == v["rows"].shape[0]
        up, down = self.up.cpu(), self.down.cpu()
        grouped._check(v["gu"], *grouped._formula("nt", v["rows"], up, o), "gate and up")
        grouped._check(v["y"], *grouped._formula("nt", v["z"], down, o), "down")
        grouped._check(v["dz"], *grouped._formula("nn", v["dy"], down, o), "dz")
        grouped._check(v["ddown"], *grouped._formula("tn", v["dy"], v["z"], o), "ddown")
        c = self.c
        c.x = v["n"]
        c.check_forward(v["loss"], v["lse"])
        c.check_backward(v["lse"], v["dn"], v["dhead"])
        ref, tol, _, _ = norm._grad_ref(v["dn"], v["h"], self.w.cpu(), v["rstd"], torch.zeros(()))
        norm._check(v["dh"].double(), ref, tol, "dh")


SIZES = [(3, 64, 4, 24, 2, 50, 0), (40, 136, 8, 72, 2, 300, 5), (300, 256, 6, 128, 2, 515, 0), (700, 264, 3, 40, 1, 130, 9)]


@pytest.mark.parametrize("size", SIZES)
def test_training_step(size):
    print(f"[training] {size}", flush=True)
    step = _Step(*size)
    step.check(step.run(g5.Workspace()))


@pytest.mark.parametrize("size", SIZES[1:3])
def test_training_step_captured(size):
    """Captured with a workspace of its own, replayed on new tokens between
    eager steps."""
    step = _Step(*size)
    ws, held = g5.Workspace(), g5.Workspace()
    step.run(ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step.run(held)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run(held)
    for n in range(3):
        step.x.copy_(step._bf(*step.x.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        want = step.run(ws)
        for k in want:
            assert torch.equal(got[k], want[k]), f"replay {n}: {k}"
    step.check(got)


def test_two_graphs_on_one_workspace():
    """A loss with its gradient and a weight gradient, both through copies and
    sums in the workspace, captured apart and replayed in turn, with eager
    calls on it between."""
    c = loss.Case(150, 300, 65, 4)
    x, w, ids, t, dl = c.x.cuda(), c.w.cuda(), c.ids.cuda(), c.t.cuda(), c.dloss.cuda()
    a, b, o = grouped._case("tn", [70, 0, 230], 65, 99, 3)
    a, b, o = a.cuda(), b.cuda(), torch.tensor(o, dtype=torch.int32).cuda()
    ws = g5.Workspace(nbytes=64 << 20)

    def one():
        value, lse = g5.linear_distill(x, w, ids, t, workspace=ws)
        return value, *g5.linear_distill_backward(dl, x, w, ids, t, lse, workspace=ws)

    def two():
        return (g5.gemm_bf16_grouped_tn(a, b, o, workspace=ws),)

    one(), two()
    held, graphs, outs = ws.buf.data_ptr(), [], []
    for call in (one, two):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call())
    g = torch.Generator().manual_seed(4)
    for turn in range(4):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        a.copy_(torch.randn(a.shape, generator=g).bfloat16())
        for graph in graphs[::1 if turn % 2 else -1]:
            graph.replay()
        got = [[v.clone() for v in out] for out in outs]
        for n, call in enumerate((one, two)):
            assert all(torch.equal(p, q) for p, q in zip(got[n], call())), f"turn {turn}, graph {n}"
    assert ws.buf.data_ptr() == held and not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()


def _rows(n, k, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, k), generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)


def test_grouped_rows_past_32_bits():
    """Rows whose elements lie past 2^31, and a weight past 2^32 bytes: the
    last groups' outputs against the formula."""
    rows, k, n, E = 560000, 4096, 64, 4
    a, b = _rows(rows, k, 1), _rows(E * n, k, 2, k ** -0.5).reshape(E, n, k)
    o = [0, 100, 300000, rows - 300, rows]
    off = torch.tensor(o, dtype=torch.int32).cuda()
    c = g5.gemm_bf16_grouped_nt(a, b, off)
    pick = torch.cat([torch.arange(rows - 310, rows), torch.arange(299990, 300010)])
    which = torch.bucketize(pick, torch.tensor(o[1:-1]), right=True)
    x, w = a[pick.cuda()].cpu().double(), b.cpu().double()
    ref = torch.stack([w[e] @ row for e, row in zip(which.tolist(), x)])
    tol = 1.01 * k * 2.0 ** -23 * torch.stack([w[e].abs() @ row.abs() for e, row in zip(which.tolist(), x)])
    grouped._check(c[pick.cuda()], ref, tol, "rows")
    # the sum over the last group alone, and over one of 300000 rows in parts
    d = _rows(rows, 8, 3)
    got = g5.gemm_bf16_grouped_tn(d, a, off)
    for e in (2, 3):
        x, y = d[o[e]:o[e + 1]].double(), a[o[e]:o[e + 1]].double()
        # (the sums' bound: their order is free, a step of the terms' sizes per addition)
        tol = 1.01 * x.shape[0] * 2.0 ** -23 * (x.abs().t() @ y.abs())
        grouped._check(got[e], (x.t() @ y).cpu(), tol.cpu(), f"group {e}")


def test_vocabulary_past_32_bits():
    """A weight of more than 2^31 elements: targets in its last rows."""
    V, K, M = 600000, 4096, 40
    w, x = _rows(V, K, 4, 2 * K ** -0.5), _rows(M, K, 5)
    ids = torch.cat([torch.arange(V - M + 4, V), torch.tensor([-1, V, 0, 5])]).cuda()
    dl = torch.rand((M,), device="cuda") + 0.5
    loss_, lse = g5.linear_cross_entropy(x, w, ids)
    l = x.double() @ w.double().t()
    ref = torch.logsumexp(l, 1)
    some = (ids >= 0) & (ids < V)
    want = torch.where(some, ref - l[torch.arange(M), ids.clamp(0, V - 1)], 0.0)
    # FP32 sums of 4096 products (a step of the terms' sizes for each), 2^-16 for the exponentials' sum
    bound = 1.01 * K * 2.0 ** -23 * float((x.abs().double() @ w.abs().double().t()).max()) + 2.0 ** -16
    assert float((lse - ref).abs().max()) <= bound and float((loss_ - want).abs().max()) <= 2 * bound
    dx, dw = g5.linear_cross_entropy_backward(dl, x, w, ids, lse)
    p = torch.exp(l - lse.double()[:, None]) * some[:, None]
    p[torch.arange(M)[some.cpu()], ids[some]] -= 1.0
    p *= dl.double()[:, None]
    del l
    slack = bound + 2.0 ** -15
    rows = torch.arange(V - 64, V).cuda()
    for got, ref, size in ((dw[rows], p[:, rows].t() @ x.double(), p[:, rows].abs().t() @ x.double().abs()),
                           (dx, p @ w.double(), p.abs() @ w.double().abs())):
        assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * slack * size + 2.0 ** -126).all())
    assert bool((dx[~some] == 0).all())


def test_many_groups():
    """As many groups as there may be, most of them empty."""
    E, n, k = 4096, 8, 16
    g = torch.Generator().manual_seed(6)
    sizes = (torch.rand((E,), generator=g) < 0.1).int() * torch.randint(1, 4, (E,), generator=g)
    o = [0] + sizes.cumsum(0).tolist()
    for kind in ("nt", "nn", "tn"):
        rows = o[-1]
        a = torch.randn((rows, n if kind == "tn" else k), generator=g).bfloat16()
        b = torch.randn((rows, k) if kind == "tn" else (E, n, k) if kind == "nt" else (E, k, n), generator=g).bfloat16()
        grouped._check(grouped._run(kind, a, b, o), *grouped._formula(kind, a, b, o), kind)
