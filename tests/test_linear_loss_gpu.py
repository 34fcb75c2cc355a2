"""The loss over a vocabulary behind the last projection, from labels and from
a teacher's best logits, and its gradients, against the formulas in 64 bits:
odd sizes and strides, rows left out, values in them that must not matter,
pieces of the vocabulary, graphs and streams."""
import math

import pytest
import torch

import dense_gemm_05_amd as g5
from _gpu_helpers import ws

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _say(msg):
    print(f"[loss] {msg}", flush=True)


class Case:
    """Inputs on the CPU.  topk 0: labels."""

    def __init__(self, M, V, K, topk=0, seed=0, scale=1.0, std=3.0, out=0.2):
        g = torch.Generator().manual_seed(seed + M + V + K + topk)
        self.M, self.V, self.K, self.topk, self.scale = M, V, K, topk, scale
        self.x = torch.randn((M, K), generator=g).bfloat16()
        self.w = (torch.randn((V, K), generator=g) * std * K ** -0.5).bfloat16()
        if topk:
            self.ids = torch.stack([torch.randperm(max(V, topk), generator=g)[:topk] for _ in range(M)])   # some past V where V < topk
            self.ids[torch.rand((M, topk), generator=g) < out] = -1
            self.t = 4 * torch.randn((M, topk), generator=g)
        else:
            self.ids = torch.randint(0, V, (M,), generator=g)
            self.ids[torch.rand((M,), generator=g) < out] = -100
            self.t = None
        self.dloss = torch.rand((M,), generator=g) + 0.25

    def targets(self):
        """(q [M, V], per row: any target, constant of the loss) in 64 bits."""
        q, const = torch.zeros((self.M, self.V)).double(), torch.zeros(self.M).double()
        some = torch.zeros(self.M, dtype=torch.bool)
        ids = self.ids if self.topk else self.ids[:, None]
        for m in range(self.M):
            has = [j for j in range(ids.shape[1]) if 0 <= ids[m, j] < self.V and not (self.topk and self.t[m, j] == -INF)]
            if not has:
                continue
            some[m] = True
            p = torch.softmax(self.t[m, has].double() * self.scale, 0) if self.topk else torch.ones(1).double()
            q[m].index_put_((ids[m, has].long(),), p, accumulate=True)
            const[m] = torch.special.xlogy(p, p).sum()
        return q, some, const

    def logits(self):
        """l and the bound of its FP32 sums (K additions in any order, a step
        of 2^-23 of the terms' sizes each) and of the factor."""
        s = float(torch.tensor(self.scale, dtype=torch.float32))
        x, w = self.x.double(), self.w.double()
        l = s * (x @ w.t())
        return l, 1.01 * (self.K + 2) * 2.0 ** -23 * s * (x.abs() @ w.abs().t())

    def forward(self, **kw):
        x, w, ids = kw.pop("x", self.x.cuda()), kw.pop("w", self.w.cuda()), kw.pop("ids", self.ids.cuda())
        kw.setdefault("workspace", ws())
        if self.topk:
            return g5.linear_distill(x, w, ids, self.t.cuda(), scale=self.scale, **kw)
        return g5.linear_cross_entropy(x, w, ids, scale=self.scale, **kw)

    def backward(self, lse, **kw):
        x, w, ids = kw.pop("x", self.x.cuda()), kw.pop("w", self.w.cuda()), kw.pop("ids", self.ids.cuda())
        kw.setdefault("workspace", ws())
        if self.topk:
            return g5.linear_distill_backward(self.dloss.cuda(), x, w, ids, self.t.cuda(), lse, scale=self.scale, **kw)
        return g5.linear_cross_entropy_backward(self.dloss.cuda(), x, w, ids, lse, scale=self.scale, **kw)

    def check_forward(self, loss, lse, what=""):
        """The sum of exponentials: every term within 2^-20 of itself (its
        argument's and the function's rounding; a term of argument -a weighs
        e^-a, and a e^-a < 1), at most 2^7 roundings of 2^-24 on the way to the
        whole.  Then the logarithm, the factor and the sums, 2^-22 of their
        values' sizes."""
        l, el = self.logits()
        q, some, const = self.targets()
        ref = torch.logsumexp(l, 1)
        tol = el.max(1).values + 2.0 ** -16 + 2.0 ** -21 * (l.abs().max(1).values + ref.abs())
        _close(lse, ref, tol, what + " lse")
        want = torch.where(some, const + (q * (ref[:, None] - l)).sum(1), 0.0)
        tol = torch.where(some, tol + (q * el).sum(1) + 2.0 ** -20 * (1 + const.abs() + (q * l.abs()).sum(1)), 0.0)
        if self.topk:      # q's own rounding (2^-19: argument, exponential, sum, quotient) meets these differences
            tol = torch.where(some, tol + 2.0 ** -19 * (q * ((ref[:, None] - l).abs() + math.log(self.topk) + 20)).sum(1), 0.0)
        _close(loss, want, tol, what + " loss")

    def gradients(self, lse):
        """((dX, bound), (dW, bound)) for the lse that was handed in."""
        s = float(torch.tensor(self.scale, dtype=torch.float32))
        l, el = self.logits()
        q, some, _ = self.targets()
        lse, g = lse.cpu().double()[:, None], torch.where(some, self.dloss.double(), 0.0)[:, None]
        p = torch.exp(l - lse) * some[:, None]
        d = g * (p - q)
        # exp's argument: the logit's sums, and roundings of its parts; the
        # exponential itself; q's rounding; D's one rounding to bf16 (half a
        # step), or up to 64 rows a second one of the first one's rest
        ed = g * (p * torch.expm1(el + 2.0 ** -21 * (l.abs() + lse.abs()) + 2.0 ** -20) + 2.0 ** -19 * q)
        ed = ed + ((2.0 ** -8 if self.M > 64 else 2.0 ** -16) + 2.0 ** -20) * (d.abs() + ed)
        # Below the normal numbers of FP32 and bf16, 2^-126, an exponential, a
        # D, a product or a sum may be a zero: each is formed relative to the
        # largest weight, so that many times it per D and per addition.
        least = float(g.max()) * 2.0 ** -126
        ed = ed + least
        x, w = torch.where(some[:, None], self.x.double(), 0.0), self.w.double()
        out = []
        for a, e, b, n in ((d, ed, w, 2 * self.V), (d.t(), ed.t(), x, 2 * self.M)):
            size = a.abs() @ b.abs()
            sums = 1.01 * (n + 8) * 2.0 ** -23 * size + 2 * (n + 8) * least
            out.append((s * (a @ b), s * (e @ b.abs() * (1 + 2.0 ** -10) + sums) + 2.0 ** -126))
        return out

    def check_backward(self, lse, dx, dw, what=""):
        for got, (ref, tol), name in zip((dx, dw), self.gradients(lse), ("dX", "dW")):
            if got is not None:
                half = torch.finfo(got.dtype).eps / 2
                _close(got, ref, half * ref.abs() + (1 + half) * tol, f"{what} {name}")


def _close(got, ref, tol, what):
    got = got.cpu().double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(got[bad][0])} for {float(ref[bad][0])} within {float(tol[bad][0])}")


SIZES = [(1, 1, 1), (1, 5, 8), (2, 17, 3), (3, 40, 64), (5, 2000, 520), (16, 1000, 100), (17, 33, 65), (32, 300, 72),
         (33, 300, 72), (64, 128, 32), (130, 515, 136), (257, 257, 31), (1000, 130, 33), (2000, 200, 40),
         (300, 33000, 264)]


@pytest.mark.parametrize("topk", [0, 1, 5, 70])
@pytest.mark.parametrize("M,V,K", SIZES)
def test_loss_and_gradients(M, V, K, topk):
    _say(f"{M} {V} {K} {topk}")
    c = Case(M, V, K, topk, scale=0.5 if topk == 5 else 1.0)
    loss, lse = c.forward()
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse)
    c.check_backward(lse, dx, dw)


@pytest.mark.parametrize("topk", [0, 7, 256])
@pytest.mark.parametrize("config", ["bf16_256x256", "bf16_128x128", "decode_nt"])
@pytest.mark.parametrize("M,V,K", [(1, 40, 8), (20, 300, 65), (32, 513, 256), (70, 260, 129), (600, 1000, 200)])
def test_every_tile_takes_every_size(monkeypatch, M, V, K, topk, config):
    if config == "decode_nt" and M > 32:
        pytest.skip("the stream is for up to 32 rows")
    monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{config} {M} {V} {K} {topk}")
    c = Case(M, V, K, topk, seed=5)
    loss, lse = c.forward(workspace=None)
    c.check_forward(loss, lse, config)
    c.check_backward(lse, *c.backward(lse, workspace=None), config)


@pytest.mark.parametrize("topk", [0, 7])
@pytest.mark.parametrize("config", ["", "bf16_256x256", "bf16_128x128"])
@pytest.mark.parametrize("M,V,K", [(40, 300, 70), (300, 515, 130), (600, 1001, 1028), (90, 260, 67)])
@pytest.mark.parametrize("pad,at", [(0, 2), (4, 4), (1, 0)])
def test_rows_of_any_alignment_with_nan_around_them(monkeypatch, M, V, K, topk, config, pad, at):
    """Rows that start at multiples of 2, 4 and 8 bytes and end inside a copy's
    16 bytes; nothing around them is read into a result."""
    if config:
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{config} {M} {V} {K} {topk} {pad} {at}")
    c = Case(M, V, K, topk, seed=6)

    def inside(t):
        block = torch.full((at + t.shape[0] * (K + pad) + 64,), NAN, dtype=t.dtype).cuda()
        view = block.as_strided(t.shape, (K + pad, 1), at)
        view.copy_(t)
        return view

    x, w = inside(c.x), inside(c.w)
    loss, lse = c.forward(x=x, w=w)
    c.check_forward(loss, lse, config)
    c.check_backward(lse, *c.backward(lse, x=x, w=w), config)


def test_a_tile_that_does_not_fit_is_refused(monkeypatch):
    c = Case(33, 40, 16)
    for config in ("decode_nt", "bf16_256x192", "f32_64x64", "no such"):
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
        with pytest.raises(g5.GemmError):
            c.forward(workspace=None)


@pytest.mark.parametrize("topk", [0, 9])
@pytest.mark.parametrize("M", [7, 200])
def test_index_and_output_types(M, topk):
    c = Case(M, 400, 96, topk)
    loss, lse = c.forward()
    c.ids = c.ids.to(torch.int32)
    again, _ = c.forward()
    assert torch.equal(loss, again)
    dx, dw = c.backward(lse, dw_dtype=torch.float32)
    assert dw.dtype == torch.float32
    c.check_backward(lse, dx, dw)
    only_x, none = c.backward(lse, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = c.backward(lse, need_dx=False, dw_dtype=torch.float32)
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("topk", [0, 6])
@pytest.mark.parametrize("M", [3, 20, 150])
@pytest.mark.parametrize("pad,at", [(8, 8), (5, 3)])
def test_strided_rows(M, topk, pad, at):
    """Rows inside wider ones, the columns between them untouched."""
    c = Case(M, 300, 72, topk)

    def wide(t):
        b = torch.full((t.shape[0], t.shape[1] + pad + at), NAN, dtype=t.dtype).cuda()
        b[:, at:at + t.shape[1]] = t.cuda()
        return b[:, at:at + t.shape[1]]

    x, w = wide(c.x), wide(c.w)
    loss, lse = c.forward(x=x, w=w)
    c.check_forward(loss, lse)
    bx, bw = (torch.full((n, 72 + pad + at), 7.0, dtype=torch.bfloat16).cuda() for n in (M, 300))
    dx, dw = c.backward(lse, x=x, w=w, dX=bx[:, at:at + 72], dW=bw[:, at:at + 72])
    c.check_backward(lse, dx, dw)
    for b in (bx, bw):
        assert bool((b[:, :at] == 7).all()) and bool((b[:, at + 72:] == 7).all())


@pytest.mark.parametrize("topk", [0, 4])
@pytest.mark.parametrize("M", [6, 40, 300])
def test_rows_left_out_do_not_matter(M, topk):
    """NaN and infinities in rows without targets, in their dloss and lse."""
    c = Case(M, 200, 64, topk)
    _, some, _ = c.targets()
    some[0] = False
    c.ids[0] = c.V if topk == 0 else torch.tensor([-1, c.V, -7, c.V + 5])
    clean_loss, clean_lse = c.forward()
    clean = c.backward(clean_lse)
    c.check_backward(clean_lse, *clean)
    out = ~some
    c.x[out], c.dloss[out] = NAN, INF
    c.x[0] = INF
    loss, lse = c.forward()
    assert torch.equal(loss.cpu()[some], clean_loss.cpu()[some]) and bool((loss.cpu()[out] == 0).all())
    lse[out.cuda()] = NAN
    dx, dw = c.backward(lse)
    assert torch.equal(dx, clean[0]) and torch.equal(dw, clean[1])
    assert bool((dx[out.cuda()] == 0).all())


@pytest.mark.parametrize("topk", [0, 4])
@pytest.mark.parametrize("M", [5, 150])
def test_no_row_has_a_target(M, topk):
    c = Case(M, 100, 40, topk)
    c.ids[:] = -1
    loss, lse = c.forward()
    assert bool((loss == 0).all())
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("M", [4, 140])
def test_nan_stays_in_its_row(M):
    c = Case(M, 150, 64, out=0.0)
    ref, _ = c.forward()
    c.x[1, 3] = NAN
    loss, lse = c.forward()
    keep = torch.arange(M) != 1
    assert torch.equal(loss.cpu()[keep], ref.cpu()[keep]) and math.isnan(float(loss[1])) and math.isnan(float(lse[1]))


@pytest.mark.parametrize("M", [4, 140])
def test_teacher_entries(M):
    """Entries of -inf, the lowest number, one that is far above the rest, rows
    that have no entry but those, an id listed twice."""
    c = Case(M, 90, 48, 6, out=0.1)
    low = torch.finfo(torch.float32).min
    c.t[0] = -INF
    c.t[1, :3] = -INF
    c.ids[1, 3:] = torch.tensor([5, 6, 7])
    c.t[2] = low
    c.t[3, 0], c.ids[3] = 1e30, torch.tensor([3, 3, 4, 4, 4, 90])
    loss, lse = c.forward()
    c.check_forward(loss, lse)
    assert float(loss[0]) == 0
    dx, dw = c.backward(lse)
    c.check_backward(lse, dx, dw)
    assert bool((dx[0] == 0).all())


@pytest.mark.parametrize("M", [2, 130])
@pytest.mark.parametrize("size", [1.0, 40.0, 1e4])
def test_large_logits(M, size):
    """Sure rows, lost rows, logits far apart: nothing overflows."""
    c = Case(M, 120, 64, std=size, out=0.0)
    c.ids = torch.where(torch.arange(M) % 2 == 0, (c.x.double() @ c.w.double().t()).argmax(1), c.ids)
    loss, lse = c.forward()
    assert bool(torch.isfinite(loss).all()) and bool((loss[0::2] >= 0).all())
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse)
    c.check_backward(lse, dx, dw)


@pytest.mark.parametrize("M", [20, 150])
def test_masked_tokens(M):
    """A weight row of large negative logits (a masked token): probability 0."""
    c = Case(M, 70, 32, out=0.0)
    c.x = c.x.abs()
    c.w[5] = -1e30
    c.w[69] = torch.finfo(torch.bfloat16).min
    c.ids[c.ids == 5] = 6
    c.ids[c.ids == 69] = 6
    loss, lse = c.forward()
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())
    keep = [v for v in range(70) if v not in (5, 69)]
    l = (c.x.double() @ c.w[keep].double().t())
    ref = torch.logsumexp(l, 1)
    sums = 1.01 * (32 + 2) * 2.0 ** -23 * (c.x.double().abs() @ c.w[keep].double().abs().t()).max(1).values
    _close(lse, ref, sums + 2.0 ** -16 + 2.0 ** -21 * (l.abs().max(1).values + ref.abs()), "lse")
    dx, dw = c.backward(lse)
    assert bool((dw[5] == 0).all()) and bool((dw[69] == 0).all()) and bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("weights", ["zero", "some zero", "one", "far apart", "negative"])
@pytest.mark.parametrize("M", [9, 140])
def test_weights_of_rows(M, weights):
    c = Case(M, 160, 64)
    if weights == "zero":
        c.dloss[:] = 0
    elif weights == "some zero":
        c.dloss[::2] = 0
    elif weights == "one":
        c.dloss[:] = 1 / 3
    elif weights == "far apart":
        c.dloss = 10.0 ** torch.linspace(-12, 6, M)
    else:
        c.dloss = -c.dloss
    _, lse = c.forward()
    dx, dw = c.backward(lse)
    if weights == "negative":
        c.dloss = -c.dloss
        px, pw = c.backward(lse)
        assert torch.equal(dx, -px) and torch.equal(dw, -pw)
    else:
        c.check_backward(lse, dx, dw)


def test_pieces_of_the_vocabulary():
    """A weight whose rows lie far apart goes in pieces of 256 tokens, a copied
    one of many columns in pieces of 512."""
    c = Case(140, 600, 40, 3)
    big = torch.zeros((600 * 2 ** 21,), dtype=torch.bfloat16, device="cuda")
    w = big.as_strided((600, 40), (2 ** 21, 1))
    w.copy_(c.w)
    loss, lse = c.forward(w=w)
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse, w=w)
    c.check_backward(lse, dx, dw)
    whole = c.backward(lse)
    assert torch.equal(dw, whole[1])
    del big, w
    c = Case(40, 700, 2 ** 18 + 1)
    loss, lse = c.forward()
    c.check_forward(loss, lse)


def test_empty_batch():
    c = Case(1, 50, 24)
    x = torch.zeros((0, 24), dtype=torch.bfloat16).cuda()
    t, f = torch.zeros((0,), dtype=torch.int64).cuda(), torch.zeros((0,)).cuda()
    loss, lse = g5.linear_cross_entropy(x, c.w.cuda(), t)
    assert loss.shape == (0,) and lse.shape == (0,)
    dw = torch.full((50, 24), 3.0).cuda()
    g5.linear_cross_entropy_backward(f, x, c.w.cuda(), t, f, dW=dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("topk", [0, 5])
@pytest.mark.parametrize("M,V,K", [(3, 300, 64), (200, 520, 72)])
def test_captured(M, V, K, topk):
    """Replays with other inputs and targets, the program's own eager calls on
    the same workspace between them."""
    c = Case(M, V, K, topk)
    x, w, ids, dl = c.x.cuda(), c.w.cuda(), c.ids.cuda(), c.dloss.cuda()
    t = c.t.cuda() if topk else None
    space = g5.Workspace()

    def step():
        if topk:
            loss, lse = g5.linear_distill(x, w, ids, t, workspace=space)
            return loss, lse, *g5.linear_distill_backward(dl, x, w, ids, t, lse, workspace=space)
        loss, lse = g5.linear_cross_entropy(x, w, ids, workspace=space)
        return loss, lse, *g5.linear_cross_entropy_backward(dl, x, w, ids, lse, workspace=space)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        other = Case(M, V, K, topk, seed=turn + 1)
        x.copy_(other.x), w.copy_(other.w), ids.copy_(other.ids), dl.copy_(other.dloss)
        if topk:
            t.copy_(other.t)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, step()):
            assert torch.equal(got, want), f"replay {turn}"
        other.check_forward(out[0], out[1], f"replay {turn}")
        other.check_backward(out[1], out[2], out[3], f"replay {turn}")


def test_two_streams():
    cases = [Case(150, 300, 64, 0, seed=1), Case(150, 300, 64, 4, seed=2)]
    inputs = [dict(x=c.x.cuda(), w=c.w.cuda(), ids=c.ids.cuda()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for c, i, s in zip(cases, inputs, streams):
        with torch.cuda.stream(s):
            space = g5.Workspace()
            loss, lse = c.forward(workspace=space, **i)
            outs.append((loss, lse, *c.backward(lse, workspace=space, **i)))
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check_forward(*o[:2])
        c.check_backward(*o[1:])


@pytest.mark.parametrize("M", [1, 16, 31])
def test_a_row_does_not_depend_on_the_others(M):
    c = Case(32, 500, 96, out=0.0)
    loss, lse = c.forward()
    ref = loss.cpu()[:M] if M > 16 else None
    part = g5.linear_cross_entropy(c.x[:M].cuda(), c.w.cuda(), c.ids[:M].cuda(), workspace=ws())[0].cpu()
    if ref is not None:
        assert torch.equal(part, ref)
    c.x[M:] = NAN
    again = c.forward()[0].cpu()[:M]
    assert torch.equal(again, loss.cpu()[:M])


@pytest.mark.parametrize("topk", [0, 3])
def test_gradients_are_the_loss_s(topk):
    """The sum of weighted losses against differences along a direction, in 64
    bits, at the gradient that the library gives."""
    c = Case(40, 90, 32, topk, std=1.0)
    _, lse = c.forward()
    dx, dw = (t.cpu().double() for t in c.backward(lse, dw_dtype=torch.float32))
    q, some, const = c.targets()
    g = torch.Generator().manual_seed(3)
    ux, uw = torch.randn(c.x.shape, generator=g).double(), torch.randn(c.w.shape, generator=g).double()

    def total(h):
        l = (c.x.double() + h * ux) @ (c.w.double() + h * uw).t()
        loss = torch.where(some, const + (q * (torch.logsumexp(l, 1)[:, None] - l)).sum(1), 0.0)
        return float((loss * c.dloss.double()).sum())

    h = 1e-4
    want = (total(h) - total(-h)) / (2 * h)
    got = float((dx * ux).sum() + (dw * uw).sum())
    (_, ex), (_, ew) = c.gradients(lse)
    # the gradients' own bounds, and the differences': h^2 / 6 of the third
    # derivative, for 40 rows whose logits move by up to 20 per unit 1e-3
    bound = float(((ex + 2.0 ** -8 * dx.abs()) * ux.abs()).sum() + ((ew + 2.0 ** -24 * dw.abs()) * uw.abs()).sum()) + 1e-4 * abs(want) + 1e-3
    assert abs(got - want) <= bound, (got, want, bound)


@pytest.mark.parametrize("M", [4, 15])
def test_gradients_of_more_tokens_than_a_piece_holds(M):
    """A vocabulary of 2^23 short rows and some more: two pieces, the first with
    D's rows 2^23 apart.  Against the formula in 64 bits on the GPU."""
    V, K = 2 ** 23 + 4096 + 5, 32
    _say(f"{M} {V} {K}")
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((V, K), generator=g, device="cuda") * 3 * K ** -0.5).bfloat16()
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    ids[:4] = torch.tensor([V - 1, 2 ** 23 - 1, 2 ** 23, 0])
    dloss = torch.rand((M,), generator=g, device="cuda") + 0.25
    loss, lse = g5.linear_cross_entropy(x, w, ids, workspace=ws())
    dx, dw = g5.linear_cross_entropy_backward(dloss, x, w, ids, lse, dw_dtype=torch.float32, workspace=ws())
    torch.cuda.synchronize()
    _say("computed")
    rows = torch.arange(M, device="cuda")
    xd, wd = x.double(), w.double()
    l = xd @ wd.t()
    # FP32 sums of K products; an exponential's argument, of up to |l| + |lse|
    el = 1.01 * (K + 2) * 2.0 ** -23 * (xd.abs() @ wd.abs().t())
    want = torch.logsumexp(l, 1)
    # a part's sum of up to 32, a thread's 1024 parts, and the joins
    tol = el.max(1).values + 1.01 * 1100 * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -21 * (l.abs().max(1).values + want)
    _close(lse, want.cpu(), tol.cpu(), "lse")
    _close(loss, (want - l[rows, ids]).cpu(), (2 * tol).cpu(), "loss")
    lse = lse.double()[:, None]
    p = torch.exp(l - lse)
    ep = p * torch.expm1(el + 2.0 ** -21 * (l.abs() + lse.abs()) + 2.0 ** -20)
    d = p
    d[rows, ids] -= 1
    d, e = dloss.double()[:, None] * d, dloss.double()[:, None] * ep
    del l, el, p, ep
    e += (2.0 ** -16 + 2.0 ** -20) * (d.abs() + e)          # D in two bf16 parts
    for got, a, ea, b, n, half in ((dx, d, e, wd, 2 * V, 2.0 ** -8), (dw, d.t().contiguous(), e.t().contiguous(), xd, 2 * M, 2.0 ** -24)):
        ref = a @ b
        # (dX's sums go in slices of 2^17 tokens, 64 of them and two pieces behind each other)
        tol = (1 + 2.0 ** -8) * (ea @ b.abs() + 1.01 * min(n, 2 * (2 ** 17 + 66)) * 2.0 ** -23 * (a.abs() @ b.abs())) + half * ref.abs() + 2.0 ** -126
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("config", ["", "bf16_128x128", "bf16_256x256"])
@pytest.mark.parametrize("K", [1, 33, 65, 129])
@pytest.mark.parametrize("V", [32, 64, 512, 2048, 2050])
@pytest.mark.parametrize("M", [3, 40, 100])
def test_last_column_of_odd_rows(monkeypatch, M, V, K, config):
    """An odd K: the weight's last element of dX's summed tokens lies in half a
    dword of its own.  Targets at the ends of every stage of 32 tokens, so at
    every slice's end and the vocabulary's."""
    if config:
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{config} {M} {V} {K}")
    c = Case(M, V, K, out=0.0, seed=8)
    c.ids = (V - 1 - 32 * torch.arange(M)) % V
    if V % 32:
        c.ids[1::2] = (31 + 32 * torch.arange(M))[1::2] % V
    c.w[c.ids, -1] = torch.where(torch.arange(M) % 2 == 0, 3.0, -3.0).bfloat16()
    loss, lse = c.forward()
    c.check_forward(loss, lse)
    c.check_backward(lse, *c.backward(lse), config)


@pytest.mark.parametrize("scale", [0.5, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("M", [5, 20, 140])
def test_teacher_entries_far_below_the_rest(M, scale):
    """The lowest number as a list's padding, beside ordinary logits, beside the
    largest and alone: a probability of 0 adds nothing to the loss."""
    c = Case(M, 90, 48, 6, out=0.1, scale=scale, seed=2)
    c.ids[:5] = torch.arange(6) * 7
    low = torch.finfo(torch.float32).min
    c.t[0, 2:] = low
    c.t[1, ::2] = low
    c.t[2, 1:] = low
    c.t[2, 0] = -low
    c.t[3] = low
    c.t[4] = torch.tensor([1e38, -1e38, 3e38, -3e38, 0.0, -INF])
    loss, lse = c.forward()
    assert bool(torch.isfinite(loss).all())
    c.check_forward(loss, lse)
    c.check_backward(lse, *c.backward(lse))


@pytest.mark.parametrize("config", ["", "bf16_128x128", "bf16_256x256"])
@pytest.mark.parametrize("V", [40, 300, 900])
@pytest.mark.parametrize("M", [3, 32, 33, 150, 300])
def test_confident_rows_keep_their_digits(monkeypatch, M, V, config):
    """Logits that FP32 holds exactly, the target's above the rest by 0 to 84:
    losses from log V to 1e-34, each to a bound relative to itself."""
    if config:
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{config} {M} {V}")
    c = Case(M, V, 16, out=0.0, seed=4)
    m = torch.arange(M)
    gap = (7 * m) % 85
    c.ids = 37 * (m % 8) % V
    c.x[:], c.w[:] = 0, 0
    c.x[m, m % 8] = gap.bfloat16()            # the logit above the rest
    c.w[c.ids[:8], torch.arange(min(M, 8))] = 1
    c.x[m, 8 + m % 8] = (m % 5).bfloat16()    # and smaller ones below them
    c.w[::3, 8:] = -1
    l = c.x.double() @ c.w.double().t()
    d = l - l.gather(1, c.ids[:, None])
    d[m, c.ids] = 0
    others = torch.exp(d)
    others[m, c.ids] = 0
    want = torch.log1p(others.sum(1))
    loss, _ = c.forward()
    # Relative: an argument's factor, product and difference (twice, where a
    # part is rescaled) 2^-22 of up to 84 + 2 * 5 each, 2^-22 for either
    # exponential, V roundings of sums of positive terms, the logarithm.  A
    # term below 2^-126 may be 0.
    tol = want * (2 * (94 + 1) * 2.0 ** -22 + 1.01 * (V + 16) * 2.0 ** -24 + 2.0 ** -21) + V * 2.0 ** -126
    # (where another logit is above the target's, their difference is added)
    tol = tol + 2.0 ** -22 * d.max(1).values.clamp(min=0)
    _close(loss, want, tol, f"{config} loss")


@pytest.mark.parametrize("topk", [0, 3])
@pytest.mark.parametrize("config", ["", "bf16_128x128", "bf16_256x256"])
@pytest.mark.parametrize("M", [3, 40, 140, 1100])
def test_gradients_of_pieces_in_slices(monkeypatch, M, config, topk):
    """A weight whose rows lie 2^18 apart goes in pieces of 2048 tokens, dX's
    product of each in slices of 256, dW's of 1100 rows in two: the last piece,
    of 52 tokens, leaves all slices but the first empty, and they keep the sums
    of the piece before."""
    if config:
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{config} {M} {topk}")
    V, K, apart = 2100, 40, 2 ** 18
    c = Case(M, V, K, topk, seed=9)
    if topk == 0:
        c.ids[:3] = torch.tensor([V - 1, 2047, 2048])
    big = torch.zeros((V * apart,), dtype=torch.bfloat16, device="cuda")
    w = big.as_strided((V, K), (apart, 1))
    w.copy_(c.w)
    loss, lse = c.forward(w=w)
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse, w=w, dw_dtype=torch.float32)
    c.check_backward(lse, dx, dw, config)


class FewColumns(Case):
    """x is zero but for some columns, so sums over the others are exact."""

    def __init__(self, M, V, K, topk=0, seed=0):
        super().__init__(M, V, K, topk, seed)
        self.cols = torch.cat([torch.arange(0, K, K // 30), torch.arange(K - 8, K)]).unique()
        self.w[:, self.cols] = (self.w[:, self.cols].float() * (K / len(self.cols)) ** 0.5).bfloat16()
        keep = torch.zeros_like(self.x)
        keep[:, self.cols] = self.x[:, self.cols]
        self.x = keep

    def logits(self):
        x, w = self.x[:, self.cols].double(), self.w[:, self.cols].double()
        return x @ w.t(), 1.01 * (len(self.cols) + 2) * 2.0 ** -23 * (x.abs() @ w.abs().t())


@pytest.mark.parametrize("M", [3, 40, 100])
def test_gradients_of_a_copied_weight_in_pieces(M):
    """Rows of 2^18 + 1 elements are copied to padded ones, 256 tokens at a time:
    D streamed, in two parts and in one, dX's sums carried from piece to piece."""
    V, K = 600, 2 ** 18 + 1
    _say(f"{M}")
    c = FewColumns(M, V, K)
    c.ids[:3] = torch.tensor([V - 1, 255, 256])
    loss, lse = c.forward()
    c.check_forward(loss, lse)
    dx, dw = c.backward(lse, dw_dtype=torch.float32)
    c.check_backward(lse, dx, dw)
