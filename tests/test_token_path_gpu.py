"""The token operators run together, as a model's layer calls them: one
residual stream through norm, adapted projection, router, experts and a
quantized product (decode), and a norm and a product with their gradients.

Each step is held to its own formula in 64 bits on the values the step before
left on the device, with the bounds of that operator's own tests; so a wrong
value anywhere is seen where it arises and no bound has to follow a whole
chain.
"""
import pytest
import torch

import dense_gemm_05_amd as g5
import test_lora_gpu as lora
import test_moe_gpu as moe
import test_norm_gpu as norm

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _say(msg):
    print(f"[path] {msg}", flush=True)


def _check(got, ref, tol, what):
    norm._check(got.cpu().double(), ref, tol, what)


def _norm_ref(h, w):
    hd = h.cpu().double()
    return hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + float(torch.tensor(EPS))) * w.cpu().double()


def _product_ref(x, w, half):
    """x . w^T and its bound: FP32 sums, the output's rounding (half a step)."""
    x, w = x.cpu().double(), w.cpu().double()
    ref = x @ w.t()
    return ref, half * ref.abs() + 1.01 * x.shape[1] * 2.0 ** -24 * (x.abs() @ w.abs().t()) + norm.TINY


class _Layer:
    def __init__(self, g, T, H, N, I, E, k, L, R, V, codes):
        self.k = k
        self.o, self.x = norm._bf((T, H), g).cuda(), norm._bf((T, H), g).cuda()
        self.w = [norm._bf((H,), g).cuda() for _ in range(3)]
        _, wq, a, b, scale, idx = lora._inputs(g, T, N, H, L, R)
        self.wq, self.a, self.b, self.scale, self.idx = (t.cuda() for t in (wq, a, b, scale, idx))
        self.wo = (torch.randn((H, N), generator=g) * N ** -0.5).bfloat16().cuda()
        self.wr = (torch.randn((E, H), generator=g) * H ** -0.5).bfloat16().cuda()
        _, _, *experts = moe._inputs(g, T, H, I, E, codes)
        self.wgu, self.wd, self.sgu, self.sd = (None if t is None else t.cuda() for t in experts)
        head = (torch.randn((V, H), generator=g) * H ** -0.5).bfloat16().cuda()
        self.head, self.shead = g5.gemm_fp8_quantize_rows(head, Q=self._codes(V, H))

    @staticmethod
    def _codes(rows, cols):
        """(the FP8 product takes rows that start at 16-byte boundaries)"""
        return torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device="cuda")[:, :cols]

    def step(self, ws):
        r = {}
        r["y1"], r["h1"] = g5.rms_norm(self.o, self.w[0], residual=self.x, eps=EPS)
        r["q"] = g5.gemm_bf16_nt_lora(r["y1"], self.wq, self.a, self.b, self.idx, scale=self.scale, workspace=ws)
        r["p"] = g5.gemm_bf16_nt(r["q"], self.wo, workspace=ws)
        r["y2"], r["h2"] = g5.rms_norm(r["p"], self.w[1], residual=r["h1"], eps=EPS)
        r["logits"] = g5.gemm_bf16_nt(r["y2"], self.wr, out_dtype=torch.float32, workspace=ws)
        r["m"], r["ids"], r["gates"] = g5.moe_swiglu(r["y2"], r["logits"], self.k, self.wgu, self.wd, scale_gu=self.sgu,
                                                     scale_d=self.sd, workspace=ws)
        # (the sum may stand in its residual's place)
        h3 = r["h2"].clone()
        r["c"], r["s"], r["h3"] = g5.rms_norm_e4m3(r["m"], self.w[2], residual=h3, eps=EPS, H=h3,
                                                   Q=self._codes(*h3.shape))
        r["out"] = g5.gemm_fp8_nt(r["c"], r["s"], self.head, self.shead, out_dtype=torch.float32, workspace=ws)
        return r

    def check(self, r):
        half = 2.0 ** -8

        def sums(got, a, b, what):
            s = a.cpu().double() + b.cpu().double()
            _check(got, s, (half + 2.0 ** -23) * s.abs() + norm.TINY, what)

        def normed(y, h, w, what):
            ref = _norm_ref(h, w)
            _check(y, ref, (half + 2.0 ** -16) * ref.abs() + norm.TINY, what)

        sums(r["h1"], self.o, self.x, "h1")
        normed(r["y1"], r["h1"], self.w[0], "y1")
        ref, tol = lora._formula(*(t.cpu() for t in (r["y1"], self.wq, self.a, self.b, self.scale, self.idx)))
        _check(r["q"], ref, half * ref.abs() + (1 + half) * tol, "q")
        _check(r["p"], *_product_ref(r["q"], self.wo, half), "p")
        sums(r["h2"], r["p"], r["h1"], "h2")
        normed(r["y2"], r["h2"], self.w[1], "y2")
        _check(r["logits"], *_product_ref(r["y2"], self.wr, 2.0 ** -24), "logits")
        ref, tol, ids, gates = moe._formula(*(None if t is None else t.cpu() for t in (
            r["y2"], r["logits"], self.wgu, self.wd, self.sgu, self.sd)), self.k, True)
        assert torch.equal(r["ids"].cpu().long(), ids)
        _check(r["gates"], gates, 2.0 ** -20 * gates, "gates")
        _check(r["m"], ref, half * ref.abs() + (1 + half) * tol, "m")
        sums(r["h3"], r["m"], r["h2"], "h3")
        y3 = g5.rms_norm(r["h3"], self.w[2], eps=EPS)
        normed(y3, r["h3"], self.w[2], "y3")
        c, s = g5.gemm_fp8_quantize_rows(y3)
        assert torch.equal(r["c"], c) and torch.equal(r["s"], s)
        x = r["c"].cpu().view(torch.float8_e4m3fn).double()
        w = self.head.cpu().view(torch.float8_e4m3fn).double()
        f = r["s"].cpu().double()[:, None] * self.shead.cpu().double()
        ref, mag = (x @ w.t()) * f, (x.abs() @ w.abs().t()) * f
        # A step, not half a step, per addition: the FP8 matrix instruction
        # adds many products at once and need not round the sums inside it to
        # nearest.  One that cuts off errs by up to a step of the partial sum,
        # 2^-23 of at most mag, at each of the K additions.
        _check(r["out"], ref, 1.01 * x.shape[1] * 2.0 ** -23 * mag + 2.0 ** -22 * ref.abs(), "out")


SIZES = [  # T, H, N, I, E, topk, adapters, rank, V, codes
    (1, 512, 384, 128, 8, 2, 3, 16, 200, False), (12, 520, 264, 72, 16, 4, 5, 12, 136, False),
    (33, 256, 512, 96, 6, 2, 4, 8, 320, True), (64, 1028, 260, 40, 40, 8, 9, 16, 100, True),
]


@pytest.mark.parametrize("size", SIZES)
def test_decode_layer(size):
    """The layer on one shared workspace, and captured with a workspace of its
    own and replayed on new tokens between eager steps."""
    _say(f"layer {size}")
    g = norm._gen(11, *size)
    layer = _Layer(g, *size)
    ws, held = g5.Workspace(), g5.Workspace()
    layer.check(layer.step(ws))
    layer.step(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(held)
    for n in range(3):
        layer.o.copy_(norm._bf(layer.o.shape, g))
        layer.idx.copy_(torch.randint(-1, layer.a.shape[0], layer.idx.shape, generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        want = layer.step(ws)
        for k in want:
            assert torch.equal(got[k], want[k]), f"replay {n}: {k}"
    layer.check(got)


@pytest.mark.parametrize("M,K,N", [(200, 264, 136), (48, 1032, 520)])
def test_norm_and_product_with_gradients(M, K, N):
    """f = sum dC (norm(X + R) . Wt^T) + sum dH (X + R): its gradients by the
    framework's calls against the formulas at the device's sum."""
    _say(f"gradients {M}x{K}x{N}")
    g = norm._gen(12, M, K, N)
    x, r, w, wt, dc, dh = (norm._bf(s, g).cuda() for s in ((M, K), (M, K), (K,), (N, K), (M, N), (M, K)))
    ws, rstd = g5.Workspace(), torch.empty((M,), device="cuda")
    y, h = g5.rms_norm(x, w, residual=r, eps=EPS, rstd=rstd)
    _check(g5.gemm_bf16_nt(y, wt, workspace=ws), *_product_ref(y, wt, 2.0 ** -8), "C")
    dy = g5.gemm_bf16(dc, wt, workspace=ws)
    dwt = g5.gemm_bf16_tn(dc, y, out_dtype=torch.float32, workspace=ws)
    dx, dw = g5.rms_norm_backward(dy, h, w, rstd, dH=dh, workspace=ws)
    _check(dwt, *_product_ref(dc.t(), y.t(), 2.0 ** -24), "dWt")
    ref, tol = _product_ref(dc, wt.t(), 2.0 ** -8)
    _check(dy, ref, tol, "dY")
    # the gradient in 64 bits by differentiation, at the device's h
    hd, wd = h.cpu().double().requires_grad_(), w.cpu().double().requires_grad_()
    rs = 1.0 / torch.sqrt((hd * hd).mean(1, keepdim=True) + float(torch.tensor(EPS)))
    c = (hd * rs * wd) @ wt.cpu().double().t()
    ((c * dc.cpu().double()).sum() + (hd * dh.cpu().double()).sum()).backward()
    # dY's own error goes through the norm's gradient, which is linear in dY;
    # rstd is within 2^-17, dX's terms have it three times at most
    _, gtol, _, wtol = norm._grad_ref(dy.cpu(), h.cpu(), w.cpu(), rstd.cpu(), dh.cpu())
    rs, xh = rs.detach(), (hd * rs).detach().abs()
    aw, ay = wd.detach().abs(), ref.abs() + tol
    through = rs * (aw * tol + xh * (aw * tol * xh).mean(1, keepdim=True))
    mag = rs * (aw * ay + xh * (aw * ay * xh).mean(1, keepdim=True))
    _check(dx, hd.grad, gtol + 1.01 * through + 2.0 ** -15 * mag, "dX")
    _check(dw, wd.grad, wtol + 1.01 * ((tol + 2.0 ** -17 * ay) * xh).sum(0), "dW")


def test_two_graphs_on_one_workspace():
    """A projection with adapters and an expert layer, both joining slices
    through the workspace, captured apart on one workspace and replayed in
    turn, with eager calls on it between."""
    g = norm._gen(13)
    M, N, K = 77, 264, 1100
    x, w, a, b, scale, idx = (t.cuda() for t in lora._inputs(g, M, N, K, 4, 24))
    T, H, I, E, k = 40, 2100, 72, 6, 3
    y, logits, gu, wd, _, _ = (None if t is None else t.cuda() for t in moe._inputs(g, T, H, I, E, False))
    ws = g5.Workspace(nbytes=64 << 20)
    one = lambda: g5.gemm_bf16_nt_lora(x, w, a, b, idx, scale=scale, workspace=ws)     # noqa: E731
    two = lambda: g5.moe_swiglu(y, logits, k, gu, wd, workspace=ws)[0]                 # noqa: E731
    want, graphs, outs = [one(), two()], [], []
    held = ws.buf.data_ptr()
    for call in (one, two):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call())
    for turn in range(4):
        x.copy_(norm._bf((M, K), g))
        y.copy_(norm._bf((T, H), g))
        for graph in graphs[::1 if turn % 2 else -1]:
            graph.replay()
        got = [o.clone() for o in outs]
        want = [one(), two()]
        for n in (0, 1):
            assert torch.equal(got[n], want[n]), f"turn {turn}, graph {n}"
    assert ws.buf.data_ptr() == held and not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()


def test_calls_on_two_streams_at_once():
    """The same two operators on two streams, each with its own workspace."""
    g = norm._gen(14)
    M, N, K = 100, 512, 2048
    x, w, a, b, scale, idx = (t.cuda() for t in lora._inputs(g, M, N, K, 4, 16))
    T, H, I, E, k = 33, 2304, 64, 8, 2
    y, logits, gu, wd, _, _ = (None if t is None else t.cuda() for t in moe._inputs(g, T, H, I, E, False))
    spaces = [g5.Workspace(), g5.Workspace()]
    calls = [lambda ws: g5.gemm_bf16_nt_lora(x, w, a, b, idx, scale=scale, workspace=ws),
             lambda ws: g5.moe_swiglu(y, logits, k, gu, wd, workspace=ws)[0]]
    want = [c(s) for c, s in zip(calls, spaces)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(calls[n](spaces[n]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[n]) for n in (0, 1) for o in got[n])
