"""GPU parity of the mixture-of-experts layer (gemm_moe_swiglu) against the
formula in 64 bits.

The bound of y, from the roundings the kernels take.  Products of bf16 (or
E4M3) values are exact in FP32; a sum of K of them is within K 2^-24 of the
sum of their magnitudes, in any order.  So
  eg, eu = H 2^-24 sum|x w|                    (the gate and up sums)
  dz = 1.1 eg |u| + |silu| eu + 2 eg eu        (1.1 bounds |silu'|)
       + (2^-20 (1 + |g|) + 2^-16) |z|         (exp and reciprocal; hi + lo)
  dy = sum_s gate (sum_i dz |wd| + (I + 4) 2^-24 sum_i |z wd|)
       + (2^-18 + topk 2^-24) sum_s |gate y_s| (the gate's exp, scales, join)
and the output's own rounding, 2^-8 |y| for bf16.  A factor of 1.01 covers
the second-order terms.  Ids are whole numbers and equal.
"""
import pytest
import torch

import dense_gemm_05_amd as g5

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[experts] {msg}", flush=True)


def _gen(*key):
    return torch.Generator().manual_seed(hash(key) % (1 << 31))


def _strided(t, kind):
    """The same values on the GPU: contig, padded rows (16-byte aligned) or
    rows at an odd offset and stride."""
    if kind == "contig":
        return t.cuda()
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    *lead, cols = raw.shape
    n = 1
    for d in lead:
        n *= d
    ld = (cols + 15) // 16 * 16 + 16 if kind == "padded" else cols + 3
    off = 0 if kind == "padded" else 1
    buf = torch.zeros((n * ld + off,), dtype=raw.dtype, device="cuda")
    v = buf[off:].view(*lead, ld)[..., :cols]
    v.copy_(raw)
    return v


def _inputs(g, T, H, I, E, codes):
    x = torch.randn((T, H), generator=g).bfloat16()
    logits = torch.randn((T, E), generator=g)
    if codes:
        wgu = (torch.randn((E, 2 * I, H), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        wd = (torch.randn((E, H, I), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        sgu = (torch.rand((E, 2 * I), generator=g) + 0.5) * (0.01 * H ** -0.5)
        sd = (torch.rand((E, H), generator=g) + 0.5) * 0.01
    else:
        wgu = (torch.randn((E, 2 * I, H), generator=g) * H ** -0.5).bfloat16()
        wd = torch.randn((E, H, I), generator=g).bfloat16()
        sgu = sd = None
    return x, logits, wgu, wd, sgu, sd


def _route(logits, k, renorm):
    l = torch.where(logits.isnan(), -torch.inf, logits).double()
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k].clone(), order.values[:, :k]
    none = top == -torch.inf
    m = torch.where(none[:, :1], 0.0, order.values[:, :1])
    e = torch.exp(top - m)
    den = e.sum(1, keepdim=True) if renorm else torch.exp(l - m).sum(1, keepdim=True)
    gates = torch.where(none, 0.0, e / torch.where(den > 0, den, 1.0))
    ids[none] = -1
    return ids, gates


def _formula(x, logits, wgu, wd, sgu, sd, k, renorm):
    """(y, its error bound before the output's rounding, ids, gates)"""
    T, H = x.shape
    I = wd.shape[2]
    ids, gates = _route(logits, k, renorm)
    y, tol = torch.zeros((T, H)).double(), torch.zeros((T, H)).double()
    x = x.double()
    for t in range(T):
        for s in range(k):
            e = int(ids[t, s])
            if e < 0:
                continue
            w, d = wgu[e].double(), wd[e].double()
            if sgu is not None:
                w, d = w * sgu[e].double()[:, None], d * sd[e].double()[:, None]
            a, mag = w @ x[t], H * 2.0 ** -24 * (w.abs() @ x[t].abs())
            g, u, eg, eu = a[:I], a[I:], mag[:I], mag[I:]
            si = g * torch.sigmoid(g)
            z = si * u
            dz = 1.1 * eg * u.abs() + si.abs() * eu + 2 * eg * eu + (2.0 ** -20 * (1 + g.abs()) + 2.0 ** -16) * z.abs()
            ys, gt = d @ z, float(gates[t, s])
            y[t] += gt * ys
            tol[t] += gt * (d.abs() @ dz + (I + 4) * 2.0 ** -24 * (d.abs() @ z.abs()))
            tol[t] += (2.0 ** -18 + k * 2.0 ** -24) * gt * ys.abs()
    return y, 1.01 * tol, ids, gates


def _check(got, ref, tol, what):
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} out of bound, worst {float((err / tol).max())}"


CASES = [  # T, H, I, E, topk, codes, renormalize, layout
    (1, 256, 64, 8, 2, False, True, "contig"), (1, 520, 72, 4, 4, False, False, "contig"),
    (5, 264, 40, 16, 3, False, True, "padded"), (7, 100, 33, 5, 2, False, False, "odd"),
    (17, 512, 130, 3, 2, False, True, "contig"), (40, 192, 48, 2, 1, False, True, "contig"),
    (50, 128, 64, 4, 3, False, False, "padded"), (64, 128, 32, 130, 8, False, True, "contig"),
    (64, 64, 32, 3, 2, False, True, "contig"), (3, 1, 1, 1, 1, False, True, "contig"),
    (9, 96, 24, 300, 16, False, False, "contig"), (2, 64, 16, 1024, 5, False, True, "contig"),
    (1, 256, 64, 8, 2, True, True, "contig"), (6, 320, 96, 6, 2, True, False, "padded"),
    (7, 100, 33, 5, 2, True, True, "odd"), (33, 528, 80, 3, 2, True, False, "contig"),
    (64, 128, 64, 2, 1, True, True, "contig"), (1, 2048, 512, 4, 2, False, True, "contig"),
    (2, 1100, 64, 3, 2, False, True, "contig"), (2, 2304, 64, 3, 2, True, True, "contig"),
    (64, 40, 24, 16, 16, False, True, "contig"),
]


@pytest.mark.parametrize("T,H,I,E,k,codes,renorm,kind", CASES)
def test_experts(T, H, I, E, k, codes, renorm, kind):
    _say(f"T={T} H={H} I={I} E={E} topk={k} codes={codes} {kind}")
    x, logits, wgu, wd, sgu, sd = _inputs(_gen(1, T, H, I, E, k), T, H, I, E, codes)
    y, tol, ids, gates = _formula(x, logits, wgu, wd, sgu, sd, k, renorm)
    dev = (_strided(x, kind), logits.cuda(), k, _strided(wgu, kind), _strided(wd, kind))
    more = dict(scale_gu=None if sgu is None else sgu.cuda(), scale_d=None if sd is None else sd.cuda(),
                renormalize=renorm)
    ws = g5.Workspace()
    got, gi, gg = g5.moe_swiglu(*dev, **more, out_dtype=torch.float32, workspace=ws)
    assert torch.equal(gi.cpu().long(), ids)
    _check(gg.cpu().double(), gates, 2.0 ** -20 * gates, "gates")
    _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), "y float")
    assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
    # scratch left by another call does not matter; a padded bf16 output
    ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
    out = torch.full((T, H + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    b16, _, _ = g5.moe_swiglu(*dev, **more, Y=out[:, :H], workspace=ws)
    assert torch.equal(b16, got.bfloat16()) and (out[:, H:] == 3.0).all()
    # a token's result does not depend on the others
    for t in {0, T // 2, T - 1}:
        one = g5.moe_swiglu(dev[0][t:t + 1], dev[1][t:t + 1], *dev[2:], **more, out_dtype=torch.float32, workspace=ws)
        assert torch.equal(one[0][0], got[t]) and torch.equal(one[1][0], gi[t]) and torch.equal(one[2][0], gg[t])


@pytest.mark.parametrize("T,H,I,E,k,codes,kind", [
    (17, 2056, 72, 40, 2, False, "contig"), (40, 2100, 33, 2, 2, False, "odd"), (64, 4096, 64, 6, 3, True, "contig"),
    (33, 2049, 200, 3, 1, True, "odd"), (64, 2080, 130, 30, 16, False, "padded"), (64, 2304, 1, 16, 4, True, "padded")])
def test_experts_for_many_tokens_and_wide_rows(T, H, I, E, k, codes, kind):
    """More than 16 tokens and 2048 hidden columns: the down kernel's halves,
    with any number of tokens per expert and odd ends; again on scratch that
    another call left."""
    _say(f"T={T} H={H} I={I} E={E} topk={k} codes={codes} {kind}")
    x, logits, wgu, wd, sgu, sd = _inputs(_gen(5, T, H, I, E, k), T, H, I, E, codes)
    logits[T // 2], logits[1, 1:] = -torch.inf, torch.nan      # a token without experts, one with one
    y, tol, ids, gates = _formula(x, logits, wgu, wd, sgu, sd, k, True)
    dev = (_strided(x, kind), logits.cuda(), k, _strided(wgu, kind), _strided(wd, kind))
    more = dict(scale_gu=None if sgu is None else sgu.cuda(), scale_d=None if sd is None else sd.cuda())
    ws, out = g5.Workspace(), torch.full((T + 1, H + 3), 7.0, device="cuda")
    for turn in range(2):
        got, gi, gg = g5.moe_swiglu(*dev, **more, Y=out[:T, :H], workspace=ws)
        assert torch.equal(gi.cpu().long(), ids)
        _check(gg.cpu().double(), gates, 2.0 ** -20 * gates, "gates")
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), "y float")
        assert (out[T:] == 7.0).all() and (out[:, H:] == 7.0).all() and not got[T // 2].any()
        assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
        ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
    b16 = g5.moe_swiglu(*dev, **more, workspace=ws)[0]
    assert torch.equal(b16, got.bfloat16())


def test_expert_choice():
    """Ties, masked experts, rows whose mask leaves fewer than topk or none,
    NaN logits, the type's lowest value."""
    g = _gen(2)
    T, H, I, E, k = 8, 64, 32, 70, 4
    x, logits, wgu, wd, _, _ = _inputs(g, T, H, I, E, False)
    low = torch.finfo(torch.float32).min
    logits[0] = 0.5                                   # all equal
    logits[1] = -torch.inf                            # none
    logits[2] = -torch.inf
    logits[2, [65, 3]] = torch.tensor([1.0, 1.0])     # two of four, equal
    logits[3, 10:] = torch.nan
    logits[4] = low                                   # masked by the lowest value: a finite logit
    logits[4, 7] = 0.0
    logits[5] = torch.nan
    logits[6, ::2] = logits[6, 0]
    logits[7, 1] = -0.0
    logits[7, 0] = 0.0
    for renorm in (True, False):
        y, tol, ids, gates = _formula(x, logits, wgu, wd, None, None, k, renorm)
        got, gi, gg = g5.moe_swiglu(x.cuda(), logits.cuda(), k, wgu.cuda(), wd.cuda(), renormalize=renorm,
                                    out_dtype=torch.float32)
        assert torch.equal(gi.cpu().long(), ids)
        _check(gg.cpu().double(), gates, 2.0 ** -20 * gates, "gates")
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), "y")
        assert (got[1] == 0).all() and (got[5] == 0).all() and (gi[1] == -1).all()
    assert list(gi[0]) == [0, 1, 2, 3] and list(gi[4]) == [7, 0, 1, 2]


def test_expert_values_stay_in_their_rows():
    """NaN and infinities of a token, or of an expert nobody chose, reach no
    other token; an infinite z stays infinite."""
    g = _gen(3)
    T, H, I, E, k = 6, 128, 48, 6, 2
    x, logits, wgu, wd, _, _ = _inputs(g, T, H, I, E, False)
    logits[:, 4] = -torch.inf
    clean = g5.moe_swiglu(x.cuda(), logits.cuda(), k, wgu.cuda(), wd.cuda())[0]
    x2, w2, d2 = x.clone(), wgu.clone(), wd.clone()
    x2[2, 5], x2[3] = torch.nan, torch.inf
    w2[4], d2[4] = torch.nan, torch.inf
    got = g5.moe_swiglu(x2.cuda(), logits.cuda(), k, w2.cuda(), d2.cuda())[0]
    for t in (0, 1, 4, 5):
        assert torch.equal(got[t], clean[t])
    assert got[2].isnan().all()
    # one expert, positive everything: z overflows bf16's range to +inf and y follows
    one = torch.full((1, 64), 1e20).bfloat16()
    w = torch.full((1, 2, 64), 1.0).bfloat16()
    d = torch.full((1, 64, 1), 1.0).bfloat16()
    y = g5.moe_swiglu(one.cuda(), torch.zeros((1, 1), device="cuda"), 1, w.cuda(), d.cuda(),
                      out_dtype=torch.float32)[0]
    assert (y == torch.inf).all()


def test_experts_empty():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w, d = torch.zeros((4, 16, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 64, 8), dtype=torch.bfloat16, device="cuda")
    y, ids, gates = g5.moe_swiglu(e, torch.empty((0, 4), device="cuda"), 2, w, d)
    assert y.shape == (0, 64) and ids.shape == gates.shape == (0, 2)
    x, l = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 4), device="cuda")
    y, ids, _ = g5.moe_swiglu(x, l, 2, w[:, :0], d[:, :, :0])
    assert not y.any() and (ids.cpu() == torch.tensor([0, 1])).all()


def test_experts_on_a_stream_and_in_a_graph():
    """Another stream with its own workspace, and a captured layer replayed on
    new tokens and logits between eager calls on another workspace."""
    g = _gen(4)
    T, H, I, E, k = 12, 512, 128, 16, 4
    x, logits, wgu, wd, _, _ = (None if t is None else t.cuda() for t in _inputs(g, T, H, I, E, False))
    eager, held = g5.Workspace(), g5.Workspace()
    want = g5.moe_swiglu(x, logits, k, wgu, wd, workspace=eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = g5.moe_swiglu(x, logits, k, wgu, wd, workspace=held)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g5.moe_swiglu(x, logits, k, wgu, wd, workspace=held)
    for r in range(4):
        x.copy_(torch.randn((T, H), generator=g).bfloat16())
        logits.copy_(torch.randn((T, E), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = g5.moe_swiglu(x, logits, k, wgu, wd, workspace=eager)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {r}"


@pytest.mark.parametrize("T,H,I,E,k,codes", [
    (17, 4096, 200, 6, 3, False), (64, 2304, 320, 5, 2, True), (33, 2100, 130, 4, 4, False)])
def test_a_token_among_many_is_the_token_alone(T, H, I, E, k, codes):
    """The bits of a token's result are the same alone, among 16 and among
    more, also at the widths where larger calls divide the work otherwise."""
    _say(f"alone T={T} H={H} I={I} E={E} topk={k} codes={codes}")
    x, logits, wgu, wd, sgu, sd = (None if t is None else t.cuda() for t in _inputs(_gen(6, T, H, I), T, H, I, E, codes))
    ws = g5.Workspace()
    call = lambda n0, n1: g5.moe_swiglu(x[n0:n1], logits[n0:n1], k, wgu, wd, scale_gu=sgu, scale_d=sd,    # noqa: E731
                                        out_dtype=torch.float32, workspace=ws)[0]
    all_of_them = call(0, T)
    assert torch.equal(call(T - 16, T), all_of_them[T - 16:])
    for t in range(0, T, 5):
        assert torch.equal(call(t, t + 1)[0], all_of_them[t]), f"token {t}"


@pytest.mark.parametrize("I", [32, 33, 120])
def test_experts_store_no_columns_past_the_inner_ones(I):
    """z's rows (128 bf16 apart, behind the routing's five parts of 256 bytes)
    hold I columns: what stands behind them is neither written nor read."""
    x, logits, wgu, wd, _, _ = _inputs(_gen(9, I), 4, 64, I, 8, False)
    dev = x.cuda(), logits.cuda(), 2, wgu.cuda(), wd.cuda()
    ws, at = g5.Workspace(), g5.GEMM_WORKSPACE_COUNTER_BYTES + 5 * 256
    want = g5.moe_swiglu(*dev, workspace=ws)[0]
    ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255         # (NaN as z)
    assert torch.equal(g5.moe_swiglu(*dev, workspace=ws)[0], want)
    z = ws.buf[at:at + 2 * 8 * 128 * 2].view(torch.int16).view(16, 128)
    assert (z[:, I:] == -1).all() and (z[:, :I] != -1).all()
