"""Products grouped by expert against the formula in 64 bits: forward, input
gradient and weight gradient, ragged and empty groups, odd sizes and strides,
rows of no group, values that must not reach other groups."""
import random

import pytest
import torch

import dense_gemm_05_amd as g5
from _gpu_helpers import ws

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _say(msg):
    print(f"[grouped] {msg}", flush=True)


def _bf(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def _offsets(sizes, first=0):
    o = [first]
    for n in sizes:
        o.append(o[-1] + n)
    return o


def _formula(kind, a, b, o):
    """(C, bound of the FP32 sums), in 64 bits: at most K additions and
    products in any order, each off by at most a step of 2^-23 of the sum of
    the terms' sizes (the matrix instruction need not round to nearest inside)."""
    a, b = a.double(), b.double()
    E = len(o) - 1
    if kind == "tn":
        c = torch.zeros((E, a.shape[1], b.shape[1])).double()
        tol = torch.zeros_like(c)
        for e in range(E):
            x, y = a[o[e]:o[e + 1]], b[o[e]:o[e + 1]]
            c[e], tol[e] = x.t() @ y, 1.01 * x.shape[0] * 2.0 ** -23 * (x.abs().t() @ y.abs())
        return c, tol
    w = b.transpose(1, 2) if kind == "nt" else b
    c = torch.zeros((a.shape[0], w.shape[2])).double()
    tol = torch.zeros_like(c)
    for e in range(E):
        x = a[o[e]:o[e + 1]]
        c[o[e]:o[e + 1]] = x @ w[e]
        tol[o[e]:o[e + 1]] = 1.01 * a.shape[1] * 2.0 ** -23 * (x.abs() @ w[e].abs())
    return c, tol


def _check(got, ref, tol, what):
    half = torch.finfo(got.dtype).eps / 2
    got = got.cpu().double()
    bad = ~((got - ref).abs() <= half * ref.abs() + (1 + half) * tol + 2.0 ** -133)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, first at {bad.nonzero()[0].tolist()}"


ENTRY = {"nt": "gemm_bf16_grouped_nt", "nn": "gemm_bf16_grouped", "tn": "gemm_bf16_grouped_tn"}


def _case(kind, sizes, n, k, seed, first=0, behind=0):
    """Operands [rows, k] and weights, or [rows, n] and [rows, k] for tn."""
    g = torch.Generator().manual_seed(seed)
    o = _offsets(sizes, first)
    rows, E = o[-1] + behind, len(sizes)
    if kind == "tn":
        return _bf((rows, n), g), _bf((rows, k), g), o
    return _bf((rows, k), g), _bf((E, n, k) if kind == "nt" else (E, k, n), g, k ** -0.5), o


def _run(kind, a, b, o, **kw):
    return getattr(g5, ENTRY[kind])(a.cuda(), b.cuda(), torch.tensor(o, dtype=torch.int32).cuda(), workspace=ws(), **kw)


SIZES = [  # group sizes, n, k
    ([1], 8, 8), ([1], 1, 1), ([3, 0, 1], 17, 33), ([0, 0, 5, 0], 64, 64), ([16, 17, 1, 32, 33], 40, 72),
    ([40, 100, 0, 64, 129], 136, 96), ([300, 1, 0, 513], 264, 200), ([256, 256], 256, 128), ([255, 257], 272, 160),
    ([700], 520, 100), ([90, 33, 47], 130, 101), ([1] * 70, 24, 40), ([0] * 65 + [2, 7], 32, 64), ([128], 96, 32),
    ([2000, 5], 48, 31), ([0, 0], 16, 16)]


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes,n,k", SIZES)
def test_grouped_matches_the_formula(kind, sizes, n, k):
    _say(f"{kind} {sizes[:6]} {n} {k}")
    a, b, o = _case(kind, sizes, n, k, seed=sum(sizes) + n)
    ref, tol = _formula(kind, a, b, o)
    for dt in (torch.bfloat16, torch.float32):
        _check(_run(kind, a, b, o, out_dtype=dt), ref, tol, f"{kind} {dt}")


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("config", ["bf16_256x256", "bf16_128x128", "decode_nt"])
@pytest.mark.parametrize("sizes,n,k", [([5, 0, 40, 1], 48, 72), ([300, 130, 2], 264, 136), ([33, 31, 65], 100, 257)])
def test_every_tile_takes_every_size(monkeypatch, kind, config, sizes, n, k):
    if config == "decode_nt" and kind != "nt":
        pytest.skip("the stream is the projection's")
    monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{kind} {config} {sizes} {n} {k}")
    a, b, o = _case(kind, sizes, n, k, seed=7)
    _check(_run(kind, a, b, o), *_formula(kind, a, b, o), f"{kind} {config}")


@pytest.mark.parametrize("sizes,n,k", [([5000], 40, 72), ([2000, 0, 3100], 130, 33), ([1, 6000], 64, 260), ([700, 700, 0, 2900], 128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_weight_gradients_of_many_rows(sizes, n, k, dtype):
    """Summed in slices of the rows: the same bits in every call, also beside
    other columns."""
    _say(f"slices {sizes} {n} {k} {dtype}")
    a, b, o = _case("tn", sizes, n, k, seed=13)
    c = _run("tn", a, b, o, out_dtype=dtype)
    _check(c, *_formula("tn", a, b, o), f"slices {sizes}")
    wide = torch.full((len(sizes), n + 2, k + 3), 7.0, dtype=dtype).cuda()
    part = wide[:, 1:n + 1, 1:k + 1]
    assert _run("tn", a, b, o, C=part) is part and torch.equal(part, c)
    part.fill_(7.0)
    assert bool((wide == 7).all())


def _inside(t, pad, at):
    """t's rows `pad` elements further apart, `at` elements behind the start of
    a block that is NaN around them and right behind the last one."""
    rows, cols = t.reshape(-1, t.shape[-1]).shape
    block = torch.full((at + rows * (cols + pad) + 64,), NAN, dtype=t.dtype).cuda()
    strides = (cols + pad, 1) if t.dim() == 2 else (t.shape[1] * (cols + pad), cols + pad, 1)
    view = block.as_strided(t.shape, strides, at)
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("config", ["", "bf16_256x256", "bf16_128x128"])
@pytest.mark.parametrize("sizes,n,k", [([300, 0, 131, 3], 130, 70), ([90, 257], 268, 196), ([64, 65, 1], 34, 1030), ([200, 70], 93, 71)])
@pytest.mark.parametrize("pad,at", [(0, 2), (4, 4), (1, 0)])
def test_rows_of_any_alignment_with_nan_around_them(monkeypatch, kind, config, sizes, n, k, pad, at):
    """Rows that start at multiples of 2, 4 and 8 bytes and end inside a copy's
    16 bytes; nothing around them is read into a result."""
    if config:
        monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    _say(f"{kind} {config} {sizes} {n} {k} {pad} {at}")
    a, b, o = _case(kind, sizes, n, k, seed=12)
    ref, tol = _formula(kind, a, b, o)
    c = getattr(g5, ENTRY[kind])(_inside(a, pad, at), _inside(b, pad, at), torch.tensor(o, dtype=torch.int32).cuda(),
                                 workspace=ws())
    _check(c, ref, tol, f"{kind} {config}")


@pytest.mark.parametrize("kind", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k,first,behind", [([3, 0, 4], 40, 64, 2, 5), ([300, 20], 136, 72, 7, 300), ([0, 0], 8, 8, 3, 0)])
def test_rows_of_no_group_stay(kind, sizes, n, k, first, behind):
    a, b, o = _case(kind, sizes, n, k, 3, first, behind)
    ref, tol = _formula(kind, a, b, o)
    # (what no group has is not read either)
    a[:o[0]], a[o[-1]:] = NAN, INF
    c = torch.full((a.shape[0], n), 7.0, dtype=torch.bfloat16).cuda()
    got = _run(kind, a, b, o, C=c)
    assert got is c
    assert bool((c[:o[0]] == 7).all()) and bool((c[o[-1]:] == 7).all())
    _check(c[o[0]:o[-1]], ref[o[0]:o[-1]], tol[o[0]:o[-1]], kind)


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes", [[3, 5, 2], [130, 200, 70]])
def test_groups_do_not_reach_each_other(kind, sizes):
    """NaN and infinities in one group's rows (and weight) stay in its outputs."""
    a, b, o = _case(kind, sizes, 72, 96, 4)
    ref, tol = _formula(kind, a, b, o)
    a[o[1]:o[2]] = NAN
    a[o[1], 0] = INF
    if kind == "tn":
        b[o[1]:o[2]] = NAN
    else:
        b[1] = NAN
    got = _run(kind, a, b, o)
    if kind == "tn":
        for e in (0, 2):
            _check(got[e], ref[e], tol[e], f"group {e}")
        assert bool(torch.isnan(got[1]).any())
    else:
        for e in (0, 2):
            _check(got[o[e]:o[e + 1]], ref[o[e]:o[e + 1]], tol[o[e]:o[e + 1]], f"group {e}")
        assert bool(torch.isnan(got[o[1]:o[2]]).all())


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes", [[2, 0, 9], [150, 60, 90]])
def test_strided_operands(kind, sizes):
    """Rows inside wider ones, at an odd offset, and a strided output."""
    a, b, o = _case(kind, sizes, 72, 88, 5)
    ref, tol = _formula(kind, a, b, o)
    for pad, at in ((8, 8), (5, 3)):
        wide = torch.full((a.shape[0], a.shape[1] + pad + at), NAN, dtype=torch.bfloat16).cuda()
        wide[:, at:at + a.shape[1]] = a.cuda()
        wb = torch.full(tuple(b.shape[:-1]) + (b.shape[-1] + pad + at,), NAN, dtype=torch.bfloat16).cuda()
        wb[..., at:at + b.shape[-1]] = b.cuda()
        shape = tuple(ref.shape[:-1]) + (ref.shape[-1] + pad + at,)
        c = torch.full(shape, 5.0, dtype=torch.float32).cuda()
        out = c[..., at:at + ref.shape[-1]]
        got = getattr(g5, ENTRY[kind])(wide[:, at:at + a.shape[1]], wb[..., at:at + b.shape[-1]],
                                       torch.tensor(o, dtype=torch.int32).cuda(), C=out, workspace=ws())
        _check(got, ref, tol, f"{kind} {pad}")
        assert bool((c[..., :at] == 5).all()) and bool((c[..., at + ref.shape[-1]:] == 5).all())


@pytest.mark.parametrize("kind", ["nt", "nn"])
def test_one_weight_for_every_group(kind):
    for sizes in ([2, 3, 1], [130, 90, 200]):
        a, b, o = _case(kind, sizes, 64, 96, 6)
        one = b[:1].expand(b.shape)
        _check(getattr(g5, ENTRY[kind])(a.cuda(), b[:1].cuda().expand(b.shape), torch.tensor(o, dtype=torch.int32).cuda(),
                                        workspace=ws()), *_formula(kind, a, one, o), kind)


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("o", [[0, 50, 20, 60], [-5, 10, 10, 9999], [70, 10, 20, 30], [0, 0, 2 ** 31 - 1, -2 ** 31], [60, 60, 60, 60]])
@pytest.mark.parametrize("rows", [60, 700])
def test_offsets_out_of_order_or_range(kind, o, rows):
    """Held to the rows there are; one lower than an earlier one counts as that."""
    held, top = [], 0
    for v in o:
        top = max(top, min(max(v, 0), rows))
        held.append(top)
    g = torch.Generator().manual_seed(8)
    a = _bf((rows, 40 if kind == "tn" else 64), g)
    b = _bf((rows, 64), g) if kind == "tn" else _bf((3, 40, 64) if kind == "nt" else (3, 64, 40), g, 0.125)
    kw = {} if kind == "tn" else {"C": torch.zeros((rows, 40), dtype=torch.bfloat16).cuda()}
    _check(_run(kind, a, b, o, **kw), *_formula(kind, a, b, held), f"{kind} {o}")


def test_empty_calls():
    e = torch.zeros((1,), dtype=torch.int32).cuda()
    a, w = torch.zeros((4, 16), dtype=torch.bfloat16).cuda(), torch.zeros((0, 8, 16), dtype=torch.bfloat16).cuda()
    c = torch.full((4, 8), 3.0, dtype=torch.bfloat16).cuda()
    assert bool((g5.gemm_bf16_grouped_nt(a, w, e, C=c) == 3).all())
    o = torch.tensor([0, 0, 0], dtype=torch.int32).cuda()
    w = torch.zeros((2, 8, 16), dtype=torch.bfloat16).cuda()
    assert g5.gemm_bf16_grouped_nt(a[:0], w, o).shape == (0, 8)
    c = torch.full((2, 16, 8), 3.0).cuda()
    assert bool((g5.gemm_bf16_grouped_tn(a[:0], torch.zeros((0, 8), dtype=torch.bfloat16).cuda(), o, C=c) == 0).all())
    # no summed elements: zeros in the groups' rows alone
    o = torch.tensor([1, 1, 3], dtype=torch.int32).cuda()
    c = torch.full((4, 8), 3.0).cuda()
    g5.gemm_bf16_grouped_nt(a[:, :0], w[:, :, :0], o, C=c)
    assert c[:, 0].tolist() == [3, 0, 0, 3]


@pytest.mark.parametrize("sizes,n,k", [([4, 2, 0, 1], 64, 96), ([200, 70, 300], 256, 160),
                                       ([2000, 0, 3100], 40, 72), ([1500, 2600], 43, 71)])
def test_captured_with_changing_groups(sizes, n, k):
    """A graph reads the offsets when it runs: replays with other groups, the
    program's own eager calls on the same workspace between them."""
    a, b, o = _case("nt", sizes, n, k, 9)
    ad, bd, od = a.cuda(), b.cuda(), torch.tensor(o, dtype=torch.int32).cuda()
    dy = _bf((a.shape[0], n), torch.Generator().manual_seed(10)).cuda()
    space = g5.Workspace()

    def step():
        c = g5.gemm_bf16_grouped_nt(ad, bd, od, C=torch.zeros((a.shape[0], n), dtype=torch.bfloat16, device="cuda"), workspace=space)
        dx = g5.gemm_bf16_grouped(dy, bd, od, C=torch.zeros((a.shape[0], k), dtype=torch.bfloat16, device="cuda"), workspace=space)
        return c, dx, g5.gemm_bf16_grouped_tn(dy, ad, od, workspace=space)

    step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    rng = random.Random(11)
    for turn in range(4):
        cuts = sorted(rng.randint(0, a.shape[0]) for _ in range(len(sizes) - 1))
        od.copy_(torch.tensor([0] + cuts + [a.shape[0]], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, step()):
            assert torch.equal(got, want), f"replay {turn}"
        _check(out[0], *_formula("nt", a, b, od.tolist()), f"replay {turn}")


def test_two_streams():
    a, b, o = _case("nt", [200, 30, 90], 136, 100, 12)
    ref, tol = _formula("nt", a, b, o)
    ad, bd, od = a.cuda(), b.cuda(), torch.tensor(o, dtype=torch.int32).cuda()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            w = g5.Workspace()
            outs.append([g5.gemm_bf16_grouped_nt(ad, bd, od, workspace=w) for _ in range(3)])
    torch.cuda.synchronize()
    for c in outs[0] + outs[1]:
        _check(c, ref, tol, "stream")


def test_gradients_are_the_projection_s():
    """sum(dY . C) against differences along a direction, through the entry points."""
    sizes, n, k = [5, 0, 40, 90], 48, 64
    a, w, o = _case("nt", sizes, n, k, 13)
    g = torch.Generator().manual_seed(14)
    dy, da, dw = _bf((a.shape[0], n), g), _bf(a.shape, g), _bf(w.shape, g)
    dx = _run("nn", dy, w, o, out_dtype=torch.float32).cpu().double()
    gw = _run("tn", dy, a, o).cpu().double()
    # the product is linear in each operand: a step in one is exact up to the sums' bounds
    for step, along, grad in ((da, (da, w), dx), (dw, (a, dw), gw)):
        c, tol = _formula("nt", *along, o)
        want, slack = (c * dy.double()).sum(), (tol * dy.double().abs()).sum()
        got = (grad * step.double()).sum()
        bound = 2 * slack + 1e-5 * (grad.abs() * step.double().abs()).sum()
        assert abs(got - want) <= bound, (float(got), float(want), float(bound))


@pytest.mark.parametrize("rows", [1, 31, 63, 65, 100, 128])
def test_rows_past_a_group_are_zeros(rows):
    """A weight gradient whose last stage is partial, behind one that leaves
    NaN and infinities in its place, rows of NaN behind the group."""
    n = k = 256
    a, b, o = _case("tn", [rows] * 300, n, k, 15)
    ref, tol = _formula("tn", a[:3 * rows], b[:3 * rows], o[:4])
    bad = torch.full((rows * 300, n), NAN, dtype=torch.bfloat16).cuda()
    ad, bd = a.cuda(), b.cuda()
    ad[3 * rows:], bd[3 * rows:] = NAN, INF
    for _ in range(2):
        _run("tn", bad, bad, o)
        got = _run("tn", ad, bd, o)
        _check(got[:3], ref, tol, f"{rows} rows")
