"""GPU parity of the projection with low-rank adapters (gemm_bf16_nt_lora)
against the formula in 64 bits.

The bound, from the roundings the kernels take.  Products of bf16 values are
exact in FP32 and a sum of n of them is within n 2^-24 of the sum of their
magnitudes in any order:
  ev = K 2^-24 scale sum|x a| + 2^-22 |v|          (v, its slices, the scale)
  e  = K 2^-24 sum|x w| + sum_r (ev + 2^-16 |v|) |b|  (v as two bf16 parts)
       + (2 R + 4) 2^-24 sum_r |v b| + 2^-23 (|x w^T| + |v b^T|)   (joined)
and the output's own rounding, 2^-8 |c| for bf16.
"""
import pytest
import torch

import dense_gemm_05_amd as g5

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[lora] {msg}", flush=True)


def _gen(*key):
    return torch.Generator().manual_seed(hash(key) % (1 << 31))


def _strided(t, kind):
    """contig; padded (16-byte aligned rows, a larger stride); odd (element
    offset 1, stride cols + 3)."""
    if kind == "contig":
        return t.cuda()
    *lead, cols = t.shape
    n = 1
    for d in lead:
        n *= d
    ld = (cols + 15) // 16 * 16 + 16 if kind == "padded" else cols + 3
    off = 0 if kind == "padded" else 1
    v = torch.full((n * ld + off,), float("nan"), dtype=t.dtype, device="cuda")[off:].view(*lead, ld)[..., :cols]
    v.copy_(t)
    return v


def _inputs(g, M, N, K, L, R):
    x = torch.randn((M, K), generator=g).bfloat16()
    w = (torch.randn((N, K), generator=g) * K ** -0.5).bfloat16()
    a = (torch.randn((L, R, K), generator=g) * K ** -0.5).bfloat16()
    b = torch.randn((L, N, R), generator=g).bfloat16()
    scale = torch.rand((L,), generator=g) + 0.5
    idx = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    return x, w, a, b, scale, idx


def _formula(x, w, a, b, scale, idx):
    x, w = x.double(), w.double()
    K, R = x.shape[1], a.shape[1]
    base = x @ w.t()
    y, tol = base.clone(), K * 2.0 ** -24 * (x.abs() @ w.abs().t()) + 2.0 ** -23 * base.abs()
    for m in range(x.shape[0]):
        i = int(idx[m])
        if not 0 <= i < a.shape[0]:
            continue
        s = 1.0 if scale is None else float(scale[i])
        ai, bi = a[i].double(), b[i].double()
        v = s * (ai @ x[m])
        ev = K * 2.0 ** -24 * s * (ai.abs() @ x[m].abs()) + 2.0 ** -22 * v.abs()
        d, mag = bi @ v, bi.abs() @ v.abs()
        y[m] += d
        tol[m] += bi.abs() @ (ev + 2.0 ** -16 * v.abs()) + (2 * R + 4) * 2.0 ** -24 * mag + 2.0 ** -23 * d.abs()
    return y, 1.01 * tol


def _check(got, ref, tol, what):
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} out of bound, worst {float((err / tol).max())}"


CASES = [  # M, N, K, L, R, layout
    (1, 64, 64, 1, 8, "contig"), (1, 200, 1100, 3, 16, "contig"), (16, 100, 4096, 64, 16, "contig"),
    (7, 50, 520, 5, 4, "padded"), (16, 256, 2048, 2, 64, "contig"), (3, 33, 31, 2, 1, "odd"),
    (5, 48, 100, 4, 7, "odd"), (1, 1, 1, 1, 1, "contig"), (12, 1000, 8, 3, 130, "contig"),
    (17, 128, 128, 3, 16, "contig"), (100, 200, 260, 7, 12, "contig"), (77, 264, 516, 16, 24, "contig"),
    (130, 90, 100, 5, 9, "odd"), (256, 384, 512, 4, 16, "contig"), (300, 512, 96, 300, 40, "padded"),
    (512, 1024, 256, 2, 64, "contig"), (40, 40, 2048, 3, 33, "padded"), (1024, 256, 64, 1, 8, "contig"),
]


@pytest.mark.parametrize("M,N,K,L,R,kind", CASES)
def test_lora(M, N, K, L, R, kind):
    _say(f"M={M} N={N} K={K} adapters={L} rank={R} {kind}")
    x, w, a, b, scale, idx = _inputs(_gen(1, M, N, K, L, R), M, N, K, L, R)
    dev = [_strided(t, kind) for t in (x, w, a, b)]
    ws = g5.Workspace()
    for order in ("mixed", "runs", "none"):
        i = {"mixed": idx, "runs": idx.sort().values, "none": torch.full_like(idx, -1)}[order]
        if order == "mixed" and M > 3:
            i = i.clone()
            i[1], i[2] = L, -(1 << 31)          # outside: no adapter
        y, tol = _formula(x, w, a, b, scale, i)
        got = g5.gemm_bf16_nt_lora(*dev, i.cuda(), scale=scale.cuda(), out_dtype=torch.float32, workspace=ws)
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), order)
        assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
        ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
        out = torch.full((M, N + 40), 3.0, dtype=torch.bfloat16, device="cuda")
        b16 = g5.gemm_bf16_nt_lora(*dev, i.cuda(), scale=scale.cuda(), C=out[:, :N], workspace=ws)
        assert torch.equal(b16, got.bfloat16()) and (out[:, N:] == 3.0).all()
        again = g5.gemm_bf16_nt_lora(*dev, i.cuda(), scale=scale.cuda(), out_dtype=torch.float32, workspace=ws)
        assert torch.equal(again, got)
        if M <= 16:      # a row's result does not depend on the others
            one = g5.gemm_bf16_nt_lora(dev[0][M - 1:], *dev[1:], i[M - 1:].cuda(), scale=scale.cuda(),
                                       out_dtype=torch.float32, workspace=ws)
            assert torch.equal(one[0], got[M - 1])


@pytest.mark.parametrize("config", ["bf16_256x192", "bf16_256x256", "bf16_128x128"])
@pytest.mark.parametrize("M,N,K", [(512, 768, 128), (300, 200, 136)])
def test_lora_tiles(monkeypatch, config, M, N, K):
    """Every tile shape, whole and masked."""
    monkeypatch.setenv("GEMM_FORCE_CONFIG", config)
    x, w, a, b, scale, idx = _inputs(_gen(2, M, N, K), M, N, K, 6, 16)
    y, tol = _formula(x, w, a, b, None, idx)
    got = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), a.cuda(), b.cuda(), idx.cuda(), out_dtype=torch.float32)
    _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), config)


@pytest.mark.parametrize("split", ["1", "4"])
def test_lora_with_k_split(monkeypatch, split):
    monkeypatch.setenv("GEMM_FORCE_CONFIG", "bf16_128x128")
    monkeypatch.setenv("GEMM_FORCE_KSPLIT", split)
    for M, N, K in ((128, 256, 1024), (50, 200, 1032)):
        x, w, a, b, scale, idx = _inputs(_gen(3, M, N, K), M, N, K, 3, 24)
        y, tol = _formula(x, w, a, b, scale, idx)
        ws = g5.Workspace()
        got = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), a.cuda(), b.cuda(), idx.cuda(), scale=scale.cuda(),
                                   out_dtype=torch.float32, workspace=ws)
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), f"split {split}")
        assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()


@pytest.mark.parametrize("M,N,K,L,R,order", [
    (17, 64, 4096, 3, 16, "mixed"), (32, 70, 1030, 2, 40, "one"), (48, 130, 515, 5, 7, "runs"),
    (49, 65, 2048, 4, 24, "one"), (80, 1, 900, 3, 33, "runs"), (81, 200, 1288, 20, 8, "mixed"),
    (128, 96, 3000, 2, 64, "one"), (128, 4200, 130, 9, 4, "mixed"), (65, 33000, 64, 2, 8, "runs")])
def test_lora_streamed_rows(M, N, K, L, R, order):
    """17 .. 128 rows: every row-block count, phases and slices of K with odd
    ends, blocks of one adapter whose last is not full, aligned and not."""
    _say(f"M={M} N={N} K={K} adapters={L} rank={R} {order}")
    x, w, a, b, scale, idx = _inputs(_gen(9, M, N, K), M, N, K, L, R)
    idx = {"mixed": idx, "one": torch.full_like(idx, L - 1), "runs": idx.sort().values}[order]
    y, tol = _formula(x, w, a, b, scale, idx)
    ws, outs = g5.Workspace(), []
    for kind in ("contig", "odd"):
        dev = [_strided(t, kind) for t in (x, w, a, b)]
        out = torch.full((M + 2, N + 3), 3.0, device="cuda")
        got = g5.gemm_bf16_nt_lora(*dev, idx.cuda(), scale=scale.cuda(), C=out[:M, :N], workspace=ws)
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), kind)
        assert (out[M:] == 3.0).all() and (out[:, N:] == 3.0).all()
        assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
        ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
        outs.append(got)
        b16 = g5.gemm_bf16_nt_lora(*dev, idx.cuda(), scale=scale.cuda(), workspace=ws)
        assert torch.equal(b16, got.bfloat16())
    assert torch.equal(outs[0], outs[1])      # the alignment does not change the sums


@pytest.mark.parametrize("M", [9, 70, 150])
def test_lora_values_stay_in_their_rows(M):
    """NaN and infinities of other rows and other adapters reach no row."""
    N, K, L, R = 96, 264, 4, 16
    x, w, a, b, scale, idx = _inputs(_gen(4, M), M, N, K, L, R)
    idx[:] = torch.arange(M) % (L + 1) - 1
    clean = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), a.cuda(), b.cuda(), idx.cuda(), scale=scale.cuda())
    x2, a2, b2, s2 = x.clone(), a.clone(), b.clone(), scale.clone()
    a2[1, 3, 7], b2[2], s2[1] = torch.nan, torch.inf, torch.nan
    x2[5, 3] = torch.inf
    got = g5.gemm_bf16_nt_lora(x2.cuda(), w.cuda(), a2.cuda(), b2.cuda(), idx.cuda(), scale=s2.cuda())
    for m in range(M):
        if m == 5 or int(idx[m]) in (1, 2):
            assert not torch.isfinite(got[m].float()).all()
        else:
            assert torch.equal(got[m], clean[m]), m


@pytest.mark.parametrize("kind", ["contig", "odd"])
@pytest.mark.parametrize("order", ["one", "halves"])
def test_lora_rows_of_sixteen_stand_alone(kind, order):
    """Sixteen rows, all of one adapter or eight of two, each as if called
    alone, at any alignment."""
    M, N, K, L, R = 16, 70, 1100, 2, 20
    x, w, a, b, scale, idx = _inputs(_gen(8), M, N, K, L, R)
    idx = torch.zeros_like(idx) if order == "one" else torch.arange(M, dtype=torch.int32) // 8
    dev = [_strided(t, kind) for t in (x, w, a, b)]
    y, tol = _formula(x, w, a, b, scale, idx)
    got = g5.gemm_bf16_nt_lora(*dev, idx.cuda(), scale=scale.cuda(), out_dtype=torch.float32)
    _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), order)
    for m in (0, 7, 8, 15):
        one = g5.gemm_bf16_nt_lora(dev[0][m:m + 1], *dev[1:], idx[m:m + 1].cuda(), scale=scale.cuda(),
                                   out_dtype=torch.float32)
        assert torch.equal(one[0], got[m]), m


def test_lora_without_adapters_is_the_product():
    x, w, a, b, scale, idx = _inputs(_gen(5), 40, 96, 264, 2, 8)
    want = g5.gemm_bf16_nt(x.cuda(), w.cuda(), workspace=g5.Workspace())
    for L, R in ((0, 8), (2, 0)):
        got = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), a[:L, :R].cuda(), b[:L, :, :R].cuda(), idx.cuda())
        y = x.double() @ w.double().t()
        assert ((got.cpu().double() - y).abs() <= 2.0 ** -8 * y.abs() + 264 * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t())).all()
        assert torch.equal(got, want)
    e = torch.empty((0, 264), dtype=torch.bfloat16, device="cuda")
    assert g5.gemm_bf16_nt_lora(e, w.cuda(), a.cuda(), b.cuda(), idx[:0].cuda()).shape == (0, 96)
    z = g5.gemm_bf16_nt_lora(x[:, :0].cuda(), w[:, :0].cuda(), a[:, :, :0].cuda(), b.cuda(), idx.cuda(),
                             C=torch.ones((40, 96), dtype=torch.bfloat16, device="cuda"))
    assert not z.any()


def test_lora_shared_halves_and_strides():
    """An expanded A (one first half for every adapter) and a permuted idx
    give what separate copies give."""
    M, N, K, L, R = 20, 64, 128, 3, 8
    x, w, a, b, scale, idx = _inputs(_gen(6), M, N, K, L, R)
    shared = a[:1].cuda().expand(L, R, K)
    got = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), shared, b.cuda(), idx.cuda())
    want = g5.gemm_bf16_nt_lora(x.cuda(), w.cuda(), shared.contiguous(), b.cuda(), idx.cuda())
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [5, 150])
def test_lora_on_a_stream_and_in_a_graph(M):
    N, K, L, R = 512, 1024, 6, 16
    g = _gen(7, M)
    x, w, a, b, scale, idx = (t.cuda() for t in _inputs(g, M, N, K, L, R))
    eager, held = g5.Workspace(), g5.Workspace()
    call = lambda ws: g5.gemm_bf16_nt_lora(x, w, a, b, idx, scale=scale, workspace=ws)   # noqa: E731
    want, side = call(eager), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(held)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(held)
    for r in range(4):
        x.copy_(torch.randn((M, K), generator=g).bfloat16())
        idx.copy_(torch.randint(-1, L, (M,), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.clone(), call(eager)), f"replay {r}"


@pytest.mark.parametrize("M,N,K,L,R,order", [
    (64, 12288, 1100, 3, 12, "mixed"), (80, 9000, 900, 2, 20, "one"), (128, 6144, 1300, 5, 8, "runs"),
    (17, 16400, 1100, 2, 30, "mixed")])
def test_lora_streamed_wide(M, N, K, L, R, order):
    """17 .. 128 rows and so many columns that one or two slices of K have
    several phases each; the next call on the same workspace, unaligned, too."""
    _say(f"wide M={M} N={N} K={K} adapters={L} rank={R} {order}")
    x, w, a, b, scale, idx = _inputs(_gen(10, M, N, K), M, N, K, L, R)
    idx = {"mixed": idx, "one": torch.full_like(idx, L - 1), "runs": idx.sort().values}[order]
    y, tol = _formula(x, w, a, b, scale, idx)
    ws, outs = g5.Workspace(), []
    for kind in ("contig", "odd"):
        dev = [_strided(t, kind) for t in (x, w, a, b)]
        out = torch.full((M + 2, N + 3), 3.0, device="cuda")
        got = g5.gemm_bf16_nt_lora(*dev, idx.cuda(), scale=scale.cuda(), C=out[:M, :N], workspace=ws)
        _check(got.cpu().double(), y, tol + 2.0 ** -24 * y.abs(), kind)
        assert (out[M:] == 3.0).all() and (out[:, N:] == 3.0).all()
        assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
        ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
        outs.append(got)
    assert torch.equal(outs[0], outs[1])
