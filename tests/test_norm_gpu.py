"""GPU parity of the RMS norm and its gradient (gemm_rms_norm,
gemm_rms_norm_backward) against the formulas in 64 bits.

Bounds, each from the roundings the kernels take:
  * h = bf16(x + r): one FP32 addition (2^-24 relative) and one rounding to
    bf16 (half a step, 2^-8 relative).
  * y: rounded to bf16 once (2^-8); before that FP32: a sum of squares whose
    longest chain of additions is below 128 terms (each 2^-24; rstd takes
    half of its relative error), the root, the quotient and two products
    -- together below 2^-17 relative.
  * codes: equal to those of gemm_fp8_quantize_rows on the bf16 rows, and
    half a step of E4M3 (2^-4 relative, 2^-10 below the normal range) from
    the quotient.
  * dX: 2^-8 of the result; FP32 products 2^-21 of each term; the row's sum
    (chains below 128 additions) 2^-17 of the sum of magnitudes.
  * dW: chains of rows/512 additions in a workgroup and at most 128 + 3 in
    the join, 3 roundings per product: (rows/512 + 140) 2^-24 of the sum of
    magnitudes.
"""
import pytest
import torch

import dense_gemm_05_amd as g5

pytestmark = pytest.mark.gpu

TINY = 1e-37          # below every bf16 normal: results that underflow


def _say(msg):
    print(f"[norm] {msg}", flush=True)


def _gen(*key):
    return torch.Generator().manual_seed(hash(key) % (1 << 31))


def _layout(rows, cols, kind, dtype=torch.bfloat16):
    """contig; padded (aligned rows, larger stride); odd (element offset 1,
    stride cols + 3)."""
    if kind == "contig":
        return torch.zeros((rows, cols), dtype=dtype, device="cuda")
    if kind == "padded":
        ld = (cols + 15) // 16 * 16 + 16
        return torch.zeros((rows, ld), dtype=dtype, device="cuda")[:, :cols]
    ld = cols + 3
    return torch.zeros((rows * ld + 1,), dtype=dtype, device="cuda")[1:].view(rows, ld)[:, :cols]


def _put(t, kind):
    d = _layout(t.shape[0], t.shape[1], kind, t.dtype)
    d.copy_(t)
    return d


def _bf(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def _check(got, ref, tol, what):
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} out of bound, worst {float((err / tol).max())}"


SHAPES = [(1, 1, "contig"), (3, 7, "contig"), (5, 64, "contig"), (9, 512, "contig"), (6, 513, "odd"),
          (300, 520, "padded"), (2, 2048, "contig"), (4, 2056, "odd"), (1, 4096, "contig"), (33, 4100, "contig"),
          (3, 4096, "padded"), (2, 8192, "contig"), (2, 8200, "contig"), (3, 12280, "padded"), (2, 16384, "contig"),
          (2, 16392, "contig"), (3, 20001, "odd")]


@pytest.mark.parametrize("rows,cols,kind", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_codes(rows, cols, kind, residual):
    _say(f"norm {rows}x{cols} {kind} residual={residual}")
    g = _gen(1, rows, cols, residual)
    x, r, w = _bf((rows, cols), g), _bf((rows, cols), g, 3.0), _bf((cols,), g)
    dx, dr, dw = _put(x, kind), (_put(r, kind) if residual else None), w.cuda()
    rstd = torch.zeros((rows,), device="cuda")
    out = g5.rms_norm(dx, dw, residual=dr, eps=1e-5, Y=_layout(rows, cols, kind),
                      H=_layout(rows, cols, kind) if residual else None, rstd=rstd)
    h = x
    if residual:
        out, h = out
        h = h.cpu()
        s = x.double() + r.double()
        _check(h.double(), s, (2.0 ** -8 + 2.0 ** -23) * s.abs() + TINY, "h")
    hd = h.double()
    ref_rstd = 1.0 / torch.sqrt((hd * hd).mean(1) + float(torch.tensor(1e-5)))
    ref = hd * ref_rstd[:, None] * w.double()
    y = out.cpu()
    _check(rstd.cpu().double(), ref_rstd, 2.0 ** -17 * ref_rstd, "rstd")
    _check(y.double(), ref, (2.0 ** -8 + 2.0 ** -16) * ref.abs() + TINY, "y")

    q = g5.rms_norm_e4m3(dx, dw, residual=dr, eps=1e-5, Q=_layout(rows, cols, kind, torch.uint8))
    wq, wscale = g5.gemm_fp8_quantize_rows(out)
    assert torch.equal(q[0].cpu(), wq.cpu()) and torch.equal(q[1].cpu(), wscale.cpu())
    if residual:
        assert torch.equal(q[2].cpu(), h)
    amax = y.double().abs().amax(1, keepdim=True)
    quot = torch.where(amax > 0, y.double() * 448.0 / amax, y.double() * 0)
    codes = q[0].cpu().view(torch.float8_e4m3fn).double()
    _check(codes, quot, 2.0 ** -4 * quot.abs() + 2.0 ** -10, "codes")
    _check(q[1].cpu().double(), amax[:, 0] / 448.0, 2.0 ** -23 * amax[:, 0] / 448.0, "factors")


def test_norm_without_weight_and_in_place_sum():
    g = _gen(2)
    x, r = _bf((37, 776), g), _bf((37, 776), g)
    want_y, want_h = g5.rms_norm(x.cuda(), None, residual=r.cuda())
    ones = g5.rms_norm(x.cuda(), torch.ones(776, dtype=torch.bfloat16, device="cuda"), residual=r.cuda())[0]
    assert torch.equal(want_y, ones)
    for inplace in ("x", "r"):
        dx, dr = x.cuda(), r.cuda()
        y, h = g5.rms_norm(dx, None, residual=dr, H=dx if inplace == "x" else dr)
        assert torch.equal(y, want_y) and torch.equal(h, want_h)
        assert h.data_ptr() == (dx if inplace == "x" else dr).data_ptr()
    # rows past the held ones, in place too
    x, r = _bf((2, 16400), g), _bf((2, 16400), g)
    want_y, want_h = g5.rms_norm(x.cuda(), None, residual=r.cuda())
    dr = r.cuda()
    y, h = g5.rms_norm(x.cuda(), None, residual=dr, H=dr)
    assert torch.equal(y, want_y) and torch.equal(h, want_h)


def test_norm_special_rows():
    """A row of zeros, an infinity and a NaN stay in their rows; what stands
    between the rows of a padded tensor is left as it was."""
    g = _gen(3)
    x = _bf((6, 1000), g)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    buf = torch.full((6, 1024), 7.0, dtype=torch.bfloat16, device="cuda")
    y = g5.rms_norm(x.cuda(), None, Y=buf[:, :1000], eps=1e-6).cpu()
    clean = _bf((6, 1000), _gen(3))
    want = g5.rms_norm(clean.cuda(), None, eps=1e-6).cpu()
    for i in (0, 4, 5):
        assert torch.equal(y[i], want[i])
    assert (y[1] == 0).all() and y[3].isnan().all()
    assert y[2, 5].isnan() and (y[2, :5] == 0).all()
    assert (buf[:, 1000:] == 7.0).all()
    q, s = g5.rms_norm_e4m3(x.cuda(), None, eps=1e-6)
    assert (q[1].cpu() & 0x7f == 0).all() and float(s[1]) == 0.0
    assert g5.rms_norm(x.cuda(), None, eps=0.0)[1].isnan().all()     # 0 / 0, as the formula


def _grad_ref(dy, h, w, rstd, dh):
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    xh, g = h * rstd, dy * w
    mean, mag = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - xh * mean) + dh.double()
    tol = (2.0 ** -8 * dx.abs() + 2.0 ** -21 * (rstd * g.abs() + rstd * xh.abs() * mag + dh.double().abs())
           + 2.0 ** -17 * rstd * xh.abs() * mag + TINY)
    p = dy * xh
    return dx, tol, p.sum(0), (h.shape[0] / 512 + 140) * 2.0 ** -24 * p.abs().sum(0) + TINY


GRAD_SHAPES = [(1, 1, "contig"), (3, 7, "contig"), (1, 4096, "contig"), (700, 264, "padded"), (1025, 513, "odd"),
               (6, 2048, "contig"), (5, 4100, "contig"), (9, 8192, "contig"), (4, 8200, "odd"), (3, 16384, "contig"),
               (1030, 16392, "contig"), (3, 20001, "odd")]


@pytest.mark.parametrize("rows,cols,kind", GRAD_SHAPES)
@pytest.mark.parametrize("branch", [False, True])
def test_norm_gradient(rows, cols, kind, branch):
    _say(f"gradient {rows}x{cols} {kind} branch={branch}")
    g = _gen(4, rows, cols, branch)
    dy, h, w, dh = _bf((rows, cols), g), _bf((rows, cols), g, 2.0), _bf((cols,), g), _bf((rows, cols), g)
    if not branch:
        dh.zero_()
    rstd = torch.zeros((rows,), device="cuda")
    g5.rms_norm(_put(h, kind), w.cuda(), rstd=rstd)
    ws = g5.Workspace()
    dx, dw = g5.rms_norm_backward(_put(dy, kind), _put(h, kind), w.cuda(), rstd, dH=_put(dh, kind) if branch else None,
                                  dX=_layout(rows, cols, kind), workspace=ws)
    ref, tol, wref, wtol = _grad_ref(dy, h, w, rstd.cpu(), dh)
    _check(dx.cpu().double(), ref, tol, "dX")
    _check(dw.cpu().double(), wref, wtol, "dW")
    # the counters other calls expect at zero, the same bits again, no dW
    assert not ws.buf[:g5.GEMM_WORKSPACE_COUNTER_BYTES].any()
    ws.buf[g5.GEMM_WORKSPACE_COUNTER_BYTES:] = 255
    again = g5.rms_norm_backward(_put(dy, kind), _put(h, kind), w.cuda(), rstd, dH=_put(dh, kind) if branch else None,
                                 workspace=ws)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only = g5.rms_norm_backward(_put(dy, kind), _put(h, kind), w.cuda(), rstd, dH=_put(dh, kind) if branch else None,
                                need_dw=False)
    assert torch.equal(only[0], dx) and only[1] is None


def test_norm_gradient_against_differences():
    """<dX, v> and <dW, u> against central differences of the forward formula
    in 64 bits: f(h, w) = sum dy y(h, w).  The differences' own error (t^2
    times a third derivative, t = 1e-4) is below 1e-6 of the bound."""
    g = _gen(5)
    rows, cols, eps, t = 7, 300, 1e-5, 1e-4
    dy, h, w = _bf((rows, cols), g), _bf((rows, cols), g), _bf((cols,), g)
    rstd = torch.zeros((rows,), device="cuda")
    g5.rms_norm(h.cuda(), w.cuda(), eps=eps, rstd=rstd)
    dx, dw = g5.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd)
    _, tol, _, wtol = _grad_ref(dy, h, w, rstd.cpu(), torch.zeros_like(h))

    def f(hh, ww):
        return float((dy.double() * hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps) * ww).sum())

    for k in range(4):
        v, u = torch.randn((rows, cols), generator=g).double(), torch.randn((cols,), generator=g).double()
        num = (f(h.double() + t * v, w.double()) - f(h.double() - t * v, w.double())) / (2 * t)
        # (the kernel's rstd is within 2^-17 of the formula's)
        slack = float((tol * v.abs()).sum()) + 2.0 ** -15 * float((dx.cpu().double() * v).abs().sum())
        assert abs(num - float((dx.cpu().double() * v).sum())) <= slack
        num = (f(h.double(), w.double() + t * u) - f(h.double(), w.double() - t * u)) / (2 * t)
        slack = float((wtol * u.abs()).sum()) + 2.0 ** -15 * float((dw.cpu().double() * u).abs().sum())
        assert abs(num - float((dw.cpu().double() * u).sum())) <= slack


def test_norm_empty():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert g5.rms_norm(e).shape == (0, 64)
    q, s = g5.rms_norm_e4m3(e)
    assert q.shape == (0, 64) and s.shape == (0,)
    dx, dw = g5.rms_norm_backward(e, e, None, torch.empty((0,), device="cuda"),
                                  dW=torch.full((64,), 5.0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()
    assert g5.rms_norm(torch.empty((4, 0), dtype=torch.bfloat16, device="cuda")).shape == (4, 0)


def test_norm_on_a_stream_and_in_a_graph():
    """Another stream, and a captured forward and backward replayed with new
    inputs between eager work."""
    g = _gen(6)
    rows, cols = 130, 4096
    x, r, w, dy = (_bf(s, g).cuda() for s in ((rows, cols), (rows, cols), (cols,), (rows, cols)))
    rstd, ws = torch.empty((rows,), device="cuda"), g5.Workspace()

    def step():
        y, h = g5.rms_norm(x, w, residual=r, rstd=rstd)
        return (y, h) + g5.rms_norm_backward(dy, h, w, rstd, workspace=ws)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        for t in (x, r, dy):
            t.copy_(_bf((rows, cols), g).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), f"replay {k}"


@pytest.mark.parametrize("cols", [64, 100, 4100, 16400])
def test_norm_weights_far_from_the_rows_scale(cols):
    """Rows and weights whose product leaves FP32's range, or falls among its
    subnormal numbers, while y does not: bf16(h rstd w) all the same."""
    g = _gen(7, cols)
    for hs, ws, eps in ((1e15, 1e25, 1e-6), (1e-16, 1e-28, 0.0)):
        h, w = (_bf((3, cols), g).double() * hs).bfloat16(), (_bf((cols,), g).double() * ws).bfloat16()
        hd = h.double()
        ref = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps) * w.double()
        assert torch.isfinite(ref.bfloat16()).all()
        y = g5.rms_norm(h.cuda(), w.cuda(), eps=eps).cpu()
        # (half a step, the sums and products in FP32; 2^-100: far below any y but the smallest)
        _check(y.double(), ref, (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -100 * ws, "y")
        q, s = g5.rms_norm_e4m3(h.cuda(), w.cuda(), eps=eps)
        wq, wscale = g5.gemm_fp8_quantize_rows(y.cuda())
        assert torch.equal(q, wq) and torch.equal(s, wscale)


@pytest.mark.parametrize("cols", [20, 24, 4100])
def test_norm_gradient_with_an_infinite_weight(cols):
    """dX is infinite or NaN where the formula's is, also when the weight
    stands among the last columns of a row that is no multiple of 8 long."""
    g = _gen(8, cols)
    for at in (3, cols - 7, cols - 1):
        dy, h, w = (_bf(s, g) for s in ((4, cols), (4, cols), (cols,)))
        w[at], dy[1, at], dy[2] = torch.inf, 0.0, dy[2].abs()
        rstd = torch.ones((4,))
        xh, gg = h.double(), dy.double() * w.double()
        ref = gg - xh * (gg * xh).sum(1, keepdim=True) / cols
        dx, _ = g5.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
        dx = dx.cpu().double()
        assert torch.equal(dx.isnan(), ref.isnan()) and torch.equal(dx.isposinf(), ref.isposinf())
        assert torch.equal(dx.isneginf(), ref.isneginf())


@pytest.mark.parametrize("cols", [9, 513, 1001, 4100, 8199, 12283])
def test_norm_ragged_rows_without_a_residual(cols):
    """The same bits as with a residual of zeros, whose sum is X, and nothing
    stored beside the rows."""
    g = _gen(9, cols)
    x, w = _bf((5, cols), g).cuda(), _bf((cols,), g).cuda()
    want, h = g5.rms_norm(x, w, residual=torch.zeros_like(x))
    assert torch.equal(h, x)
    buf = torch.full((7, cols + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(g5.rms_norm(x, w, Y=buf[1:6, 1:cols + 1]), want)
    buf[1:6, 1:cols + 1] = 5.0
    assert (buf == 5.0).all()
    codes = torch.full((7, cols + 3), 9, dtype=torch.uint8, device="cuda")
    q, s = g5.rms_norm_e4m3(x, w, Q=codes[1:6, 1:cols + 1])
    wq, wscale = g5.gemm_fp8_quantize_rows(want)
    assert torch.equal(q, wq) and torch.equal(s, wscale)
    codes[1:6, 1:cols + 1] = 9
    assert (codes == 9).all()


def test_norm_gradient_of_very_long_rows():
    """More columns than one launch of dW's join can have threads for: dW of
    one row, and the empty sum of none.  Every product is exact (dy one of
    +-1, h a power of two, w and rstd 1), so dW is exact and dX is 2^-8 off at
    most but for the row's mean: cols / 256 additions in a thread and 10 in the
    join, of terms of at most 2."""
    cols = (1 << 26) + 40
    _say(f"gradient 1x{cols}")
    g = torch.Generator(device="cuda").manual_seed(10)
    dy = torch.randint(0, 2, (1, cols), generator=g, device="cuda").mul_(2).sub_(1).bfloat16()
    h = torch.randint(0, 2, (1, cols), generator=g, device="cuda").add_(1).bfloat16()
    rstd, ws = torch.ones((1,), device="cuda"), g5.Workspace()
    dx, dw = g5.rms_norm_backward(dy, h, None, rstd, workspace=ws)
    p = dy.double() * h.double()
    assert torch.equal(dw.double(), p[0])
    c, off = float(p.mean()), (cols / 256 + 10) * 2.0 ** -24 * float(p.abs().mean())
    ref = dy.double() - h.double() * c
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * h.double() * off).all()
    dw.fill_(3.0)
    g5.rms_norm_backward(dy[:0], h[:0], None, rstd[:0], dW=dw, workspace=ws)
    assert not dw.any()
