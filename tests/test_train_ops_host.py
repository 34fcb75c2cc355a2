"""Host-only checks of the operators of a training step: arguments refused
before anything is enqueued (no GPU), and the sizes their workspaces need."""
import ctypes

import pytest
import torch

import dense_gemm_05_amd as g5
from dense_gemm_05_amd import train_ops as ops
from test_binding_host import FakeGpuTensor as _Fake


class FakeGpuTensor(_Fake):
    def is_contiguous(self):
        return True


P = 0x7F0000000000     # fake, aligned addresses 16 GiB apart, never dereferenced
A, B, C, O, T, W = (P + (i << 34) for i in range(6))
INV, WS, OK, UNS = g5.GEMM_ERR_INVALID_ARG, g5.GEMM_ERR_WORKSPACE, g5.GEMM_OK, g5.GEMM_ERR_UNSUPPORTED
CR = g5.GEMM_WORKSPACE_COUNTER_BYTES


def grouped(kind, **kw):
    """4 groups, 600 rows (more than are streamed): nt and nn [600, 64] by [4, ., .] to 48 columns; tn
    [600, 48] by [600, 64]."""
    tn = kind == 2
    a = dict(E=4, rows=600, M=48, N=64 if tn else 48, K=64, O=O, A=A, lda=48 if tn else 64, B=B,
             ldb=64 if kind in (0, 2) else 48, sB=64 * 48, C=C, ldc=64 if tn else 48, sC=48 * 64, t=0, ws=None, n=0)
    a.update(kw)
    L = g5.lib()
    if tn:
        return L.gemm_bf16_grouped_tn(a["E"], a["rows"], a["M"], a["N"], a["O"], a["A"], a["lda"], a["B"], a["ldb"],
                                      a["C"], a["ldc"], a["sC"], a["t"], a["ws"], a["n"], None)
    fn = L.gemm_bf16_grouped if kind else L.gemm_bf16_grouped_nt
    return fn(a["E"], a["rows"], a["N"], a["K"], a["O"], a["A"], a["lda"], a["B"], a["ldb"], a["sB"], a["C"], a["ldc"],
              a["t"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("bad,status", [
    (dict(E=-1), INV), (dict(E=4097), INV), (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(N=-1), INV),
    (dict(N=(1 << 30) + 1), INV), (dict(O=None), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(C=None), INV),
    (dict(O=O + 2), INV), (dict(A=A + 1), INV), (dict(B=B + 1), INV), (dict(C=C + 1), INV), (dict(t=1, C=C + 2), INV),
    (dict(lda=47), INV), (dict(ldb=47), INV), (dict(ldc=47), INV), (dict(t=2), INV), (dict(t=-1), INV),
    (dict(C=A), INV), (dict(C=B), INV), (dict(C=O), INV), (dict(lda=(1 << 21) + 8), UNS), (dict(ldb=(1 << 21) + 8), UNS),
    (dict(lda=65), WS), (dict(A=A + 2), WS), (dict(B=B + 2, ws=W, n=CR), WS), (dict(A=A + 2, ws=W + 128, n=1 << 30), INV),
    (dict(A=A + 2, ws=B, n=1 << 30), INV), (dict(A=A + 2, ws=C, n=1 << 30), INV)])
def test_grouped_refuses(kind, bad, status):
    assert grouped(kind, **bad) == status


def test_grouped_refuses_of_one_kind():
    assert grouped(0, K=-1) == INV and grouped(1, sB=-1) == INV and grouped(2, M=-1) == INV
    assert grouped(2, sC=-1) == INV and grouped(2, sC=47 * 64 + 63) == INV
    assert grouped(1, N=43, ldb=48) == WS and grouped(2, N=61) == WS and grouped(2, M=45) == WS
    assert grouped(0, lda=65) == WS and grouped(0, A=A + 4, K=60) == grouped(0, lda=66)        # (dwords suffice)
    # more workgroups than a launch takes
    assert grouped(2, E=4096, M=1 << 20, N=1 << 20, lda=1 << 20, ldb=1 << 20, ldc=1 << 20, sC=1 << 40) == UNS


def test_grouped_empty_calls_do_nothing():
    for kind in (0, 1, 2):
        assert grouped(kind, E=0, O=None, A=None) == OK and grouped(kind, N=0, C=None) == OK
    assert grouped(0, rows=0, C=None) == OK and grouped(2, M=0, C=None) == OK


def test_grouped_workspace_size():
    n = ctypes.c_uint64(1)

    def size(kind, E=4, rows=600, M=48, N=64, K=64, a=A, lda=64, b=B, ldb=64, sB=4096):
        st = g5.lib().gemm_grouped_workspace_size(kind, E, rows, M, N, K, a, lda, b, ldb, sB, ctypes.byref(n))
        return st, n.value

    assert size(0) == size(1) == size(2) == (OK, 0)
    up = lambda b: -(-b // 256) * 256                                      # noqa: E731
    assert size(0, a=A + 2) == (OK, CR + up(600 * 64 * 2))
    assert size(0, K=61, ldb=61, sB=64 * 61) == (OK, CR + up(4 * 64 * 64 * 2))
    assert size(1, N=61) == (OK, CR + up(4 * 64 * 64 * 2)) and size(1, N=61, sB=0) == (OK, CR + up(64 * 64 * 2))
    assert size(2, M=43, N=61) == (OK, CR + up(600 * 48 * 2) + up(600 * 64 * 2))
    # rows of whole dwords are read where they are
    assert size(0, K=58, lda=58, ldb=58, sB=64 * 58, a=A + 4, b=B + 8) == (OK, 0)
    assert size(1, N=58, b=B + 4) == size(2, M=42, N=62, a=A + 12) == (OK, 0)
    # small weight gradients of many rows: slices' sums, one per 512 rows of a group here
    assert size(2, rows=1 << 13) == (OK, CR + up(4 * 4 * 48 * 64 * 4))
    assert size(2, rows=1 << 13, M=1024, N=1024, lda=1024, ldb=1024) == (OK, 0)
    # the stream takes rows of any alignment
    assert size(0, rows=512, a=A + 2, b=B + 2) == (OK, 0) and size(0, rows=512, lda=1 << 23, ldb=1 << 25) == (OK, 0)
    assert size(3)[0] == INV and size(0, E=-1)[0] == INV and size(0, rows=0) == (OK, 0)


@pytest.fixture
def no_lib(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(ops, "lib", boom)


def _bf(*shape):
    return FakeGpuTensor(shape, torch.bfloat16)


def _i32(*shape):
    return FakeGpuTensor(shape, torch.int32)


def _f32(*shape):
    return FakeGpuTensor(shape, torch.float32)


@pytest.mark.parametrize("fn,a,b", [(g5.gemm_bf16_grouped_nt, (300, 64), (4, 48, 64)),
                                    (g5.gemm_bf16_grouped, (300, 64), (4, 64, 48)),
                                    (g5.gemm_bf16_grouped_tn, (300, 48), (300, 64))])
def test_grouped_binding_refuses(no_lib, fn, a, b):
    o = _i32(5)
    for bad in ((_f32(*a), _bf(*b)), (_bf(*a), _f32(*b))):
        with pytest.raises(TypeError):
            fn(*bad, o)
    for bad in ((_bf(*a), _bf(4, *b), o), (_bf(2, *a), _bf(*b), o), (_bf(*a), _bf(*b), _i32(5, 1)),
                (_bf(*a), _bf(*b), _i32(0)), (_bf(*a), _bf(*b), torch.zeros(5, dtype=torch.int32)),
                (torch.zeros(a, dtype=torch.bfloat16), _bf(*b), o)):
        with pytest.raises(ValueError):
            fn(*bad)
    with pytest.raises(ValueError):
        fn(_bf(*a), _bf(*b), FakeGpuTensor((5,), torch.int64))
    # sizes that do not fit each other, an output of another shape
    with pytest.raises(ValueError):
        fn(_bf(*a), _bf(*b[:-1], 65) if fn is g5.gemm_bf16_grouped_nt else _bf(b[0], 63, 48) if len(b) == 3 else _bf(299, 64), o)
    with pytest.raises(ValueError):
        fn(_bf(*a), _bf(*b), o, C=_bf(300, 47))
    with pytest.raises(TypeError):
        fn(_bf(*a), _bf(*b), o, C=FakeGpuTensor((4, 48, 64) if len(b) == 2 else (300, 48), torch.float16))


def test_grouped_binding_counts_groups(no_lib):
    with pytest.raises(ValueError):
        g5.gemm_bf16_grouped_nt(_bf(300, 64), _bf(4, 48, 64), _i32(4))
    with pytest.raises(ValueError):
        g5.gemm_bf16_grouped(_bf(300, 64), _bf(4, 64, 48), _i32(6))


X, D = P + (6 << 34), P + (7 << 34)


def loss(kind, **kw):
    """kind: 'ce', 'ce_grad', 'kd', 'kd_grad'; 300 rows of 64, 1000 tokens, 4 entries."""
    a = dict(M=300, V=1000, K=64, X=A, ldx=64, W=B, ldw=64, scale=1.0, topk=4, ids=O, nb=8, t=T, dl=X, lse=X + 4096,
             loss=C, out=C + 4096, dX=C, lddx=64, dW=D, lddw=64, dt=0, ws=W, n=1 << 30)
    a.update(kw)
    L = g5.lib()
    head = (a["M"], a["V"], a["K"], a["X"], a["ldx"], a["W"], a["ldw"], a["scale"])
    head += (a["topk"], a["ids"], a["nb"], a["t"]) if kind.startswith("kd") else (a["ids"], a["nb"])
    tail = (a["ws"], a["n"], None)
    grad = (a["dl"], a["lse"], a["dX"], a["lddx"], a["dW"], a["lddw"], a["dt"])
    fn = {"ce": L.gemm_linear_cross_entropy, "ce_grad": L.gemm_linear_cross_entropy_backward,
          "kd": L.gemm_linear_distill, "kd_grad": L.gemm_linear_distill_backward}[kind]
    return fn(*head, *(grad if kind.endswith("grad") else (a["loss"], a["out"])), *tail)


KINDS = ["ce", "ce_grad", "kd", "kd_grad"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INV), (dict(M=(1 << 24) + 1), INV), (dict(V=0), INV), (dict(V=1 << 31), INV), (dict(K=0), INV),
    (dict(K=(1 << 21) + 1), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(nb=2), INV), (dict(X=None), INV), (dict(W=None), INV), (dict(ids=None), INV),
    (dict(ldx=63), INV), (dict(ldw=63), INV), (dict(X=A + 1), INV), (dict(W=B + 1), INV), (dict(ids=O + 4), INV),
    (dict(nb=4, ids=O + 2), INV), (dict(ws=None), WS), (dict(n=CR), WS), (dict(ws=W + 128), INV), (dict(ws=A), INV),
    (dict(ws=B), INV), (dict(ldx=(1 << 21) + 8), UNS), (dict(ldw=(1 << 21) + 8), UNS)])
def test_loss_refuses(kind, bad, status):
    assert loss(kind, **bad) == status


@pytest.mark.parametrize("kind", ["ce", "kd"])
@pytest.mark.parametrize("bad", [dict(loss=None), dict(loss=C + 2), dict(out=C + 4098), dict(loss=A), dict(out=B), dict(out=C),
                                 dict(loss=O), dict(ws=C)])
def test_loss_forward_refuses(kind, bad):
    assert loss(kind, **bad) == INV


@pytest.mark.parametrize("kind", ["ce_grad", "kd_grad"])
@pytest.mark.parametrize("bad", [dict(dl=None), dict(lse=None), dict(dl=X + 2), dict(lse=X + 2), dict(lddx=63),
                                 dict(lddw=63), dict(dX=C + 1), dict(dW=D + 1), dict(dt=1, dW=D + 2), dict(dt=2),
                                 dict(dX=A), dict(dX=B), dict(dW=B), dict(dW=C), dict(dX=X), dict(dW=O), dict(ws=D)])
def test_loss_gradient_refuses(kind, bad):
    assert loss(kind, **bad) == INV


@pytest.mark.parametrize("kind", ["kd", "kd_grad"])
@pytest.mark.parametrize("bad", [dict(topk=0), dict(topk=257), dict(t=None), dict(t=T + 2)])
def test_distill_refuses(kind, bad):
    assert loss(kind, **bad) == INV


def test_loss_empty_calls_do_nothing():
    assert loss("ce", M=0, X=None, ids=None, loss=None) == OK and loss("kd", M=0, t=None, loss=None) == OK
    assert loss("ce_grad", dX=None, dW=None, dl=X) == OK and loss("kd_grad", M=0, dW=None, t=None) == OK


def test_loss_workspace_size():
    n = ctypes.c_uint64(1)

    def size(back, M=300, V=1000, K=64, topk=1, x=A, ldx=64, w=B, ldw=64):
        st = g5.lib().gemm_linear_loss_workspace_size(back, M, V, K, topk, x, ldx, w, ldw, ctypes.byref(n))
        return st, n.value

    up = lambda b: -(-b // 256) * 256                                      # noqa: E731
    assert size(0) == (OK, CR + up(8 * 300 * 8) + up(300 * 4))             # 8 column tiles, the targets' logits
    assert size(0, x=A + 2) == (OK, CR + up(300 * 64 * 2) + up(8 * 300 * 8) + up(300 * 4))
    assert size(0, K=58, x=A + 4, ldx=58, w=B + 8, ldw=62) == size(0)
    assert size(0, M=32, x=A + 2, w=B + 2) == (OK, CR + up(32 * 32 * 8) + up(32 * 4))     # the stream
    assert size(0, M=0) == size(1, M=0) == (OK, 0)
    st, whole = size(1)
    assert st == OK and whole >= CR + 300 * 64 * 2 + 300 * 1000 * 2 + 300 * 64 * 4
    # a large vocabulary goes in pieces: far less than the logits
    st, b = size(1, M=1 << 15, V=1 << 17, K=1024, ldx=1024, ldw=1024)
    assert st == OK and b < 1 << 29
    assert size(0, V=0)[0] == INV and size(0, K=0)[0] == INV and size(1, topk=0)[0] == INV
    assert g5.lib().gemm_linear_loss_workspace_size(1, 300, 1000, 64, 1, A, 64, B, 64, None) == OK


@pytest.mark.parametrize("M,K", [(1, 2), (4, 32), (8, 32), (15, 32), (15, 31), (4, 56), (40, 2)])
def test_loss_gradient_pieces_end(M, K):
    """Few rows and a vocabulary of short rows: a piece holds no more tokens
    than 64 rows of its D have 32-bit offsets for, so a vocabulary of more needs
    no more than one of 2^23."""
    def size(V):
        n = ctypes.c_uint64(0)
        assert g5.lib().gemm_linear_loss_workspace_size(1, M, V, K, 1, A, K, B, K, ctypes.byref(n)) == OK
        return n.value

    most = size(1 << 23)
    for V in ((1 << 23) + 1, (1 << 23) + 4096, 10_000_000, 1 << 24, 1 << 27, (1 << 31) - 257):
        assert size(V) == most, V


def test_loss_binding_refuses(no_lib):
    x, w, t, f = _bf(30, 64), _bf(100, 64), FakeGpuTensor((30,), torch.int64), _f32(30)
    ids, lg = _i32(30, 4), _f32(30, 4)
    for bad in ((_f32(30, 64), w, t), (x, _f32(100, 64), t), (x, w, _f32(30))):
        with pytest.raises(TypeError):
            g5.linear_cross_entropy(*bad)
        with pytest.raises(TypeError):
            g5.linear_cross_entropy_backward(f, *bad, f)
    for bad in ((_bf(30, 65), w, t), (_bf(2, 30, 64), w, t), (x, w, _i32(31)), (x, w, _i32(30, 1)),
                (torch.zeros((30, 64), dtype=torch.bfloat16), w, t), (x, w, torch.zeros(30, dtype=torch.int32))):
        with pytest.raises(ValueError):
            g5.linear_cross_entropy(*bad)
        with pytest.raises(ValueError):
            g5.linear_cross_entropy_backward(f, *bad, f)
    for kw in (dict(loss=_f32(31)), dict(lse=_bf(30)), dict(loss=torch.zeros(30))):
        with pytest.raises(ValueError):
            g5.linear_cross_entropy(x, w, t, **kw)
    with pytest.raises(ValueError):
        g5.linear_cross_entropy_backward(_f32(29), x, w, t, f)
    with pytest.raises(ValueError):
        g5.linear_cross_entropy_backward(f, x, w, t, None)
    for kw in (dict(dX=_bf(30, 65)), dict(dX=_f32(30, 64)), dict(dW=_bf(99, 64)), dict(dW=torch.zeros((100, 64)))):
        with pytest.raises(ValueError):
            g5.linear_cross_entropy_backward(f, x, w, t, f, **kw)
    with pytest.raises(TypeError):
        g5.linear_cross_entropy_backward(f, x, w, t, f, dw_dtype=torch.float16)
    for bad in ((t, lg), (_i32(31, 4), lg), (_i32(30, 257), _f32(30, 257)), (_i32(30, 0), _f32(30, 0)), (ids, _f32(30, 5)),
                (ids, _bf(30, 4)), (ids, None)):
        with pytest.raises(ValueError):
            g5.linear_distill(x, w, *bad)
        with pytest.raises(ValueError):
            g5.linear_distill_backward(f, x, w, *bad, f)
