"""Host-only checks of the operators of a training step: arguments refused
before anything is enqueued (no GPU), and the sizes their workspaces need."""
import ctypes

import pytest
import torch

import dense_gemm_05_amd as g5
from dense_gemm_05_amd import train_ops as ops
from test_binding_host import FakeGpuTensor

P = 0x7F0000000000     # fake, aligned addresses 16 GiB apart, never dereferenced
A, B, C, O, T, W = (P + (i << 34) for i in range(6))
INV, WS, OK, UNS = g5.GEMM_ERR_INVALID_ARG, g5.GEMM_ERR_WORKSPACE, g5.GEMM_OK, g5.GEMM_ERR_UNSUPPORTED
CR = g5.GEMM_WORKSPACE_COUNTER_BYTES


def grouped(kind, **kw):
    """4 groups, 300 rows: nt and nn [300, 64] by [4, ., .] to 48 columns; tn [300, 48] by [300, 64]."""
    tn = kind == 2
    a = dict(E=4, rows=300, M=48, N=64 if tn else 48, K=64, O=O, A=A, lda=48 if tn else 64, B=B,
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
    assert grouped(1, N=44, ldb=48) == WS and grouped(2, N=60) == WS and grouped(2, M=44) == WS
    # more workgroups than a launch takes
    assert grouped(2, E=4096, M=1 << 20, N=1 << 20, lda=1 << 20, ldb=1 << 20, ldc=1 << 20, sC=1 << 40) == UNS


def test_grouped_empty_calls_do_nothing():
    for kind in (0, 1, 2):
        assert grouped(kind, E=0, O=None, A=None) == OK and grouped(kind, N=0, C=None) == OK
    assert grouped(0, rows=0, C=None) == OK and grouped(2, M=0, C=None) == OK


def test_grouped_workspace_size():
    n = ctypes.c_uint64(1)

    def size(kind, E=4, rows=300, M=48, N=64, K=64, a=A, lda=64, b=B, ldb=64, sB=4096):
        st = g5.lib().gemm_grouped_workspace_size(kind, E, rows, M, N, K, a, lda, b, ldb, sB, ctypes.byref(n))
        return st, n.value

    assert size(0) == size(1) == size(2) == (OK, 0)
    up = lambda b: -(-b // 256) * 256                                      # noqa: E731
    assert size(0, a=A + 2) == (OK, CR + up(300 * 64 * 2))
    assert size(0, K=60, ldb=60, sB=64 * 60) == (OK, CR + up(4 * 64 * 64 * 2))
    assert size(1, N=60) == (OK, CR + up(4 * 64 * 64 * 2)) and size(1, N=60, sB=0) == (OK, CR + up(64 * 64 * 2))
    assert size(2, M=44, N=60) == (OK, CR + up(300 * 48 * 2) + up(300 * 64 * 2))
    # the stream takes rows of any alignment
    assert size(0, rows=128, a=A + 2, b=B + 2) == (OK, 0)
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
