"""Host-only checks of the operators around a projection: arguments refused
before anything is enqueued (no GPU), and the sizes their workspaces need."""
import ctypes

import pytest
import torch

import dense_gemm_05_amd as g5
from dense_gemm_05_amd import token_ops as ops
from test_binding_host import FakeGpuTensor

P = 0x7F0000000000     # fake, aligned addresses 16 GiB apart, never dereferenced
X, R, H, W, Y, S, T = (P + (i << 34) for i in range(7))
INV, WS, OK = g5.GEMM_ERR_INVALID_ARG, g5.GEMM_ERR_WORKSPACE, g5.GEMM_OK
CR = g5.GEMM_WORKSPACE_COUNTER_BYTES


def norm(**kw):
    a = dict(rows=4, cols=64, X=X, ldx=64, R=R, ldr=64, H=H, ldh=64, W=W, eps=1e-6, Y=Y, ldy=64, t=0, scale=None,
             rstd=None)
    a.update(kw)
    return g5.lib().gemm_rms_norm(a["rows"], a["cols"], a["X"], a["ldx"], a["R"], a["ldr"], a["H"], a["ldh"], a["W"],
                                  a["eps"], a["Y"], a["ldy"], a["t"], a["scale"], a["rstd"], None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(X=None), dict(Y=None), dict(ldx=63), dict(ldr=63),
    dict(ldh=63), dict(ldy=63), dict(t=1), dict(t=3), dict(t=2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(R=None), dict(X=X + 1), dict(R=R + 1), dict(H=H + 1), dict(W=W + 1), dict(Y=Y + 1),
    dict(rstd=T + 2), dict(t=2, scale=S + 2),
    dict(Y=X), dict(Y=R), dict(Y=H), dict(Y=W), dict(H=X + 128), dict(H=X, ldh=128), dict(H=R, ldh=72),
    dict(rstd=X), dict(rstd=Y), dict(t=2, scale=Y), dict(t=2, scale=S, rstd=S), dict(H=W),
    dict(Y=X + 2 * 3 * 64 + 126)])
def test_norm_refuses(bad):
    assert norm(**bad) == INV


def grad(**kw):
    a = dict(rows=4, cols=64, dY=X, lddy=64, H=H, ldh=64, W=W, rstd=S, dH=R, lddh=64, dX=Y, lddx=64, dW=T, ws=P + (8 << 34),
             n=CR + 4096)
    a.update(kw)
    return g5.lib().gemm_rms_norm_backward(a["rows"], a["cols"], a["dY"], a["lddy"], a["H"], a["ldh"], a["W"], a["rstd"],
                                           a["dH"], a["lddh"], a["dX"], a["lddx"], a["dW"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), INV), (dict(cols=-2), INV), (dict(rows=1 << 31), INV), (dict(dY=None), INV), (dict(H=None), INV),
    (dict(rstd=None), INV), (dict(dX=None), INV), (dict(lddy=63), INV), (dict(ldh=63), INV), (dict(lddh=63), INV),
    (dict(lddx=63), INV), (dict(dY=X + 1), INV), (dict(H=H + 1), INV), (dict(W=W + 1), INV), (dict(dH=R + 1), INV),
    (dict(dX=Y + 1), INV), (dict(rstd=S + 2), INV), (dict(dW=T + 2), INV), (dict(dX=X), INV), (dict(dX=H), INV),
    (dict(dX=R), INV), (dict(dW=S), INV), (dict(dW=Y), INV), (dict(ws=None), WS), (dict(n=CR + 1023), WS),
    (dict(ws=P + (8 << 34) + 128), INV), (dict(ws=H), INV), (dict(rows=0, dW=T + 2), INV)])
def test_norm_gradient_refuses(bad, status):
    assert grad(**bad) == status


def test_norm_empty_calls_do_nothing():
    assert norm(rows=0, X=None, Y=None) == OK and norm(cols=0, X=None, Y=None) == OK
    assert grad(cols=0, dY=None) == OK and grad(rows=0, dW=None, dY=None) == OK


def test_norm_workspace_size():
    n = ctypes.c_uint64(1)
    f = g5.lib().gemm_rms_norm_workspace_size
    assert f(0, 64, ctypes.byref(n)) == OK and n.value == 0
    assert f(3, 64, ctypes.byref(n)) == OK and n.value == CR + 3 * 64 * 4
    big = n.value
    assert f(1 << 20, 4096, ctypes.byref(n)) == OK and n.value > big
    assert f(-1, 64, ctypes.byref(n)) == INV and f(4, -1, ctypes.byref(n)) == INV
    assert f(4, 64, None) == OK


@pytest.fixture
def no_lib(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(ops, "lib", boom)


def _bf(*shape):
    return FakeGpuTensor(shape, torch.bfloat16)


def _f32(*shape):
    return FakeGpuTensor(shape, torch.float32)


def test_norm_binding_refuses(no_lib):
    x = _bf(4, 64)
    for fn in (g5.rms_norm, g5.rms_norm_e4m3):
        with pytest.raises(TypeError):
            fn(_f32(4, 64))
        with pytest.raises(TypeError):
            fn(_bf(4, 2, 32))
        with pytest.raises(ValueError):
            fn(x, _bf(65))
        with pytest.raises(ValueError):
            fn(x, _f32(64))
        with pytest.raises(ValueError):
            fn(x, residual=_bf(4, 65))
        with pytest.raises(ValueError):
            fn(x, H=_bf(4, 64))
        with pytest.raises(ValueError):
            fn(x, rstd=_f32(5))
        with pytest.raises(ValueError):
            fn(x, residual=torch.empty((4, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        g5.rms_norm(x, Y=_f32(4, 64))
    with pytest.raises(ValueError):
        g5.rms_norm_e4m3(x, Q=_bf(4, 64))
    with pytest.raises(ValueError):
        g5.rms_norm_e4m3(x, Q=FakeGpuTensor((4, 64), torch.uint8), scale=_f32(3))


def test_norm_gradient_binding_refuses(no_lib):
    x, s = _bf(4, 64), _f32(4)
    with pytest.raises(TypeError):
        g5.rms_norm_backward(_f32(4, 64), x, None, s)
    for bad in (dict(H=_bf(4, 65)), dict(W=_bf(63)), dict(rstd=_f32(3)), dict(rstd=None), dict(dH=_bf(3, 64)),
                dict(dX=_f32(4, 64)), dict(dX=torch.empty((4, 64), dtype=torch.bfloat16))):
        a = dict(H=x, W=None, rstd=s)
        a.update(bad)
        with pytest.raises(ValueError):
            g5.rms_norm_backward(x, a.pop("H"), a.pop("W"), a.pop("rstd"), **a)


def moe(**kw):
    a = dict(T=4, H=64, I=32, E=8, k=2, renorm=1, X=X, ldx=64, L=S, ldl=8, wt=0, Wgu=W, ldgu=64, sgu=64 * 64, fgu=None,
             Wd=H, ldd=32, sd=64 * 32, fd=None, Y=Y, ldy=64, ct=0, ids=T, gates=T + 4096, ws=P + (8 << 34), n=CR + (1 << 20))
    a.update(kw)
    return g5.lib().gemm_moe_swiglu(a["T"], a["H"], a["I"], a["E"], a["k"], a["renorm"], a["X"], a["ldx"], a["L"],
                                    a["ldl"], a["wt"], a["Wgu"], a["ldgu"], a["sgu"], a["fgu"], a["Wd"], a["ldd"],
                                    a["sd"], a["fd"], a["Y"], a["ldy"], a["ct"], a["ids"], a["gates"], a["ws"], a["n"],
                                    None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INV), (dict(T=65), INV), (dict(H=-1), INV), (dict(H=65537), INV), (dict(I=-1), INV),
    (dict(I=65537), INV), (dict(E=0), INV), (dict(E=1025), INV), (dict(k=0), INV), (dict(k=9), INV),
    (dict(E=64, ldl=64, k=17), INV), (dict(wt=1), INV), (dict(ct=2), INV), (dict(X=None), INV), (dict(L=None), INV),
    (dict(Wgu=None), INV), (dict(Wd=None), INV), (dict(Y=None), INV), (dict(ldx=63), INV), (dict(ldl=7), INV),
    (dict(ldgu=63), INV), (dict(ldd=31), INV), (dict(ldy=63), INV), (dict(sgu=-1), INV), (dict(sd=-1), INV),
    (dict(X=X + 1), INV), (dict(L=S + 2), INV), (dict(Wgu=W + 1), INV), (dict(Wd=H + 1), INV), (dict(Y=Y + 1), INV),
    (dict(ct=1, Y=Y + 2), INV), (dict(ids=T + 2), INV), (dict(gates=T + 4098), INV), (dict(fgu=R), INV),
    (dict(wt=2, fgu=R + 2), INV), (dict(wt=2, fd=R + 1), INV), (dict(Y=X), INV), (dict(Y=W), INV), (dict(ids=S), INV),
    (dict(gates=T), INV), (dict(ids=Y), INV), (dict(ws=None), WS), (dict(n=CR), WS), (dict(ws=P + (8 << 34) + 64), INV),
    (dict(ws=H), INV), (dict(ws=Y), INV)])
def test_moe_refuses(bad, status):
    assert moe(**bad) == status


@pytest.mark.parametrize("far", [dict(ldx=1 << 24), dict(ldgu=1 << 26, sgu=1 << 33), dict(ldd=1 << 26, sd=1 << 33),
                                 dict(wt=2, ldgu=1 << 27, sgu=1 << 33), dict(wt=2, ldd=1 << 27, sd=1 << 33)])
def test_moe_far_rows_are_refused(far):
    """Rows farther apart than the kernels' 32-bit byte offsets reach."""
    apart = dict(X=P + (16 << 44), L=P + (17 << 44), Wgu=P + (18 << 44), Wd=P + (19 << 44), Y=P + (20 << 44),
                 ids=P + (21 << 44), gates=P + (22 << 44), ws=P + (23 << 44))
    assert moe(**apart, **far) == g5.GEMM_ERR_UNSUPPORTED


def test_moe_workspace_size():
    n = ctypes.c_uint64(1)
    f = g5.lib().gemm_moe_workspace_size
    assert f(0, 64, 32, 8, 2, ctypes.byref(n)) == OK and n.value == 0
    assert f(4, 64, 32, 8, 2, ctypes.byref(n)) == OK
    # routing (2 x 8 words), the number of experts, 8 of them, 8 pairs, z in
    # two planes of 8 x 128 bf16
    assert n.value == CR + 256 + 256 + 256 + 256 + 256 + 4096
    assert f(65, 64, 32, 8, 2, ctypes.byref(n)) == INV and f(4, 64, 32, 8, 9, ctypes.byref(n)) == INV
    assert moe(T=0, X=None, L=None) == OK


def test_moe_binding_refuses(no_lib):
    x, l, w, d = _bf(4, 64), _f32(4, 8), _bf(8, 64, 64), _bf(8, 64, 32)
    with pytest.raises(TypeError):
        g5.moe_swiglu(_f32(4, 64), l, 2, w, d)
    with pytest.raises(TypeError):
        g5.moe_swiglu(x, _bf(4, 8), 2, w, d)
    with pytest.raises(TypeError):
        g5.moe_swiglu(x, l, 2, w, FakeGpuTensor((8, 64, 32), torch.uint8))
    with pytest.raises(TypeError):
        g5.moe_swiglu(x, l, 2, _f32(8, 64, 64), d)
    for bad in (dict(X=_bf(4, 63)), dict(logits=_f32(4, 9)), dict(Wgu=_bf(8, 63, 64)), dict(Wd=_bf(8, 64, 33)),
                dict(Wgu=_bf(64, 64)), dict(scale_gu=_f32(8, 64)),
                dict(logits=torch.empty((4, 8)))):
        a = dict(X=x, logits=l, topk=2, Wgu=w, Wd=d)
        a.update(bad)
        with pytest.raises(ValueError):
            g5.moe_swiglu(**a)


def lora(**kw):
    a = dict(M=4, N=64, K=32, X=X, ldx=32, Wt=W, ldw=32, L=2, R=8, A=R, lda=32, sA=256, B=H, ldb=8, sB=512, scale=S,
             idx=S + 4096, C=Y, ldc=64, ct=0, ws=T, n=CR + 4096)
    a.update(kw)
    return g5.lib().gemm_bf16_nt_lora(a["M"], a["N"], a["K"], a["X"], a["ldx"], a["Wt"], a["ldw"], a["L"], a["R"], a["A"],
                                      a["lda"], a["sA"], a["B"], a["ldb"], a["sB"], a["scale"], a["idx"], a["C"],
                                      a["ldc"], a["ct"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-1), INV), (dict(L=-1), INV), (dict(L=1 << 31), INV),
    (dict(R=-1), INV), (dict(R=4097, ldb=4097), INV), (dict(X=None), INV), (dict(Wt=None), INV), (dict(C=None), INV),
    (dict(A=None), INV), (dict(B=None), INV), (dict(idx=None), INV), (dict(ldx=31), INV), (dict(ldw=31), INV),
    (dict(lda=31), INV), (dict(ldb=7), INV), (dict(ldc=63), INV), (dict(sA=-1), INV), (dict(sB=-1), INV),
    (dict(ct=2), INV), (dict(A=R + 1), INV), (dict(B=H + 1), INV), (dict(scale=S + 2), INV), (dict(idx=S + 4097), INV),
    (dict(C=X), INV), (dict(C=W), INV), (dict(C=R), INV), (dict(C=H), INV), (dict(C=S), INV), (dict(ws=None), WS),
    (dict(n=CR), WS), (dict(ws=T + 128), INV), (dict(ws=H), INV), (dict(ws=Y), INV), (dict(ws=S), INV)])
def test_lora_refuses(bad, status):
    assert lora(**bad) == status


def lora_size(M, N, K, L, R, ldx=None):
    n = ctypes.c_uint64(1)
    st = g5.lib().gemm_lora_workspace_size(M, N, K, L, R, X, ldx or K, W, K, Y, N, 0, ctypes.byref(n))
    return st, n.value


def test_lora_workspace_size():
    # one slice of 4 rows of 8 floats; four slices of 16 rows of 24
    assert lora_size(4, 64, 32, 2, 8) == (OK, CR + 256)
    assert lora_size(16, 64, 2048, 2, 17) == (OK, CR + 4 * 16 * 24 * 4)
    # the product's own scratch comes first
    st, own = g5.plan_query(g5.GEMM_OP_BF16_NT, 128, 1536, 4096)[0], g5.plan_query(g5.GEMM_OP_BF16_NT, 128, 1536, 4096)[1]
    st2, n = lora_size(128, 1536, 4096, 2, 16)
    assert st == st2 == OK and n > own.workspace_bytes >= CR
    assert lora_size(0, 64, 32, 2, 8) == (OK, 0) and lora_size(4, 64, 0, 2, 8)[1] == 0
    assert lora_size(4, 64, 32, -1, 8)[0] == INV and lora_size(-4, 64, 32, 1, 8)[0] == INV
    # rows that only 4-byte copies could read are realigned: their copy is counted
    assert lora_size(200, 640, 1024, 2, 8, ldx=1026)[1] >= CR + 200 * 1024 * 2


def test_lora_far_rows():
    """Rows of 2^27 elements or more do not reach the small-M kernel's 32-bit
    offsets: a few of them go to the tiled kernels (a workspace of two bf16
    parts instead of four slices), an operand past 2 GiB is refused."""
    def size(M, ldx):
        n = ctypes.c_uint64(1)
        st = g5.lib().gemm_lora_workspace_size(M, 64, 2048, 2, 16, P + (16 << 44), ldx, P + (17 << 44), 2048,
                                               P + (18 << 44), 64, 0, ctypes.byref(n))
        return st, n.value
    assert size(16, (1 << 27) - 8) == (OK, CR + 4 * 16 * 16 * 4)
    assert size(3, 1 << 27)[0] == OK and size(3, 1 << 27)[1] != CR + 4 * 3 * 16 * 4
    assert size(16, 1 << 27)[0] == g5.GEMM_ERR_UNSUPPORTED


def test_lora_long_rows():
    """Past 2^30 columns, or 128 rows, an operand of 2 GiB is refused."""
    def status(M, K):
        n = ctypes.c_uint64(1)
        return g5.lib().gemm_lora_workspace_size(M, 64, K, 2, 16, P + (16 << 44), K, P + (17 << 44), K, P + (18 << 44), 64,
                                                 0, ctypes.byref(n))
    assert status(17, 1 << 30) == OK and status(128, 1 << 26) == OK
    assert status(17, (1 << 30) + 8) == g5.GEMM_ERR_UNSUPPORTED
    assert status(129, 1 << 26) == g5.GEMM_ERR_UNSUPPORTED


def test_lora_empty_calls_do_nothing():
    assert lora(M=0, X=None, ws=None) == OK and lora(N=0, ldc=0, ws=None) == OK


def test_lora_binding_refuses(no_lib):
    good = dict(X=_bf(4, 32), Wt=_bf(64, 32), A=_bf(2, 8, 32), B=_bf(2, 64, 8), idx=FakeGpuTensor((4,), torch.int32))
    for bad in (dict(X=_f32(4, 32)), dict(Wt=_f32(64, 32)), dict(A=_f32(2, 8, 32)), dict(B=_f32(2, 64, 8)),
                dict(idx=FakeGpuTensor((4,), torch.int64))):
        with pytest.raises(TypeError):
            g5.gemm_bf16_nt_lora(**{**good, **bad})
    for bad in (dict(X=_bf(4, 33)), dict(A=_bf(8, 32)), dict(B=_bf(2, 64, 9)), dict(B=_bf(3, 64, 8)),
                dict(idx=FakeGpuTensor((5,), torch.int32)), dict(scale=_f32(3)), dict(C=_bf(4, 63)),
                dict(idx=torch.zeros(4, dtype=torch.int32)), dict(C=torch.empty((4, 64), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            g5.gemm_bf16_nt_lora(**{**good, **bad})


def test_lora_launches_stay_below_their_threads():
    """What one launch has threads for: up to 16 rows of X, 2^26 weight rows
    on the small-M kernel (beyond, the tiled kernels, as long as Wt spans less
    than 2 GiB); 2^27 - 16 rows of X."""
    def status(M, N, K):
        n = ctypes.c_uint64(1)
        return g5.lib().gemm_lora_workspace_size(M, N, K, 2, 16, P + (16 << 44), K, P + (17 << 44), K, P + (18 << 44), N,
                                                 0, ctypes.byref(n))
    for M in (1, 16):
        assert status(M, 1 << 26, 1024) == OK
        assert status(M, (1 << 26) + 1, 1024) == g5.GEMM_ERR_UNSUPPORTED
        assert status(M, (1 << 26) + 1, 8) == OK
    assert status((1 << 27) - 16, 8, 8) == OK
    assert status((1 << 27) - 15, 8, 8) == g5.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,N,K,R,slices", [
    (17, 64, 4096, 16, 8), (80, 1, 900, 33, 3), (128, 4200, 130, 4, 1), (64, 12288, 1100, 12, 1), (80, 9000, 900, 20, 1),
    (128, 6144, 1300, 8, 2), (17, 16400, 1100, 30, 1)])
def test_lora_sizes_of_the_streaming_kernel(M, N, K, R, slices):
    """17 .. 128 rows up to M N = 786432: K's slices of the low-rank values in
    FP32, and 16-row blocks of 64 columns for each slice of the product (a
    tiled kernel's call has one slice of values and none of these)."""
    blocks = 3 if M <= 48 else 5 if M <= 80 else 8
    values = max(1, min(4, K // 512)) * M * ((R + 7) // 8 * 8) * 4
    parts = (N + 63) // 64 * slices * 4 * blocks * 1024 if slices > 1 else 0
    assert lora_size(M, N, K, 3, R) == (OK, CR + (values + 255) // 256 * 256 + parts)


def test_lora_rows_and_columns_choose_the_kernel():
    """Both sides of M N = 786432: four slices of FP32 values, or the tiled
    kernels' one."""
    for M in (32, 64, 128):
        N = 786432 // M
        assert lora_size(M, N, 2048, 3, 16) == (OK, CR + 4 * M * 16 * 4 + (2 * 96 * 4 * 8 * 1024 if M == 128 else 0))
        st, n = lora_size(M, N + 8, 2048, 3, 16)
        product = g5.plan_query(g5.GEMM_OP_BF16_NT, M, N + 8, 2048)[1].workspace_bytes
        assert st == OK and n == max(product, CR) + M * 16 * 4
