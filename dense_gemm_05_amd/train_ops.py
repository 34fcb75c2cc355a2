"""Binding of the operators at both ends of a training step's products: the
experts' products with ragged numbers of rows.  As gemm.py: argument
marshalling only; the arithmetic runs in the gfx950 kernels of libgemm05.so.
"""
import ctypes

import torch

from ._lib import GEMM_ERR_WORKSPACE, GemmError, lib
from .gemm import Workspace, _bstride, _check_dev, _launch, _out_code
from .token_ops import _ptr, _scratch, _stride, _vector

__all__ = ["gemm_bf16_grouped_nt", "gemm_bf16_grouped", "gemm_bf16_grouped_tn"]

_NT, _NN, _TN = range(3)


def _with_scratch(what, workspace, dev, key, size, run):
    """run(scratch or None) with the bytes that size(ref) asks for, kept by
    the workspace under `key`.  A kept size that went stale (the plan also
    follows the library's environment overrides) is asked for again: nothing
    was launched then."""
    held = workspace._need if isinstance(workspace, Workspace) else {}

    def ask():
        n = ctypes.c_uint64(0)
        st = size(ctypes.byref(n))
        if st != 0:
            raise GemmError(st, what)
        held[key] = n.value
        return n.value

    def call(need):
        return run(_scratch(workspace, dev, need) if need else None)

    need = held.get(key)
    st = call(ask() if need is None else need)
    if st == GEMM_ERR_WORKSPACE and need is not None:
        st = call(ask())
    if st != 0:
        raise GemmError(st, what)


def _grouped(what, kind, A, B, offsets, C, shape, out_dtype, workspace, E, rows, M, N, K):
    _vector(offsets, E + 1, torch.int32, "offsets")
    dev = _check_dev(A, B, offsets, C)
    if C is None:
        C = torch.empty(shape, dtype=out_dtype, device=dev)
    if tuple(C.shape) != shape:
        raise ValueError(f"C must be {list(shape)}")
    code = _out_code(C.dtype)
    pa, pb, pc = A.data_ptr(), B.data_ptr(), C.data_ptr()
    lda, ldb, ldc = _stride(A, A.shape[1]), _stride(B, B.shape[-1]), _stride(C, N)
    sB = 0 if kind == _TN else _bstride(B)
    # (the size depends on the pointers only through their alignment)
    key = (what, E, rows, M, N, K, pa % 256, lda, pb % 256, ldb, sB)
    fn = getattr(lib(), what)

    def run(buf):
        ws = (_ptr(buf), 0 if buf is None else buf.numel())
        if kind == _TN:
            return _launch(fn, dev, E, rows, M, N, offsets.data_ptr(), pa, lda, pb, ldb, pc, ldc, _bstride(C), code, *ws)
        return _launch(fn, dev, E, rows, N, K, offsets.data_ptr(), pa, lda, pb, ldb, sB, pc, ldc, code, *ws)

    _with_scratch(what, workspace, dev, key,
                  lambda n: lib().gemm_grouped_workspace_size(kind, E, rows, M, N, K, pa, lda, pb, ldb, sB, n), run)
    return C


def _operands(what, A, B, dims):
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError(f"{what} takes bfloat16 operands")
    if A.dim() != 2 or B.dim() != dims:
        raise ValueError(f"{what} takes a 2-D first and a {dims}-D second operand")


def _groups(offsets):
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a vector of one more element than there are groups")
    return offsets.shape[0] - 1


def gemm_bf16_grouped_nt(A, Bt, offsets, C=None, out_dtype=torch.bfloat16, workspace=None):
    """C[r] = A[r] . Bt[e]^T for the rows r of group e, offsets[e] ..
    offsets[e + 1] - 1 (gemm_bf16_grouped_nt): the experts' projection of A
    [M, K] by the weights Bt [E, N, K] (bfloat16), offsets int32 [E + 1] on the
    GPU.  Returns C [M, N] in out_dtype; rows of no group are left as they
    are (in a C of the caller's; else their contents are undefined)."""
    _operands("gemm_bf16_grouped_nt", A, Bt, 3)
    E, (M, K), N = _groups(offsets), A.shape, Bt.shape[1]
    if Bt.shape[0] != E or Bt.shape[2] != K:
        raise ValueError("expected A [M, K], Bt [E, N, K] and offsets [E + 1]")
    return _grouped("gemm_bf16_grouped_nt", _NT, A, Bt, offsets, C, (M, N), out_dtype, workspace, E, M, 0, N, K)


def gemm_bf16_grouped(A, B, offsets, C=None, out_dtype=torch.bfloat16, workspace=None):
    """C[r] = A[r] . B[e] for the rows r of group e (gemm_bf16_grouped): with
    A = dY [M, K] and B the projection's weights [E, K, N], its input gradient
    [M, N].  Otherwise as gemm_bf16_grouped_nt."""
    _operands("gemm_bf16_grouped", A, B, 3)
    E, (M, K), N = _groups(offsets), A.shape, B.shape[2]
    if B.shape[0] != E or B.shape[1] != K:
        raise ValueError("expected A [M, K], B [E, K, N] and offsets [E + 1]")
    return _grouped("gemm_bf16_grouped", _NN, A, B, offsets, C, (M, N), out_dtype, workspace, E, M, 0, N, K)


def gemm_bf16_grouped_tn(At, B, offsets, C=None, out_dtype=torch.float32, workspace=None):
    """C[e] = At_e^T . B_e over the rows of group e (gemm_bf16_grouped_tn):
    with At = dY [rows, M] and B = the projection's input [rows, N], its weight
    gradient [E, M, N] (zeros for a group without rows)."""
    _operands("gemm_bf16_grouped_tn", At, B, 2)
    E, (rows, M), N = _groups(offsets), At.shape, B.shape[1]
    if B.shape[0] != rows:
        raise ValueError("expected At [rows, M], B [rows, N] and offsets [E + 1]")
    return _grouped("gemm_bf16_grouped_tn", _TN, At, B, offsets, C, (E, M, N), out_dtype, workspace, E, rows, M, N, 0)
