"""Binding of the operators at both ends of a training step's products: the
experts' products with ragged numbers of rows, and the loss over a vocabulary
behind the last projection with its gradient, from labels or from a teacher's
best logits.  As gemm.py: argument marshalling only; the arithmetic runs in the
gfx950 kernels of libgemm05.so.
"""
import ctypes

import torch

from ._lib import GEMM_ERR_WORKSPACE, GemmError, lib
from .gemm import Workspace, _bstride, _check_dev, _launch, _out_code
from .token_ops import _ptr, _rows, _scratch, _stride, _vector

__all__ = ["gemm_bf16_grouped_nt", "gemm_bf16_grouped", "gemm_bf16_grouped_tn",
           "linear_cross_entropy", "linear_cross_entropy_backward", "linear_distill", "linear_distill_backward"]

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


def _loss_operands(what, X, Wt, ids, teacher):
    """(M, V, K, topk, bytes of an index)"""
    if X.dtype != torch.bfloat16 or Wt.dtype != torch.bfloat16:
        raise TypeError(f"{what} takes a bfloat16 X and Wt")
    if X.dim() != 2 or Wt.dim() != 2 or X.shape[1] != Wt.shape[1]:
        raise ValueError(f"{what} takes X [M, K] and Wt [V, K]")
    M, K = X.shape
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what} takes int32 or int64 indices")
    if teacher is None:
        if ids.dim() != 1 or ids.shape[0] != M or (M > 1 and ids.stride(0) != 1):
            raise ValueError("targets must be a contiguous vector of M elements")
        topk = 1
    else:
        if ids.dim() != 2 or ids.shape[0] != M or not ids.is_contiguous():
            raise ValueError("ids must be contiguous [M, topk]")
        topk = ids.shape[1]
        if not 1 <= topk <= 256:
            raise ValueError("topk must be 1 to 256")
        _rows(teacher, ids.shape, torch.float32, "teacher")
        if not teacher.is_contiguous():
            raise ValueError("teacher must be contiguous [M, topk]")
    return M, Wt.shape[0], K, topk, 4 if ids.dtype == torch.int32 else 8


def _loss(what, X, Wt, ids, teacher, scale, loss, lse, workspace):
    M, V, K, topk, nb = _loss_operands(what, X, Wt, ids, teacher)
    _vector(loss, M, torch.float32, "loss")
    _vector(lse, M, torch.float32, "lse")
    dev = _check_dev(X, Wt, ids, teacher, loss, lse)
    if loss is None:
        loss = torch.empty((M,), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((M,), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = Workspace(dev)
    px, pw, ldx, ldw = X.data_ptr(), Wt.data_ptr(), _stride(X, K), _stride(Wt, K)
    picks = (ids.data_ptr(), nb) if teacher is None else (topk, ids.data_ptr(), nb, teacher.data_ptr())
    fn = getattr(lib(), what)

    def run(buf):
        return _launch(fn, dev, M, V, K, px, ldx, pw, ldw, scale, *picks, loss.data_ptr(), lse.data_ptr(), _ptr(buf),
                       0 if buf is None else buf.numel())

    # (the size depends on the pointers only through their alignment)
    _with_scratch(what, workspace, dev, (what, M, V, K, topk, px % 256, ldx, pw % 256, ldw),
                  lambda n: lib().gemm_linear_loss_workspace_size(0, M, V, K, topk, px, ldx, pw, ldw, n), run)
    return loss, lse


def _loss_backward(what, dloss, X, Wt, ids, teacher, lse, scale, dX, dW, need_dx, need_dw, dw_dtype, workspace):
    M, V, K, topk, nb = _loss_operands(what, X, Wt, ids, teacher)
    if dloss is None or lse is None:
        raise ValueError("dloss and the forward call's lse are needed")
    _vector(dloss, M, torch.float32, "dloss")
    _vector(lse, M, torch.float32, "lse")
    _rows(dX, (M, K), torch.bfloat16, "dX")
    if dW is not None and tuple(dW.shape) != (V, K):
        raise ValueError("dW must be [V, K]")
    code = _out_code(dw_dtype if dW is None else dW.dtype)
    dev = _check_dev(X, Wt, ids, teacher, dloss, lse, dX, dW)
    if not need_dx:
        dX = None
    elif dX is None:
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    if not need_dw:
        dW = None
    elif dW is None:
        dW = torch.empty((V, K), dtype=dw_dtype, device=dev)
    if workspace is None:
        workspace = Workspace(dev)
    px, pw, ldx, ldw = X.data_ptr(), Wt.data_ptr(), _stride(X, K), _stride(Wt, K)
    picks = (ids.data_ptr(), nb) if teacher is None else (topk, ids.data_ptr(), nb, teacher.data_ptr())
    fn = getattr(lib(), what)

    def run(buf):
        return _launch(fn, dev, M, V, K, px, ldx, pw, ldw, scale, *picks, dloss.data_ptr(), lse.data_ptr(), _ptr(dX),
                       K if dX is None else _stride(dX, K), _ptr(dW), K if dW is None else _stride(dW, K), code,
                       _ptr(buf), 0 if buf is None else buf.numel())

    _with_scratch(what, workspace, dev, (what, M, V, K, topk, px % 256, ldx, pw % 256, ldw),
                  lambda n: lib().gemm_linear_loss_workspace_size(1, M, V, K, topk, px, ldx, pw, ldw, n), run)
    return dX, dW


def linear_cross_entropy(X, Wt, targets, scale=1.0, loss=None, lse=None, workspace=None):
    """The cross entropy of softmax(scale X . Wt^T) with targets, without the
    logits in memory (gemm_linear_cross_entropy): X [M, K] and the vocabulary's
    weight Wt [V, K] in bfloat16, targets [M] int32 or int64; a target outside
    [0, V) (-100, -1) leaves its row out.  Returns (loss, lse), float32 [M]:
    loss 0 in rows left out, lse what the gradient needs."""
    return _loss("gemm_linear_cross_entropy", X, Wt, targets, None, scale, loss, lse, workspace)


def linear_cross_entropy_backward(dloss, X, Wt, targets, lse, scale=1.0, dX=None, dW=None, need_dx=True, need_dw=True,
                                  dw_dtype=torch.bfloat16, workspace=None):
    """The gradient of linear_cross_entropy (gemm_linear_cross_entropy_backward):
    from dloss float32 [M] (1 / rows for a mean) and the forward call's lse,
    returns (dX bfloat16 [M, K], dW [V, K] in dw_dtype, bfloat16 or float32);
    None for one that is not needed."""
    return _loss_backward("gemm_linear_cross_entropy_backward", dloss, X, Wt, targets, None, lse, scale, dX, dW, need_dx,
                          need_dw, dw_dtype, workspace)


def _teacher(teacher):
    if teacher is None:
        raise ValueError("teacher: the logits of ids")
    return teacher


def linear_distill(X, Wt, ids, teacher, scale=1.0, loss=None, lse=None, workspace=None):
    """The distance (Kullback-Leibler) of softmax(scale X . Wt^T) to a teacher of
    which each row's topk best tokens are kept (gemm_linear_distill): ids [M,
    topk] (int32 or int64, outside [0, V): no entry) and their logits teacher
    [M, topk] (float32; -inf: no entry), weighted by softmax(scale teacher).
    scale: 1 over the temperature.  Returns (loss, lse), float32 [M]; a row
    without entries has loss 0."""
    return _loss("gemm_linear_distill", X, Wt, ids, _teacher(teacher), scale, loss, lse, workspace)


def linear_distill_backward(dloss, X, Wt, ids, teacher, lse, scale=1.0, dX=None, dW=None, need_dx=True, need_dw=True,
                            dw_dtype=torch.bfloat16, workspace=None):
    """The gradient of linear_distill in X and Wt (gemm_linear_distill_backward);
    otherwise as linear_cross_entropy_backward."""
    return _loss_backward("gemm_linear_distill_backward", dloss, X, Wt, ids, _teacher(teacher), lse, scale, dX, dW, need_dx,
                          need_dw, dw_dtype, workspace)
