"""Binding of the operators around a projection: the RMS norm with the
residual's addition and its gradient, the projection with low-rank adapters
and the mixture-of-experts layer for a few tokens.  As gemm.py: argument marshalling only;
the arithmetic runs in the gfx950 kernels of libgemm05.so.
"""
import ctypes

import torch

from . import _lib
from ._lib import GEMM_ERR_WORKSPACE, GemmError, lib
from .gemm import Workspace, _bstride, _check_dev, _codes, _launch, _ld, _out_code

__all__ = ["rms_norm", "rms_norm_e4m3", "rms_norm_backward", "moe_swiglu", "gemm_bf16_nt_lora"]


def _ptr(t):
    return None if t is None else t.data_ptr()


# (A small norm's kernel takes 3 us: what the binding does per call counts.)
def _stride(t, cols):
    """Row stride of a tensor whose last dimension has `cols` elements."""
    return cols if t.is_contiguous() else _ld(t, cols)


def _like(t, dtype):
    """A new contiguous tensor of t's shape on its device."""
    return torch.empty_like(t, dtype=dtype) if t.is_contiguous() else torch.empty(t.shape, dtype=dtype, device=t.device)


def _vector(t, n, dtype, name):
    """A contiguous vector of n elements, or None."""
    if t is not None and (t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1)):
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements")


def _rows(t, shape, dtype, name):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} {list(shape)}")


def _need(workspace, what, *args):
    """Workspace bytes of a call (`what`: the size query, host only), kept by
    the workspace: the answer depends on the arguments alone."""
    if isinstance(workspace, Workspace):
        n = workspace._need.get((what, args))
        if n is not None:
            return n
    out = ctypes.c_uint64(0)
    st = getattr(lib(), what)(*args, ctypes.byref(out))
    if st != 0:
        raise GemmError(st, what)
    if isinstance(workspace, Workspace):
        workspace._need[(what, args)] = out.value
    return out.value


def _scratch(workspace, dev, need):
    """The memory of a Workspace (grown to `need` bytes) or of a uint8 tensor."""
    if workspace is None:
        workspace = Workspace(dev)
    if isinstance(workspace, Workspace):
        if workspace.device != dev:
            raise ValueError("the workspace must be on the operands' GPU")
        return workspace.reserve(need)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or workspace.dim() != 1:
        raise ValueError("a workspace tensor must be a 1-D uint8 tensor")
    if workspace.device != dev:
        raise ValueError("the workspace must be on the operands' GPU")
    return workspace


def _rms_norm(what, X, W, residual, eps, Y, H, rstd, codes, scale):
    shape = X.shape
    if X.dtype != torch.bfloat16 or len(shape) != 2:
        raise TypeError(f"{what} takes a 2-D bfloat16 X")
    rows, cols = shape
    _rows(residual, shape, torch.bfloat16, "residual")
    _vector(W, cols, torch.bfloat16, "W")
    _vector(rstd, rows, torch.float32, "rstd")
    if H is not None and residual is None:
        raise ValueError("H is the sum with a residual: none was given")
    dev = _check_dev(X, W, residual, Y, H, rstd, scale)
    ydt = torch.uint8 if codes else torch.bfloat16
    if Y is None:
        Y = _like(X, ydt)
    else:
        if codes and str(Y.dtype) == "torch.float8_e4m3fn":
            Y = Y.view(torch.uint8)
        _rows(Y, shape, ydt, "Q" if codes else "Y")
    if codes:
        if scale is None:
            scale = torch.empty((rows,), dtype=torch.float32, device=dev)
        else:
            _vector(scale, rows, torch.float32, "scale")
    if residual is not None and H is None:
        H = _like(X, torch.bfloat16)
    else:
        _rows(H, shape, torch.bfloat16, "H")
    st = _launch(lib().gemm_rms_norm, dev, rows, cols, X.data_ptr(), _stride(X, cols), _ptr(residual),
                 cols if residual is None else _stride(residual, cols), _ptr(H), cols if H is None else _stride(H, cols),
                 _ptr(W), eps, Y.data_ptr(), _stride(Y, cols), _lib.GEMM_OUT_E4M3 if codes else _lib.GEMM_OUT_BF16,
                 scale.data_ptr() if codes else None, _ptr(rstd))
    if st != 0:
        raise GemmError(st, "gemm_rms_norm")
    return Y, scale, H


def rms_norm(X, W=None, residual=None, eps=1e-6, Y=None, H=None, rstd=None):
    """Y = bf16(h * rstd * W) per row of a bfloat16 [rows, cols] tensor, with
    h = bf16(X + residual) (h = X without a residual) and
    rstd = 1 / sqrt(mean(h^2) + eps) (gemm_rms_norm).  W: a bfloat16 vector
    of cols elements or None (ones).  Returns Y, or (Y, H) with a residual:
    H, the sum, may be X or residual itself.  rstd: a float32 vector of rows
    elements to be filled for rms_norm_backward."""
    Y, _, H = _rms_norm("rms_norm", X, W, residual, eps, Y, H, rstd, False, None)
    return Y if residual is None else (Y, H)


def rms_norm_e4m3(X, W=None, residual=None, eps=1e-6, Q=None, scale=None, H=None, rstd=None):
    """The rows of rms_norm as E4M3FN codes (uint8 [rows, cols]) with
    float32 factors scale[rows]: those of gemm_fp8_quantize_rows on rms_norm's
    bf16 output, and the first operand of gemm_fp8_nt.  Returns (Q, scale),
    or (Q, scale, H) with a residual."""
    Q, scale, H = _rms_norm("rms_norm_e4m3", X, W, residual, eps, Q, H, rstd, True, scale)
    return (Q, scale) if residual is None else (Q, scale, H)


def rms_norm_backward(dY, H, W, rstd, dH=None, dX=None, dW=None, need_dw=True, workspace=None):
    """The gradient of rms_norm (gemm_rms_norm_backward): from dY [rows, cols]
    (bfloat16), H what was normed, W and the forward call's rstd, and dH the
    gradient that reaches H from the residual stream (or None), returns
    (dX bfloat16 [rows, cols], dW float32 [cols]; None without need_dw).
    dX is the gradient of X and of the residual.  workspace: as for the
    products (one is created for the call when None is given)."""
    if dY.dtype != torch.bfloat16 or dY.dim() != 2:
        raise TypeError("rms_norm_backward takes a 2-D bfloat16 dY")
    rows, cols = dY.shape
    _rows(H, (rows, cols), torch.bfloat16, "H")
    _rows(dH, (rows, cols), torch.bfloat16, "dH")
    _vector(W, cols, torch.bfloat16, "W")
    if rstd is None:
        raise ValueError("rstd: the vector the forward call filled")
    _vector(rstd, rows, torch.float32, "rstd")
    dev = _check_dev(dY, H, W, rstd, dH, dX, dW)
    if dX is None:
        dX = _like(dY, torch.bfloat16)
    _rows(dX, (rows, cols), torch.bfloat16, "dX")
    buf = None
    if need_dw:
        if dW is None:
            dW = torch.empty((cols,), dtype=torch.float32, device=dev)
        _vector(dW, cols, torch.float32, "dW")
        buf = _scratch(workspace, dev, _need(workspace, "gemm_rms_norm_workspace_size", rows, cols))
    else:
        dW = None
    st = _launch(lib().gemm_rms_norm_backward, dev, rows, cols, dY.data_ptr(), _stride(dY, cols), H.data_ptr(),
                 _stride(H, cols), _ptr(W), rstd.data_ptr(), _ptr(dH), cols if dH is None else _stride(dH, cols),
                 dX.data_ptr(), _stride(dX, cols), _ptr(dW), _ptr(buf), 0 if buf is None else buf.numel())
    if st != 0:
        raise GemmError(st, "gemm_rms_norm_backward")
    return dX, dW


def moe_swiglu(X, logits, topk, Wgu, Wd, scale_gu=None, scale_d=None, renormalize=True, Y=None,
               out_dtype=torch.bfloat16, ids=None, gates=None, workspace=None):
    """A mixture-of-experts SwiGLU layer for up to 64 tokens, behind the
    router's product (gemm_moe_swiglu): X [T, H] bfloat16, logits [T, E]
    float32, Wgu [E, 2I, H] (gate rows, then up rows) and Wd [E, H, I] in
    bfloat16, or as E4M3FN codes with float32 factors scale_gu [E, 2I] and
    scale_d [E, H].  Each token's topk experts (ties to the lowest index; -inf
    and NaN never) are weighted by the softmax of their logits, over the
    chosen ones (renormalize) or over all.  Returns (Y [T, H] in out_dtype,
    ids int32 [T, topk], gates float32 [T, topk])."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or logits.dtype != torch.float32 or logits.dim() != 2:
        raise TypeError("moe_swiglu takes a 2-D bfloat16 X and 2-D float32 logits")
    if Wgu.dim() != 3 or Wd.dim() != 3:
        raise ValueError("Wgu must be [E, 2I, H] and Wd [E, H, I]")
    coded = Wgu.dtype != torch.bfloat16
    if coded:
        Wgu, Wd = _codes(Wgu), _codes(Wd)
    elif Wd.dtype != torch.bfloat16:
        raise TypeError("Wgu and Wd must both be bfloat16 or both codes")
    T, H = X.shape
    E, I2, H2 = Wgu.shape
    I = I2 // 2
    topk = int(topk)
    if I2 % 2 or H2 != H or tuple(Wd.shape) != (E, H, I) or tuple(logits.shape) != (T, E):
        raise ValueError("expected X [T, H], logits [T, E], Wgu [E, 2I, H] and Wd [E, H, I]")
    if not coded and (scale_gu is not None or scale_d is not None):
        raise ValueError("factors belong to E4M3FN weights")
    for s, shape, name in ((scale_gu, (E, I2), "scale_gu"), (scale_d, (E, H), "scale_d")):
        if s is not None and (s.dtype != torch.float32 or tuple(s.shape) != shape or not s.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32 {list(shape)}")
    dev = _check_dev(X, logits, Wgu, Wd, scale_gu, scale_d, Y, ids, gates)
    need = _need(workspace, "gemm_moe_workspace_size", T, H, I, E, topk)
    if Y is None:
        Y = torch.empty((T, H), dtype=out_dtype, device=dev)
    if ids is None:
        ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, topk), dtype=torch.float32, device=dev)
    if tuple(Y.shape) != (T, H):
        raise ValueError("Y must be [T, H]")
    for t, dt, name in ((ids, torch.int32, "ids"), (gates, torch.float32, "gates")):
        if tuple(t.shape) != (T, topk) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dt} [T, topk]")
    buf = _scratch(workspace, dev, need)
    st = _launch(lib().gemm_moe_swiglu, dev, T, H, I, E, topk, 1 if renormalize else 0, X.data_ptr(), _stride(X, H),
                 logits.data_ptr(), _stride(logits, E), _lib.GEMM_OUT_E4M3 if coded else _lib.GEMM_OUT_BF16,
                 Wgu.data_ptr(), _stride(Wgu, H), _bstride(Wgu), _ptr(scale_gu), Wd.data_ptr(), _stride(Wd, I), _bstride(Wd),
                 _ptr(scale_d), Y.data_ptr(), _stride(Y, H), _out_code(Y.dtype), ids.data_ptr(), gates.data_ptr(),
                 _ptr(buf), 0 if buf is None else buf.numel())
    if st != 0:
        raise GemmError(st, "gemm_moe_swiglu")
    return Y, ids, gates


def gemm_bf16_nt_lora(X, Wt, A, B, idx, scale=None, C=None, out_dtype=torch.bfloat16, workspace=None):
    """C[m] = X[m] . Wt^T + scale[a] * (X[m] . A[a]^T) . B[a]^T with
    a = idx[m] (gemm_bf16_nt_lora): a projection Wt [N, K] shared by the rows
    of X [M, K], and low-rank adapters A [L, R, K], B [L, N, R] (bfloat16),
    scale float32 [L] or None (1).  idx: int32 [M]; rows whose index is not
    in [0, L) (e.g. -1) have no adapter."""
    if any(t.dtype != torch.bfloat16 for t in (X, Wt, A, B)) or idx.dtype != torch.int32:
        raise TypeError("gemm_bf16_nt_lora takes bfloat16 operands and an int32 idx")
    if X.dim() != 2 or Wt.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("expected X [M, K], Wt [N, K], A [L, R, K] and B [L, N, R]")
    M, K = X.shape
    N, K2 = Wt.shape
    L, R, K3 = A.shape
    if K2 != K or K3 != K or tuple(B.shape) != (L, N, R):
        raise ValueError("expected X [M, K], Wt [N, K], A [L, R, K] and B [L, N, R]")
    _vector(idx, M, torch.int32, "idx")
    _vector(scale, L, torch.float32, "scale")
    dev = _check_dev(X, Wt, A, B, idx, scale, C)
    if C is None:
        C = torch.empty((M, N), dtype=out_dtype, device=dev)
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be [M, N]")
    code = _out_code(C.dtype)
    ldx, ldw, ldc = _stride(X, K), _stride(Wt, K), _stride(C, N)
    px, pw, pc = X.data_ptr(), Wt.data_ptr(), C.data_ptr()
    if workspace is None:
        workspace = Workspace(dev)
    # the size depends on the pointers only through their alignment
    key = ("lora", M, N, K, L, R, px % 256, ldx, pw % 256, ldw, pc % 256, ldc, code)
    held = workspace._need if isinstance(workspace, Workspace) else {}

    def size():
        n = ctypes.c_uint64(0)
        st = lib().gemm_lora_workspace_size(M, N, K, L, R, px, ldx, pw, ldw, pc, ldc, code, ctypes.byref(n))
        if st != 0:
            raise GemmError(st, "gemm_bf16_nt_lora")
        held[key] = n.value
        return n.value

    def run(buf):
        return _launch(lib().gemm_bf16_nt_lora, dev, M, N, K, px, ldx, pw, ldw, L, R, A.data_ptr(), _stride(A, K),
                       _bstride(A), B.data_ptr(), _stride(B, R), _bstride(B), _ptr(scale), idx.data_ptr(), pc, ldc, code,
                       buf.data_ptr(), buf.numel())

    need = held.get(key)
    st = run(_scratch(workspace, dev, size() if need is None else need))
    if st == GEMM_ERR_WORKSPACE and need is not None:
        # the kept size went stale (the plan also follows the library's
        # environment overrides): nothing was launched, so ask again
        st = run(_scratch(workspace, dev, size()))
    if st != 0:
        raise GemmError(st, "gemm_bf16_nt_lora")
    return C
