"""Binding of the feed-forward operators in 8 bits (include/dg.h): dg_rms_norm_fp8 and
dg_rms_norm_backward, the gated block's dg_gated_fp8_nt, dg_grouped_gated_fp8_contiguous,
dg_grouped_gated_fp8_masked and dg_gated_backward, the weight gradients dg_wgrad_fp8 and
dg_grouped_wgrad_fp8_contiguous, and gated_ffn, the whole block as a differentiable torch
function.  As in binding.py: argument checks and marshalling, no arithmetic, no fallback.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding, moe_ops
from .binding import (_FORMATS, _FP8_DTYPES, _FP8_OF, _IN_DTYPES, DG_CONTIGUOUS, DG_DENSE, DG_MASKED, DGError)
from .moe_ops import _device, _load_native

DG_ACT_SILU, DG_ACT_GELU = 0, 1
_ACTS = {"silu": DG_ACT_SILU, "gelu": DG_ACT_GELU}


def dg_rms_norm_backward_workspace_bytes(T: int, K: int) -> int:
    return _load_native().dg_rms_norm_backward_workspace_bytes(T, K)


def dg_gated_workspace_bytes(kind: int, rows_or_cap: int, N: int, K: int, G: int = 1) -> int:
    return _load_native().dg_gated_workspace_bytes(kind, rows_or_cap, N, K, G)


def dg_wgrad_workspace_bytes(T: int, N: int, K: int, G: int = 1) -> int:
    return _load_native().dg_wgrad_workspace_bytes(T, N, K, G)


# ------------------------------------------------------------------------ marshalling
def _away(dev, stream):
    """Whether a call has to be made in another context (binding._elsewhere)."""
    return stream is not None or dev.index != torch._C._cuda_getDevice()


def _code_of(t, name, fmt=None):
    """Format code of an operand: its float8 dtype's, or for uint8 bytes fmt's (None: E4M3)."""
    code = _FP8_DTYPES.get(t.dtype)
    if fmt is not None and fmt not in _FORMATS:
        raise ValueError(f"{name}: unknown operand format {fmt!r}")
    if code is None:
        if t.dtype is not torch.uint8:
            raise TypeError(f"{name} must be uint8, float8_e4m3fn or float8_e5m2, got {t.dtype}")
        return _FORMATS[fmt or "e4m3"]
    if fmt is not None and _FORMATS[fmt] != code:
        raise ValueError(f"{name}: format {fmt!r} contradicts dtype {t.dtype}")
    return code


def _format(fmt):
    if fmt not in _FORMATS:
        raise ValueError(f"unknown fp8 format {fmt!r}")
    return _FORMATS[fmt]


def _codes_out(t, name, fmt, shape, dev, zeros=False):
    """A matrix of codes to write, as a float8 tensor: the given one or a new one."""
    if t is None:
        make = torch.zeros if zeros else torch.empty
        return make(shape, dtype=torch.uint8, device=dev).view(_FP8_OF[fmt])
    _code_of(t, name, fmt)
    return t if t.dtype is not torch.uint8 else t.view(_FP8_OF[fmt])


def _scales_out(t, shape, dev, zeros=False):
    if t is not None:
        return t
    return (torch.zeros if zeros else torch.empty)(shape, dtype=torch.float32, device=dev)


def _act(activation):
    code = _ACTS.get(activation)
    if code is None:
        raise ValueError(f"unknown activation {activation!r} (silu or gelu)")
    return code


def _in_dtype(t, name):
    code = _IN_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _weight(native, weight, K, dev):
    """Pointer and dtype code of a norm's weight (None: ones)."""
    if weight is None:
        return None, 0
    code = _in_dtype(weight, "weight")
    return native.vector(weight, "weight", weight.dtype, (K,), dev), code


# ------------------------------------------------------------------------------- norm
def dg_rms_norm_fp8(X, weight=None, *, residual=None, eps=1e-6, fmt="e4m3", codes=True, bf16=False,
                    save=False, Q=None, S=None, H=None, Y=None, rstd=None, stream=None):
    """Root-mean-square norm of the rows of X (T x K, float32 or bfloat16, rows may lie apart)
    behind the residual's addition: h = X + residual, y = h / sqrt(mean h^2 + eps) * weight,
    out as fp8 codes with 1x128 scales, the A operand of the GEMM calls.

    residual: of X's shape and dtype; weight: K float32 or bfloat16 (None: ones).
    Returns (Q float8 T x K, S float32 T x K/128, H, Y bfloat16 T x K or None, rstd float32 T or
    None): codes=False leaves Q and S None; Y with bf16=True or a Y; rstd, for
    dg_rms_norm_backward, with save=True or an rstd.  H is X itself without a residual, else a
    new tensor or the given one, which may be X or residual.  Row strides are multiples of 8 and
    matrices start on 16 bytes.  Nothing that is returned carries a gradient."""
    native = moe_ops._native or _load_native()
    dev, dtype = X.device, X.dtype
    index = dev.index
    if stream is not None or index is None or index != torch._C._cuda_getDevice():
        with binding._elsewhere(_device(X, "X"), stream):
            return dg_rms_norm_fp8(X, weight, residual=residual, eps=eps, fmt=fmt, codes=codes, bf16=bf16,
                                   save=save, Q=Q, S=S, H=H, Y=Y, rstd=rstd)
    code = _IN_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"X must be float32 or bfloat16, got {dtype}")
    shape = X.shape
    if len(shape) != 2:
        raise ValueError("X must be 2-D (T x K)")
    T, K = shape
    p_x, ldx = native.rows(X, "X", dtype, shape, dev)
    p_w, w_code = (None, 0) if weight is None else _weight(native, weight, K, dev)
    fmt_code = _FORMATS.get(fmt)
    if fmt_code is None:
        raise ValueError(f"unknown fp8 format {fmt!r}")
    p_q = p_s = p_r = p_h = p_y = None
    ldr = ldh = ldy = 0
    if codes:
        fp8 = _FP8_OF[fmt]
        if Q is None or Q.dtype is not fp8:
            Q = _codes_out(Q, "Q", fmt, shape, dev)
        if S is None:
            S = torch.empty((T, K // 128), dtype=torch.float32, device=dev)
        p_q = native.vector(Q, "Q", fp8, shape, dev)
        p_s = native.vector(S, "S", torch.float32, (T, K // 128), dev)
    elif Q is not None or S is not None:
        raise ValueError("Q and S are written with codes=True")
    if residual is not None:
        p_r, ldr = native.rows(residual, "residual", dtype, shape, dev)
        if H is None:
            H = torch.empty(shape, dtype=dtype, device=dev)
        p_h, ldh = native.rows(H, "H", dtype, shape, dev)
    elif H is not None:
        raise ValueError("H is written with a residual")
    else:
        H = X
    if Y is None and bf16:
        Y = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if Y is not None:
        p_y, ldy = native.rows(Y, "Y", torch.bfloat16, shape, dev)
    if rstd is None and save:
        rstd = torch.empty((T,), dtype=torch.float32, device=dev)
    p_rstd = native.vector(rstd, "rstd", torch.float32, (T,), dev)
    st = native.dg_rms_norm_fp8(p_x, code, ldx, p_r, ldr, p_w, w_code, eps, p_h, ldh, p_q, p_s, fmt_code, p_y,
                                ldy, p_rstd, T, K, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise DGError(st, "dg_rms_norm_fp8")
    return Q, S, H, Y, rstd


def dg_rms_norm_backward(grad_y, H, rstd, weight=None, *, grad_h=None, grad_x=None, grad_weight=None,
                         workspace=None, stream=None):
    """Gradient of dg_rms_norm_fp8 from its H and rstd: grad_y (T x K), the gradient by the
    normalized output, and grad_h (None: none), the gradient that reaches H itself, give
    grad_x, the gradient by X and by the residual alike (all of H's dtype, rows may lie apart;
    grad_x may be grad_y, grad_h or H), and, with a weight, grad_weight (K float32).
    Returns (grad_x, grad_weight or None); a weight without a gradient: grad_weight=False."""
    native = moe_ops._native or _load_native()
    dev = _device(grad_y, "grad_y")
    if _away(dev, stream):
        with binding._elsewhere(dev, stream):
            return dg_rms_norm_backward(grad_y, H, rstd, weight, grad_h=grad_h, grad_x=grad_x,
                                        grad_weight=grad_weight, workspace=workspace)
    dtype, code = grad_y.dtype, _in_dtype(grad_y, "grad_y")
    if grad_y.dim() != 2:
        raise ValueError("grad_y must be 2-D (T x K)")
    shape = T, K = grad_y.shape
    p_y, ldy = native.rows(grad_y, "grad_y", dtype, shape, dev)
    p_h, ldh = native.rows(H, "H", dtype, shape, dev)
    p_rstd = native.vector(rstd, "rstd", torch.float32, (T,), dev)
    p_w, w_code = _weight(native, weight, K, dev)
    p_gh, ld_gh = (None, 0) if grad_h is None else native.rows(grad_h, "grad_h", dtype, shape, dev)
    if grad_x is None:
        grad_x = torch.empty(shape, dtype=dtype, device=dev)
    p_gx, ld_gx = native.rows(grad_x, "grad_x", dtype, shape, dev)
    if grad_weight is False:
        grad_weight = None
    elif grad_weight is None and weight is not None:
        grad_weight = torch.empty((K,), dtype=torch.float32, device=dev)
    p_gw = native.vector(grad_weight, "grad_weight", torch.float32, (K,), dev)
    raw = torch._C._cuda_getCurrentRawStream(dev.index)
    ws, p_ws, ws_bytes = None, None, 0
    if grad_weight is not None:
        ws, p_ws, ws_bytes = moe_ops._workspace(native.dg_rms_norm_backward_workspace_bytes(T, K), dev, workspace,
                                                raw)
    st = native.dg_rms_norm_backward(p_y, code, ldy, p_h, ldh, p_rstd, p_w, w_code, p_gh, ld_gh, p_gx, ld_gx,
                                     p_gw, T, K, p_ws, ws_bytes, raw)
    if st != 0:
        raise DGError(st, "dg_rms_norm_backward")
    return grad_x, grad_weight


# ------------------------------------------------------------------------ gated block
def _gated(call, kind, A, sA, B, sB, rows_of, H, sH, activation, a_format, b_format, fmt, save, GU, sGU,
           workspace, stream):
    native = moe_ops._native or _load_native()
    dev = _device(A, "A")
    if _away(dev, stream):
        with binding._elsewhere(dev, stream):
            return _gated(call, kind, A, sA, B, sB, rows_of, H, sH, activation, a_format, b_format, fmt, save, GU,
                          sGU, workspace, None)
    act, out = _act(activation), _format(fmt)
    fa, fb = _code_of(A, "A", a_format), _code_of(B, "B", b_format)
    masked = kind == DG_MASKED
    if A.dim() != (3 if masked else 2) or B.dim() != (2 if kind == DG_DENSE else 3):
        raise ValueError("A must be rows x K (masked: G x cap x K), B 2N x K (grouped: G x 2N x K)")
    lead, K = tuple(A.shape[:-1]), A.shape[-1]
    rows = lead[-1]
    G, N2 = 1 if kind == DG_DENSE else B.shape[0], B.shape[-2]
    if N2 % 256 != 0:
        raise ValueError(f"B must have 2N rows, N a multiple of 128, got {N2}")
    if masked and lead[0] != G:
        raise ValueError(f"A has {lead[0]} groups, B {G}")
    N, nkb, groups = N2 // 2, -(-K // 128), () if kind == DG_DENSE else (G,)
    p_a = native.vector(A, "A", A.dtype, (*lead, K), dev)
    p_sa = native.vector(sA, "sA", torch.float32, (*lead, nkb), dev)
    p_b = native.vector(B, "B", B.dtype, (*groups, N2, K), dev)
    p_sb = native.vector(sB, "sB", torch.float32, (*groups, N2 // 128, nkb), dev)
    p_rows = None
    if kind == DG_CONTIGUOUS:
        p_rows = native.vector(rows_of, "group_idx", torch.int32, lead, dev)
    elif masked:
        p_rows = native.vector(rows_of, "masked_m", torch.int32, (G,), dev)
    # rows that a grouped call leaves alone are zeros in what it allocates itself
    zeros = kind != DG_DENSE
    H = _codes_out(H, "H", fmt, (*lead, N), dev, zeros)
    sH = _scales_out(sH, (*lead, N // 128), dev, zeros)
    p_h = native.vector(H, "H", H.dtype, (*lead, N), dev)
    p_sh = native.vector(sH, "sH", torch.float32, (*lead, N // 128), dev)
    p_gu = p_sgu = None
    if save or GU is not None or sGU is not None:
        GU = _codes_out(GU, "GU", fmt, (*lead, N2), dev, zeros)
        sGU = _scales_out(sGU, (*lead, N2 // 128), dev, zeros)
        p_gu = native.vector(GU, "GU", GU.dtype, (*lead, N2), dev)
        p_sgu = native.vector(sGU, "sGU", torch.float32, (*lead, N2 // 128), dev)
    raw = torch._C._cuda_getCurrentRawStream(dev.index)
    ws, p_ws, ws_bytes = moe_ops._workspace(native.dg_gated_workspace_bytes(kind, rows, N, K, G), dev, workspace,
                                            raw)
    if kind == DG_DENSE:
        st = native.dg_gated_fp8_nt(p_a, fa, p_sa, p_b, fb, p_sb, p_h, p_sh, out, p_gu, p_sgu, act, rows, N, K,
                                    p_ws, ws_bytes, raw)
    elif masked:
        st = native.dg_grouped_gated_fp8_masked(p_a, fa, p_sa, p_b, fb, p_sb, p_rows, p_h, p_sh, out, act, G,
                                                rows, N, K, p_ws, ws_bytes, raw)
    else:
        st = native.dg_grouped_gated_fp8_contiguous(p_a, fa, p_sa, p_b, fb, p_sb, p_rows, p_h, p_sh, out, p_gu,
                                                    p_sgu, act, rows, N, K, G, p_ws, ws_bytes, raw)
    if st != 0:
        raise DGError(st, call)
    return H, sH, GU, sGU


def dg_gated_fp8_nt(A, sA, B, sB, H=None, sH=None, *, activation="silu", a_format=None, b_format=None,
                    fmt="e4m3", save=False, GU=None, sGU=None, workspace=None, stream=None):
    """The first half of a gated feed-forward block in one kernel: h = act(A Bg^T) * (A Bu^T) as
    fp8 codes with 1x128 scales.  A (M x K), sA as for dg_gemm_fp8_nt; B (2N x K): the gate's N
    rows, then the up matrix's, with sB (2N/128 x K/128); activation "silu" or "gelu" (tanh).

    Returns (H float8 M x N, sH float32 M x N/128, GU float8 M x 2N, sGU float32 M x 2N/128):
    with save=True (or a GU or sGU) GU and sGU hold both projections, the checkpoint for
    dg_gated_backward, else they are None.  fmt is the format of all codes that are written."""
    return _gated("dg_gated_fp8_nt", DG_DENSE, A, sA, B, sB, None, H, sH, activation, a_format, b_format, fmt,
                  save, GU, sGU, workspace, stream)


def dg_grouped_gated_fp8_contiguous(A, sA, B, sB, group_idx, H=None, sH=None, *, activation="silu",
                                    a_format=None, b_format=None, fmt="e4m3", save=False, GU=None, sGU=None,
                                    workspace=None, stream=None):
    """dg_gated_fp8_nt over the contiguous grouped form: A (M_total x K), B (G x 2N x K),
    group_idx (M_total int32) as for dg_grouped_gemm_fp8_contiguous.  Rows that belong to no
    group keep what the outputs held (zeros where the call allocates them)."""
    return _gated("dg_grouped_gated_fp8_contiguous", DG_CONTIGUOUS, A, sA, B, sB, group_idx, H, sH, activation,
                  a_format, b_format, fmt, save, GU, sGU, workspace, stream)


def dg_grouped_gated_fp8_masked(A, sA, B, sB, masked_m, H=None, sH=None, *, activation="silu", a_format=None,
                                b_format=None, fmt="e4m3", workspace=None, stream=None):
    """dg_gated_fp8_nt over the masked grouped form: A (G x cap x K), B (G x 2N x K), masked_m (G
    int32) as for dg_grouped_gemm_fp8_masked.  Returns (H G x cap x N, sH G x cap x N/128, None,
    None): a decode step keeps no checkpoint."""
    return _gated("dg_grouped_gated_fp8_masked", DG_MASKED, A, sA, B, sB, masked_m, H, sH, activation, a_format,
                  b_format, fmt, False, None, None, workspace, stream)


def dg_gated_backward(grad_H, GU, sGU, D=None, sD=None, *, group_idx=None, groups=None, activation="silu",
                      gu_format=None, fmt="e4m3", stream=None):
    """Gradient of the gated block's first half by both projections, from grad_H (T x N float32
    or bfloat16) and the checkpoint GU, sGU: D (T x 2N: by the gate, by up) as fp8 codes of fmt
    with scales sD (T x 2N/128), which may be GU and sGU.  With group_idx (T int32) and groups,
    their number, rows that the contiguous forward call leaves alone are left alone here (zeros
    where this call allocates).  Returns (D, sD)."""
    if group_idx is not None and groups is None:
        raise ValueError("group_idx needs groups, the number of them")
    native = moe_ops._native or _load_native()
    dev = _device(grad_H, "grad_H")
    if _away(dev, stream):
        with binding._elsewhere(dev, stream):
            return dg_gated_backward(grad_H, GU, sGU, D, sD, group_idx=group_idx, groups=groups,
                                     activation=activation, gu_format=gu_format, fmt=fmt)
    act, out, code = _act(activation), _format(fmt), _in_dtype(grad_H, "grad_H")
    if grad_H.dim() != 2:
        raise ValueError("grad_H must be 2-D (T x N)")
    T, N = grad_H.shape
    gu = _code_of(GU, "GU", gu_format)
    p_g = native.vector(grad_H, "grad_H", grad_H.dtype, (T, N), dev)
    p_gu = native.vector(GU, "GU", GU.dtype, (T, 2 * N), dev)
    p_sgu = native.vector(sGU, "sGU", torch.float32, (T, 2 * N // 128), dev)
    p_idx = native.vector(group_idx, "group_idx", torch.int32, (T,), dev)
    zeros = group_idx is not None
    D = _codes_out(D, "D", fmt, (T, 2 * N), dev, zeros)
    sD = _scales_out(sD, (T, 2 * N // 128), dev, zeros)
    p_d = native.vector(D, "D", D.dtype, (T, 2 * N), dev)
    p_sd = native.vector(sD, "sD", torch.float32, (T, 2 * N // 128), dev)
    st = native.dg_gated_backward(p_g, code, p_gu, gu, p_sgu, p_idx, act, p_d, p_sd, out, T, N,
                                  1 if groups is None else groups,
                                  torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        raise DGError(st, "dg_gated_backward")
    return D, sD


# ------------------------------------------------------------------- weights' gradients
def _wgrad(call, P, sP, Q, sQ, group_idx, G, dW, p_format, q_format, accumulate, dtype, workspace, stream):
    native = moe_ops._native or _load_native()
    dev = _device(P, "P")
    if _away(dev, stream):
        with binding._elsewhere(dev, stream):
            return _wgrad(call, P, sP, Q, sQ, group_idx, G, dW, p_format, q_format, accumulate, dtype, workspace,
                          None)
    fp, fq = _code_of(P, "P", p_format), _code_of(Q, "Q", q_format)
    if P.dim() != 2 or Q.dim() != 2:
        raise ValueError("P must be 2-D (T x N), Q 2-D (T x K)")
    (T, N), K = P.shape, Q.shape[1]
    grouped = G is not None
    shape = (G, N, K) if grouped else (N, K)
    p_p = native.vector(P, "P", P.dtype, (T, N), dev)
    p_sp = native.vector(sP, "sP", torch.float32, (T, N // 128), dev)
    p_q = native.vector(Q, "Q", Q.dtype, (T, K), dev)
    p_sq = native.vector(sQ, "sQ", torch.float32, (T, K // 128), dev)
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs a dW to add to")
        dW = torch.empty(shape, dtype=dtype or torch.float32, device=dev)
    elif dtype is not None and dtype is not dW.dtype:
        raise ValueError(f"dtype {dtype} contradicts dW's {dW.dtype}")
    code = _in_dtype(dW, "dW")
    p_w = native.vector(dW, "dW", dW.dtype, shape, dev)
    raw = torch._C._cuda_getCurrentRawStream(dev.index)
    ws, p_ws, ws_bytes = moe_ops._workspace(native.dg_wgrad_workspace_bytes(T, N, K, G or 1), dev, workspace, raw)
    if grouped:
        p_idx = native.vector(group_idx, "group_idx", torch.int32, (T,), dev)
        st = native.dg_grouped_wgrad_fp8_contiguous(p_p, fp, p_sp, p_q, fq, p_sq, p_idx, p_w, code,
                                                    bool(accumulate), T, N, K, G, p_ws, ws_bytes, raw)
    else:
        st = native.dg_wgrad_fp8(p_p, fp, p_sp, p_q, fq, p_sq, p_w, code, bool(accumulate), T, N, K, p_ws,
                                 ws_bytes, raw)
    if st != 0:
        raise DGError(st, call)
    return dW


def dg_wgrad_fp8(P, sP, Q, sQ, dW=None, *, p_format=None, q_format=None, accumulate=False, dtype=None,
                 workspace=None, stream=None):
    """A weight's gradient from two matrices of fp8 codes with 1x128 scales that lie row by row:
    dW (N x K) = sum over rows of (sP P)[t,n] (sQ Q)[t,k], P (T x N) such as a gradient's codes, Q
    (T x K) such as an activation's checkpoint.  dW is float32 or bfloat16 (dtype, float32 by
    default, or the given dW's); accumulate adds to it.  Returns dW."""
    return _wgrad("dg_wgrad_fp8", P, sP, Q, sQ, None, None, dW, p_format, q_format, accumulate, dtype, workspace,
                  stream)


def dg_grouped_wgrad_fp8_contiguous(P, sP, Q, sQ, group_idx, groups, dW=None, *, p_format=None, q_format=None,
                                    accumulate=False, dtype=None, workspace=None, stream=None):
    """dg_wgrad_fp8 for each group of the contiguous form: dW (groups x N x K), of group g the sum
    over the rows that group_idx (T int32) gives it.  Rows of no group count nowhere, whatever
    they hold; a group without rows has a gradient of zeros."""
    if groups is None:
        raise TypeError("groups must be a number")
    return _wgrad("dg_grouped_wgrad_fp8_contiguous", P, sP, Q, sQ, group_idx, groups, dW, p_format, q_format,
                  accumulate, dtype, workspace, stream)


# ------------------------------------------------------------------- the whole block
def _transposed(codes, scales):
    """A weight's codes and 128x128 scales the other way round."""
    return binding.dg_transpose_fp8(codes), scales.t().contiguous()


def _dense(grad):
    """A gradient as the calls take it; torch's may be broadcast, turned or a part of another."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, norm_weight, w13, w2, eps, activation):
        q, s, h, _, rstd = dg_rms_norm_fp8(x, norm_weight, residual=residual, eps=eps, save=True)
        b13, b2 = binding.dg_quantize_fp8_128x128(w13), binding.dg_quantize_fp8_128x128(w2)
        a, sa, gu, sgu = dg_gated_fp8_nt(q, s, *b13, activation=activation, save=True)
        out = binding.dg_gemm_fp8_nt(a, sa, *b2)
        ctx.save_for_backward(h, rstd, norm_weight, q, s, a, sa, gu, sgu, *b13, *b2)
        ctx.activation, ctx.has_residual = activation, residual is not None
        ctx.dtypes = w13.dtype, w2.dtype, None if norm_weight is None else norm_weight.dtype
        ctx.set_materialize_grads(False)
        return out, h if ctx.has_residual else None

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_h):
        h, rstd, norm_weight, q, s, a, sa, gu, sgu, b13, s13, b2, s2 = ctx.saved_tensors
        need = ctx.needs_input_grad
        if grad_out is None:
            return (grad_h, grad_h if ctx.has_residual else None) + (None,) * 5
        grad_h = None if grad_h is None else _dense(grad_h)
        d, sd = binding.dg_quantize_fp8_1x128(_dense(grad_out))
        da = binding.dg_gemm_fp8_nt(d, sd, *_transposed(b2, s2))
        dw2 = dg_wgrad_fp8(d, sd, a, sa, dtype=ctx.dtypes[1]) if need[4] else None
        d, sd = dg_gated_backward(da, gu, sgu, activation=ctx.activation)
        dw13 = dg_wgrad_fp8(d, sd, q, s, dtype=ctx.dtypes[0]) if need[3] else None
        dx = dw = None
        if need[0] or need[1] or need[2]:
            dy = binding.dg_gemm_fp8_nt(d, sd, *_transposed(b13, s13)).to(h.dtype)
            dx, dw = dg_rms_norm_backward(dy, h, rstd, norm_weight, grad_h=grad_h,
                                          grad_weight=None if need[2] else False)
        return (dx, dx if ctx.has_residual else None, None if dw is None else dw.to(ctx.dtypes[2]), dw13, dw2,
                None, None)


def gated_ffn(x, w13, w2, *, residual=None, norm_weight=None, eps=1e-6, activation="silu"):
    """A feed-forward block for training, in 8 bits: norm(x + residual), both projections with w13
    (2N x K: gate, up), the activation and the product, and the down projection with w2 (M x N).
    x and residual T x K, the weights, all float32 or bfloat16, are quantised here; what is
    kept for the backward pass is the stream x + residual and codes.

    Between the calls of the backward pass gradients are bfloat16 and E4M3 codes, an fp32 stream's
    as well: where gradients span more than E4M3's range within 128 columns, the calls themselves
    take E5M2 ones.

    Returns (out T x M bfloat16, x + residual or None without a residual), differentiable once
    by x, residual, norm_weight, w13 and w2; the backward pass takes M of a multiple of 128.  A
    step may be captured in a graph, if no graph of autograd's that was built outside the capture
    on the same leaves is alive then."""
    return _GatedFFN.apply(x, residual, norm_weight, w13, w2, eps, activation)
