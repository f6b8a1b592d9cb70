"""Binding of the gate and the adapters (include/dg.h): dg_moe_route,
dg_moe_route_backward, dg_lora_bf16, and moe_route, the gate as a differentiable torch
function.  As in binding.py: argument checks and marshalling, no arithmetic, no fallback.
The calls and the checks of their usual arguments go through _marshal (csrc/dg_marshal.cpp).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import _IN_DTYPES, DGError, load_library

DG_SCORE_SOFTMAX, DG_SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": DG_SCORE_SOFTMAX, "sigmoid": DG_SCORE_SIGMOID}
_workspaces: dict = {}
_native = None


def _load_native():
    """_marshal, with libdg (raises if either was not built)."""
    global _native
    if _native is None:
        load_library()
        try:
            from . import _marshal
        except ImportError as e:
            raise RuntimeError("_marshal.so is missing or does not load: build it with "
                               "`python -m moe_grouped_gemm_lhs_amd.build`") from e
        _marshal.use_slow(_vector, _rows)
        _native = _marshal
    return _native


def dg_moe_route_workspace_bytes(T: int, E: int) -> int:
    return (_native or _load_native()).dg_moe_route_workspace_bytes(T, E)


def dg_lora_workspace_bytes(T: int, N: int, K: int, R: int, L: int) -> int:
    return (_native or _load_native()).dg_lora_workspace_bytes(T, N, K, R, L)


# ------------------------------------------------------------------------ marshalling
# What _marshal's vector() and rows() hand on: arguments that are not the usual ones.
def _vector(t, name, dtype, shape, device):
    """Pointer of an optional dense argument (None: a null pointer)."""
    binding._check(t, name, dtype, shape, device)
    return t.data_ptr()


def _rows(t, name, dtype, shape, device):
    """Pointer and row stride of a matrix whose rows are dense but may lie apart."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        ld, one = t.stride()
        if shape[0] == 0 or shape[1] <= 1 or one == 1:
            # of no or one row the row stride says nothing
            return t.data_ptr(), ld if shape[0] > 1 else shape[1]
        raise ValueError(f"{name} must have dense rows, got strides {(ld, one)}")
    binding._check(t, name, dtype, shape, device)
    raise ValueError(f"{name}: not a matrix this call takes")


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.device


def _workspace(need, device, workspace, raw):
    """The caller's workspace, or one kept per (device, launch stream) and grown as needed,
    whatever it holds: the tensor (kept by the caller until the launch), its pointer and
    size.  Threads on one stream share it (the calls keep their launches together).  Under
    graph capture each call gets one from the graph's memory."""
    if need == 0:
        return None, None, 0
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    key = (device, raw)
    kept = _workspaces.get(key)
    capturing = torch.cuda.is_current_stream_capturing()
    if kept is not None and kept[2] >= need and not capturing:
        return kept
    ws = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
    kept = ws, ws.data_ptr(), ws.numel()
    if not capturing:
        # a smaller one was used on this stream only, so the allocator may hand its memory out
        # again in this stream's order
        with binding._lock:
            _workspaces[key] = kept
    return kept


def _unknown(score):
    return ValueError(f"unknown score function {score!r} (softmax or sigmoid)")


def _logits(logits):
    """Device, its index, dtype and the dtype's code."""
    dtype = logits.dtype
    code = _IN_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D (T x E)")
    dev = _device(logits, "logits")
    return dev, dev.index, dtype, code


# ------------------------------------------------------------------------------- gate
def dg_moe_route(logits, k, *, bias=None, row_valid=None, score="softmax", normalize=False,
                 scale=1.0, balance=None, count=False, ids=None, weights=None, counts=None,
                 loss=None, coef=None, workspace=None, stream=None):
    """The gate of a mixture of experts: the k experts of each row of logits (T x E, float32
    or bfloat16, rows may lie apart), their weights and what training needs.

    bias (E float32) is added to the logits, not to the scores, for the choice only (-inf
    closes an expert);
    row_valid (T uint8 or bool) marks padding rows with 0; score is "softmax" or "sigmoid";
    normalize divides a row's weights by the sum of its chosen scores; scale multiplies
    them.  balance: the factor of the balance loss (None: no loss).

    Returns (ids T x k int32, weights T x k float32, counts E int32 or None, loss float32
    scalar or None, coef E float32 or None): counts with count=True, a counts tensor or a
    balance; loss and coef with a balance.  ids, weights, counts, loss, coef may be given
    to be written in place.  include/dg.h has the formulas.

    Nothing that is returned carries a gradient, also where logits does: moe_route is the
    differentiable form."""
    native = _native or _load_native()
    dev, index, dtype, code = _logits(logits)
    if stream is not None or index != torch._C._cuda_getDevice():
        with binding._elsewhere(dev, stream):
            return dg_moe_route(logits, k, bias=bias, row_valid=row_valid, score=score,
                                normalize=normalize, scale=scale, balance=balance, count=count,
                                ids=ids, weights=weights, counts=counts, loss=loss, coef=coef,
                                workspace=workspace)
    T, E = logits.shape
    sc = _SCORES.get(score)
    if sc is None:
        raise _unknown(score)
    p_logits, ld = native.rows(logits, "logits", dtype, (T, E), dev)
    p_bias = native.vector(bias, "bias", torch.float32, (E,), dev)
    if row_valid is not None and row_valid.dtype is torch.bool:
        row_valid = row_valid.view(torch.uint8)
    p_valid = native.vector(row_valid, "row_valid", torch.uint8, (T,), dev)
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    if balance is not None:
        if loss is None:
            loss = torch.empty((), dtype=torch.float32, device=dev)
        if coef is None:
            coef = torch.empty((E,), dtype=torch.float32, device=dev)
    elif loss is not None or coef is not None:
        raise ValueError("loss and coef need a balance")
    if counts is None and (count or balance is not None):
        counts = torch.empty((E,), dtype=torch.int32, device=dev)
    p_ids = native.vector(ids, "ids", torch.int32, (T, k), dev)
    p_weights = native.vector(weights, "weights", torch.float32, (T, k), dev)
    p_counts = native.vector(counts, "counts", torch.int32, (E,), dev)
    p_loss = native.vector(loss, "loss", torch.float32, (), dev)
    p_coef = native.vector(coef, "coef", torch.float32, (E,), dev)
    raw = torch._C._cuda_getCurrentRawStream(index)
    ws, p_ws, ws_bytes = None, None, 0
    if counts is not None:
        ws, p_ws, ws_bytes = _workspace(native.dg_moe_route_workspace_bytes(T, E), dev, workspace, raw)
    st = native.dg_moe_route(p_logits, code, ld, p_bias, p_valid, T, E, k, sc, bool(normalize), scale,
                             balance or 0.0, p_ids, p_weights, p_counts, p_loss, p_coef, p_ws,
                             ws_bytes, raw)
    if st != 0:
        raise DGError(st, "dg_moe_route")
    return ids, weights, counts, loss, coef


def dg_moe_route_backward(logits, ids, *, grad_weights=None, coef=None, grad_loss=None,
                          row_valid=None, score="softmax", normalize=False, scale=1.0,
                          grad_logits=None, stream=None):
    """Gradient of dg_moe_route by its logits (same shape and dtype), from the gradients of
    its weights (T x k float32 or None) and of its loss (coef as returned by the forward
    call, grad_loss a float32 scalar; None: 1).  ids, row_valid, score, normalize and scale
    as in the forward call."""
    native = _native or _load_native()
    dev, index, dtype, code = _logits(logits)
    if stream is not None or index != torch._C._cuda_getDevice():
        with binding._elsewhere(dev, stream):
            return dg_moe_route_backward(logits, ids, grad_weights=grad_weights, coef=coef,
                                         grad_loss=grad_loss, row_valid=row_valid, score=score,
                                         normalize=normalize, scale=scale, grad_logits=grad_logits)
    T, E = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D (T x k)")
    k = ids.shape[1]
    sc = _SCORES.get(score)
    if sc is None:
        raise _unknown(score)
    p_logits, ld = native.rows(logits, "logits", dtype, (T, E), dev)
    if row_valid is not None and row_valid.dtype is torch.bool:
        row_valid = row_valid.view(torch.uint8)
    p_valid = native.vector(row_valid, "row_valid", torch.uint8, (T,), dev)
    p_ids = native.vector(ids, "ids", torch.int32, (T, k), dev)
    p_gw = native.vector(grad_weights, "grad_weights", torch.float32, (T, k), dev)
    p_coef = native.vector(coef, "coef", torch.float32, (E,), dev)
    p_gl = native.vector(grad_loss, "grad_loss", torch.float32, (), dev)
    if grad_logits is None:
        grad_logits = torch.empty((T, E), dtype=dtype, device=dev)
    p_out, ld_out = native.rows(grad_logits, "grad_logits", dtype, (T, E), dev)
    st = native.dg_moe_route_backward(
        p_logits, code, ld, p_valid, T, E, k, sc, bool(normalize), scale, p_ids,
        p_gw, p_coef, p_gl, p_out, ld_out, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise DGError(st, "dg_moe_route_backward")
    return grad_logits


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, row_valid, score, normalize, scale, balance):
        ids, weights, counts, loss, coef = dg_moe_route(
            logits, k, bias=bias, row_valid=row_valid, score=score, normalize=normalize, scale=scale,
            balance=balance, count=True)
        ctx.save_for_backward(logits, ids, coef, row_valid)
        ctx.how = dict(score=score, normalize=normalize, scale=scale)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(ids, counts)
        return ids, weights, counts, loss

    @staticmethod
    @once_differentiable
    def backward(ctx, _ids, grad_weights, _counts, grad_loss):
        logits, ids, coef, row_valid = ctx.saved_tensors
        if grad_weights is None and grad_loss is None:
            return (None,) * 8
        grad = dg_moe_route_backward(
            logits, ids, grad_weights=None if grad_weights is None else grad_weights.contiguous(),
            coef=None if grad_loss is None else coef, grad_loss=grad_loss, row_valid=row_valid,
            **ctx.how)
        return (grad,) + (None,) * 7


def moe_route(logits, k, *, bias=None, row_valid=None, score="softmax", normalize=False, scale=1.0,
              balance=None):
    """dg_moe_route for training: (ids, weights, counts, loss), weights and loss
    differentiable by logits once (loss None without a balance)."""
    return _Route.apply(logits, k, bias, row_valid, score, normalize, scale, balance)


# --------------------------------------------------------------------------- adapters
def dg_lora_bf16(X, A, B, ids, base=None, out=None, *, scales=None, ranks=None, workspace=None,
                 stream=None):
    """Low-rank adapters of many requests beside a shared projection:
    out[t] = base[t] + scales[i] (X[t] A[i]^T) B[i]^T with i = ids[t] (outside [0, L): no
    adapter, out[t] = base[t]).

    X (T x K), base and out (T x N) are bfloat16 with rows that may lie apart; A (L x R x
    K) and B (L x N x R) bfloat16; ids (T) int32; scales (L) float32, None: 1; ranks (L)
    int32, None: all R.  base None: zero; out may be base itself.  Returns out, which carries
    no gradient whatever X, A, B or base do: there is no differentiable form."""
    native = _native or _load_native()
    dev = _device(X, "X")
    index = dev.index
    if stream is not None or index != torch._C._cuda_getDevice():
        with binding._elsewhere(dev, stream):
            return dg_lora_bf16(X, A, B, ids, base, out, scales=scales, ranks=ranks,
                                workspace=workspace)
    if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("X must be 2-D (T x K), A (L x R x K) and B (L x N x R) 3-D")
    T, K = X.shape
    L, R, _ = A.shape
    N = B.shape[1]
    bf16 = torch.bfloat16
    p_x, ldx = native.rows(X, "X", bf16, (T, K), dev)
    p_a = native.vector(A, "A", bf16, (L, R, K), dev)
    p_b = native.vector(B, "B", bf16, (L, N, R), dev)
    p_ids = native.vector(ids, "ids", torch.int32, (T,), dev)
    p_s = native.vector(scales, "scales", torch.float32, (L,), dev)
    p_r = native.vector(ranks, "ranks", torch.int32, (L,), dev)
    p_base, ld_base = (None, 0) if base is None else native.rows(base, "base", bf16, (T, N), dev)
    if out is None:
        out = torch.empty((T, N), dtype=bf16, device=dev)
    p_out, ld_out = native.rows(out, "out", bf16, (T, N), dev)
    raw = torch._C._cuda_getCurrentRawStream(index)
    ws, p_ws, ws_bytes = _workspace(native.dg_lora_workspace_bytes(T, N, K, R, L), dev, workspace, raw)
    st = native.dg_lora_bf16(p_x, ldx, p_a, p_b, p_ids, p_s, p_r, p_base, ld_base, p_out, ld_out, T, N,
                          K, R, L, p_ws, ws_bytes, raw)
    if st != 0:
        raise DGError(st, "dg_lora_bf16")
    return out
