"""Tensor entry points of the operators around the products.

    quantize_fp4_*(w), gemv_fp4_*(x, W, sW)         4-bit weights and a product of a few rows with them
    rmsnorm_*(x, weight, residual), rmsnorm_fp8_*   the norm before a product, its output in 16 or 8 bits
    rmsnorm_grad_*(dy, h, weight, rstd)             its gradients
    route_topk_*(logits, k), route_topk_grad_*      the experts of each token, their weights, and the logits' gradient
    route_sort(ids, E)                              where each expert's rows begin, and the row of each token's choice
    route_gather_*(X, pos), route_combine_*(D, pos, weights), route_combine_grad_*
                                                    rows to the experts and back

A mixture of experts is route_topk, route_sort, route_gather, gemm_grouped and route_combine, with no synchronisation
between them; backwards it is route_combine_grad, gemm_grouped_dgrad and _wgrad, route_combine without weights (the
gradient of route_gather) and route_topk_grad.  Like the rest of the package this only marshals arguments
(include/gemvtile.h states each call's contract); names end in the 16-bit format of the inputs (or f32 for logits).
"""
from __future__ import annotations

import torch
from torch import Tensor
from torch._C import _cuda_getCurrentRawStream as _raw_stream
from torch._C import _cuda_getDevice as _current_device

from . import LAYER_CALLS, _check, load_library
from .blocks import FP8, _blocks, _first, _output, _shaped

__all__ = list(LAYER_CALLS) + ["alloc_rmsnorm_grad_workspace", "alloc_route_sort_workspace"]

SCORES = {"softmax": 0, "sigmoid": 1}


def _run(dev, stream, call, *args):
    s = _raw_stream(dev) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    if _current_device() == dev:
        status = call(*args, s)
    else:
        with torch.cuda.device(dev):
            status = call(*args, s)
    if status:
        _check(status)


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def _optional(t, name, dtype, shape, dev):
    """The address of a tensor that may be None."""
    if t is None:
        return None
    _shaped(t, name, dtype, shape, dev)
    return t.data_ptr()


def _workspace(t, dev):
    if t is None:
        return None, 0
    if not (isinstance(t, Tensor) and t.is_cuda and t.is_contiguous()):
        raise TypeError("workspace must be a contiguous device tensor")
    if t.get_device() != dev:
        raise ValueError(f"workspace must be on device {dev}, got {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


# ---- 4-bit weights -------------------------------------------------------------
def _quantize_fp4(x, q, scale, stream, dtype, call):
    dev = _first(x, "x", dtype, 3 if isinstance(x, Tensor) and x.dim() == 3 else 2)
    *lead, N, K = x.shape
    if K % 32 != 0:
        raise ValueError(f"K must be a multiple of 32, got {K}")
    q = _output(q, "q", torch.uint8, (*lead, N, K // 2), dev)
    scale = _output(scale, "scale", torch.uint8, (*lead, N, K // 32), dev)
    _run(dev, stream, call, x.data_ptr(), q.data_ptr(), scale.data_ptr(), (lead[0] if lead else 1) * N, K)
    return q, scale


def quantize_fp4_f16(x, q=None, scale=None, stream=None):
    """(q, scale) of a weight x [N,K], or of each of x [E,N,K], fp16: q [..,N,K/2] uint8 with two e2m1 numbers a byte
    (the even column in the low half) and scale [..,N,K/32] uint8, byte s of 32 columns standing for 2^(s - 127): the
    least with which no number is beyond 6.  K % 32 == 0.  gemv_fp4_* takes one matrix at a time (q[e], scale[e]).
    Enqueued on `stream` (default: the current stream), not synchronised."""
    return _quantize_fp4(x, q, scale, stream, torch.float16, load_library().quantize_fp4_f16)


def quantize_fp4_bf16(x, q=None, scale=None, stream=None):
    """quantize_fp4_f16 of a bfloat16 tensor."""
    return _quantize_fp4(x, q, scale, stream, torch.bfloat16, load_library().quantize_fp4_bf16)


def _gemv_fp4(x, W, scale_W, y, stream, dtype, call):
    one = isinstance(x, Tensor) and x.dim() == 1
    dev = _first(x, "x", dtype, 1 if one else 2)
    if _first(W, "W", torch.uint8, 2) != dev:
        raise ValueError(f"W must be on device {dev}, got {W.device}")
    K = x.shape[-1]
    M = 1 if one else x.shape[0]
    N = W.shape[0]
    if 2 * W.shape[1] != K:
        raise ValueError(f"K mismatch: x is {tuple(x.shape)}, W (two numbers a byte) is {tuple(W.shape)}")
    if K % 32 != 0:
        raise ValueError(f"K must be a multiple of 32, got {K}")
    _shaped(scale_W, "scale_W", torch.uint8, (N, K // 32), dev)
    y = _output(y, "y", dtype, (N,) if one else (M, N), dev)
    _run(dev, stream, call, x.data_ptr(), W.data_ptr(), scale_W.data_ptr(), y.data_ptr(), M, N, K)
    return y


def gemv_fp4_f16(x, W, scale_W, y=None, stream=None):
    """y = x · (W scaled)ᵀ for one row x [K] or a decode batch x [M,K], fp16, rounded once: W [N,K/2] and scale_W
    [N,K/32] uint8 as quantize_fp4_f16 gives them, y [N] or [M,N].  Up to 48 rows share a read of W; a prompt's hundreds
    of rows are faster by gemm_f16 on 16-bit weights."""
    return _gemv_fp4(x, W, scale_W, y, stream, torch.float16, load_library().gemv_fp4_f16)


def gemv_fp4_bf16(x, W, scale_W, y=None, stream=None):
    """gemv_fp4_f16 with bfloat16 rows."""
    return _gemv_fp4(x, W, scale_W, y, stream, torch.bfloat16, load_library().gemv_fp4_bf16)


# ---- norm ----------------------------------------------------------------------
def _norm_inputs(x, weight, residual, h, rstd, dtype):
    dev = _first(x, "x", dtype, 2)
    T, C = x.shape
    _shaped(weight, "weight", dtype, (C,), dev)
    r = _optional(residual, "residual", dtype, (T, C), dev)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual (without one it is x)")
        h = x
        hp = None
    else:
        h = _output(h, "h", dtype, (T, C), dev)
        hp = h.data_ptr()
    return dev, T, C, r, h, hp, _optional(rstd, "rstd", torch.float32, (T,), dev)


def _rmsnorm(x, weight, residual, eps, h, y, rstd, stream, dtype, call):
    dev, T, C, r, h, hp, sp = _norm_inputs(x, weight, residual, h, rstd, dtype)
    y = _output(y, "y", dtype, (T, C), dev)
    _run(dev, stream, call, x.data_ptr(), r, weight.data_ptr(), hp, y.data_ptr(), sp, T, C, eps)
    return y, h


def rmsnorm_f16(x, weight, residual=None, eps=1e-6, h=None, y=None, rstd=None, stream=None):
    """(y, h): h = x + residual rounded to fp16 (x itself without a residual), y = h / sqrt(mean(h²) + eps) · weight.
    x, residual, h, y [T,C], weight [C] fp16; C % 8 == 0, C <= 32768.  h may be x or residual; rstd [T] FP32 takes
    1 / sqrt(mean(h²) + eps) for rmsnorm_grad_f16; eps, the sum and the root are FP64.  Enqueued on `stream`, not synchronised."""
    return _rmsnorm(x, weight, residual, eps, h, y, rstd, stream, torch.float16, load_library().rmsnorm_f16)


def rmsnorm_bf16(x, weight, residual=None, eps=1e-6, h=None, y=None, rstd=None, stream=None):
    """rmsnorm_f16 on bfloat16 tensors."""
    return _rmsnorm(x, weight, residual, eps, h, y, rstd, stream, torch.bfloat16, load_library().rmsnorm_bf16)


def _rmsnorm_fp8(x, weight, residual, eps, h, q, scale, y, rstd, stream, dtype, call):
    dev, T, C, r, h, hp, sp = _norm_inputs(x, weight, residual, h, rstd, dtype)
    q = _output(q, "q", FP8, (T, C), dev)
    scale = _output(scale, "scale", torch.float32, (T, _blocks(C)), dev)
    yp = _optional(y, "y", dtype, (T, C), dev)
    _run(dev, stream, call, x.data_ptr(), r, weight.data_ptr(), hp, yp, q.data_ptr(), scale.data_ptr(), sp, T, C, eps)
    return q, scale, h


def rmsnorm_fp8_f16(x, weight, residual=None, eps=1e-6, h=None, q=None, scale=None, y=None, rstd=None, stream=None):
    """(q, scale, h): rmsnorm_f16 whose y leaves as q [T,C] float8_e4m3fn and scale [T, ceil(C/128)] FP32, the operands
    of gemm_fp8_* and gemm_grouped_fp8_*; C % 16 == 0.  y [T,C] is written too if it is given (a router's logits are
    made of it)."""
    return _rmsnorm_fp8(x, weight, residual, eps, h, q, scale, y, rstd, stream, torch.float16,
                        load_library().rmsnorm_fp8_f16)


def rmsnorm_fp8_bf16(x, weight, residual=None, eps=1e-6, h=None, q=None, scale=None, y=None, rstd=None, stream=None):
    """rmsnorm_fp8_f16 on bfloat16 tensors."""
    return _rmsnorm_fp8(x, weight, residual, eps, h, q, scale, y, rstd, stream, torch.bfloat16,
                        load_library().rmsnorm_fp8_bf16)


def alloc_rmsnorm_grad_workspace(h):
    """A uint8 tensor on h's device that is large enough a workspace for the gradient of a norm of h [T,C]."""
    T, C = h.shape
    need = int(load_library().gemvtile_rmsnorm_grad_workspace(T, C))
    return torch.empty((max(need, 16),), dtype=torch.uint8, device=h.device)


def _rmsnorm_grad(dy, h, weight, rstd, dh, dx, dweight, workspace, stream, dtype, call):
    dev = _first(h, "h", dtype, 2)
    T, C = h.shape
    _shaped(dy, "dy", dtype, (T, C), dev)
    _shaped(weight, "weight", dtype, (C,), dev)
    _shaped(rstd, "rstd", torch.float32, (T,), dev)
    ep = _optional(dh, "dh", dtype, (T, C), dev)
    dx = _output(dx, "dx", dtype, (T, C), dev)
    dweight = _output(dweight, "dweight", torch.float32, (C,), dev)
    wp, wb = _workspace(workspace, dev)
    _run(dev, stream, call, dy.data_ptr(), ep, h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
         dweight.data_ptr(), T, C, wp, wb)
    return dx, dweight


def rmsnorm_grad_f16(dy, h, weight, rstd, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """(dx, dweight) of rmsnorm_f16 (or, straight through the rounding to 8 bits, of rmsnorm_fp8_f16): dy and h [T,C],
    weight [C] fp16, rstd [T] FP32 as the norm gave it, dh [T,C] the gradient that reaches h along the residual (None:
    none).  dx [T,C] is the gradient of x and of residual alike; dweight [C] is FP32.  `workspace`: a device tensor
    (alloc_rmsnorm_grad_workspace makes one) owned by the caller; without one the call raises GemvTileError."""
    return _rmsnorm_grad(dy, h, weight, rstd, dh, dx, dweight, workspace, stream, torch.float16,
                         load_library().rmsnorm_grad_f16)


def rmsnorm_grad_bf16(dy, h, weight, rstd, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """rmsnorm_grad_f16 on bfloat16 tensors."""
    return _rmsnorm_grad(dy, h, weight, rstd, dh, dx, dweight, workspace, stream, torch.bfloat16,
                         load_library().rmsnorm_grad_bf16)


# ---- routing -------------------------------------------------------------------
def _route_topk(logits, k, bias, groups, top_groups, group_best, score, norm, scale, ids, weights, stream, dtype, call):
    dev = _first(logits, "logits", dtype, 2)
    T, E = logits.shape
    bp = _optional(bias, "bias", torch.float32, (E,), dev)
    code = _score(score)
    if not 1 <= k <= E:
        raise ValueError(f"k must be 1 .. {E}, got {k}")
    ids = _output(ids, "ids", torch.int32, (T, k), dev)
    weights = _output(weights, "weights", torch.float32, (T, k), dev)
    _run(dev, stream, call, logits.data_ptr(), bp, ids.data_ptr(), weights.data_ptr(), T, E, k, groups, top_groups, group_best,
         code, 1 if norm else 0, scale)
    return ids, weights


def route_topk_f16(logits, k, bias=None, groups=1, top_groups=1, group_best=1, score="softmax", norm=True, scale=1.0,
                   ids=None, weights=None, stream=None):
    """(ids, weights), int32 and FP32 [T,k]: the k best experts of each token by score ("softmax" or "sigmoid" of logits
    [T,E]) plus bias [E] FP32 (which counts for the choice only), best first, ties to the lowest, and scale · score,
    over the k scores' sum if norm.  With groups > 1 only experts of the top_groups best of that many equal groups are
    chosen, a group counting by its best choice or, with group_best 2, by the sum of its two best.  The choice is that
    of 64-bit arithmetic.  E <= 1024, k <= 32."""
    return _route_topk(logits, k, bias, groups, top_groups, group_best, score, norm, scale, ids, weights, stream, torch.float16,
                       load_library().route_topk_f16)


def route_topk_bf16(logits, k, bias=None, groups=1, top_groups=1, group_best=1, score="softmax", norm=True, scale=1.0,
                    ids=None, weights=None, stream=None):
    """route_topk_f16 of bfloat16 logits."""
    return _route_topk(logits, k, bias, groups, top_groups, group_best, score, norm, scale, ids, weights, stream, torch.bfloat16,
                       load_library().route_topk_bf16)


def route_topk_f32(logits, k, bias=None, groups=1, top_groups=1, group_best=1, score="softmax", norm=True, scale=1.0,
                   ids=None, weights=None, stream=None):
    """route_topk_f16 of FP32 logits."""
    return _route_topk(logits, k, bias, groups, top_groups, group_best, score, norm, scale, ids, weights, stream, torch.float32,
                       load_library().route_topk_f32)


def _route_topk_grad(logits, ids, dweights, score, norm, scale, dlogits, stream, dtype, call):
    dev = _first(logits, "logits", dtype, 2)
    T, E = logits.shape
    if _first(ids, "ids", torch.int32, 2) != dev or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, k] on device {dev}, got {tuple(ids.shape)} on {ids.device}")
    k = ids.shape[1]
    _shaped(dweights, "dweights", torch.float32, (T, k), dev)
    dlogits = _output(dlogits, "dlogits", dtype, (T, E), dev)
    _run(dev, stream, call, logits.data_ptr(), ids.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), T, E, k, _score(score),
         1 if norm else 0, scale)
    return dlogits


def route_topk_grad_f16(logits, ids, dweights, score="softmax", norm=True, scale=1.0, dlogits=None, stream=None):
    """dlogits [T,E] fp16 for the gradient dweights [T,k] FP32 of route_topk_f16's weights; ids as it gave them, and
    score, norm and scale as it was called with."""
    return _route_topk_grad(logits, ids, dweights, score, norm, scale, dlogits, stream, torch.float16,
                            load_library().route_topk_grad_f16)


def route_topk_grad_bf16(logits, ids, dweights, score="softmax", norm=True, scale=1.0, dlogits=None, stream=None):
    """route_topk_grad_f16 of bfloat16 logits."""
    return _route_topk_grad(logits, ids, dweights, score, norm, scale, dlogits, stream, torch.bfloat16,
                            load_library().route_topk_grad_bf16)


def route_topk_grad_f32(logits, ids, dweights, score="softmax", norm=True, scale=1.0, dlogits=None, stream=None):
    """route_topk_grad_f16 of FP32 logits."""
    return _route_topk_grad(logits, ids, dweights, score, norm, scale, dlogits, stream, torch.float32,
                            load_library().route_topk_grad_f32)


def alloc_route_sort_workspace(T, E, k, device):
    """A uint8 tensor on `device` that is large enough a workspace for route_sort of ids [T,k] over E experts."""
    need = int(load_library().gemvtile_route_sort_workspace(T, k, E))
    return torch.empty((max(need, 16),), dtype=torch.uint8, device=device)


def route_sort(ids, E, offsets=None, pos=None, workspace=None, stream=None):
    """(offsets, pos): the slots of ids [T,k] int32 sorted by expert, in their order within one.  offsets [E+1] int32 as
    gemm_grouped_* take it, pos [T,k] int32 the row of each slot; -1 for a slot whose id is outside 0 .. E - 1.
    `workspace`: a device tensor (alloc_route_sort_workspace makes one) owned by the caller, needed above 2048 slots;
    without one the call then raises GemvTileError."""
    dev = _first(ids, "ids", torch.int32, 2)
    T, k = ids.shape
    offsets = _output(offsets, "offsets", torch.int32, (E + 1,), dev)
    pos = _output(pos, "pos", torch.int32, (T, k), dev)
    wp, wb = _workspace(workspace, dev)
    _run(dev, stream, load_library().route_sort, ids.data_ptr(), offsets.data_ptr(), pos.data_ptr(), T, k, E, wp, wb)
    return offsets, pos


# ---- rows ----------------------------------------------------------------------
def _pos(pos, T, dev):
    """The number of slots of a token."""
    if _first(pos, "pos", torch.int32, 2) != dev:
        raise ValueError(f"pos must be on device {dev}, got {pos.device}")
    if pos.shape[0] != T:
        raise ValueError(f"pos must be [{T}, k], got {tuple(pos.shape)}")
    return pos.shape[1]


def _rows(t, name, dtype, K, dev):
    """The number of rows of [R, K]."""
    if _first(t, name, dtype, 2) != dev:
        raise ValueError(f"{name} must be on device {dev}, got {t.device}")
    if t.shape[1] != K:
        raise ValueError(f"{name} must be [R, {K}], got {tuple(t.shape)}")
    return t.shape[0]


def _route_gather(X, pos, Xs, stream, dtype, call):
    dev = _first(X, "X", dtype, 2)
    T, K = X.shape
    k = _pos(pos, T, dev)
    if Xs is None:
        Xs = torch.empty((T * k, K), dtype=dtype, device=X.device)
    R = _rows(Xs, "Xs", dtype, K, dev)
    _run(dev, stream, call, X.data_ptr(), pos.data_ptr(), Xs.data_ptr(), T, k, R, K)
    return Xs


def route_gather_f16(X, pos, Xs=None, stream=None):
    """Xs[pos[t,j]] = X[t]: the rows of X [T,K] fp16 in the order that route_sort found.  Xs [R,K], R = T k if it is not
    given; rows that no slot has stay as they were (uninitialised when Xs is None).  K % 8 == 0.  Its gradient is
    route_combine_f16 without weights."""
    return _route_gather(X, pos, Xs, stream, torch.float16, load_library().route_gather_f16)


def route_gather_bf16(X, pos, Xs=None, stream=None):
    """route_gather_f16 on bfloat16 tensors."""
    return _route_gather(X, pos, Xs, stream, torch.bfloat16, load_library().route_gather_bf16)


def route_gather_fp8(X, scale, pos, Xs=None, scales=None, stream=None):
    """(Xs, scales): route_gather_f16 of an 8-bit operand, X [T,K] float8_e4m3fn with scale [T, ceil(K/128)] FP32, for
    gemm_grouped_fp8_*.  K % 16 == 0."""
    dev = _first(X, "X", FP8, 2)
    T, K = X.shape
    k = _pos(pos, T, dev)
    _shaped(scale, "scale", torch.float32, (T, _blocks(K)), dev)
    if Xs is None:
        Xs = torch.empty((T * k if scales is None else scales.shape[0], K), dtype=FP8, device=X.device)
    R = _rows(Xs, "Xs", FP8, K, dev)
    scales = _output(scales, "scales", torch.float32, (R, _blocks(K)), dev)
    _run(dev, stream, load_library().route_gather_fp8, X.data_ptr(), scale.data_ptr(), pos.data_ptr(), Xs.data_ptr(),
         scales.data_ptr(), T, k, R, K)
    return Xs, scales


def _route_combine(D, pos, weights, Y, stream, dtype, call):
    dev = _first(D, "D", dtype, 2)
    R, K = D.shape
    if _first(pos, "pos", torch.int32, 2) != dev:
        raise ValueError(f"pos must be on device {dev}, got {pos.device}")
    T, k = pos.shape
    wp = _optional(weights, "weights", torch.float32, (T, k), dev)
    Y = _output(Y, "Y", dtype, (T, K), dev)
    _run(dev, stream, call, D.data_ptr(), pos.data_ptr(), wp, Y.data_ptr(), T, k, R, K)
    return Y


def route_combine_f16(D, pos, weights=None, Y=None, stream=None):
    """Y[t] = sum over j of weights[t,j] · D[pos[t,j]]: the experts' rows D [R,K] fp16 back to their tokens, summed in
    FP32 and rounded once.  weights [T,k] FP32 (None: ones); a slot whose pos is outside 0 .. R - 1 counts nothing.
    K % 8 == 0."""
    return _route_combine(D, pos, weights, Y, stream, torch.float16, load_library().route_combine_f16)


def route_combine_bf16(D, pos, weights=None, Y=None, stream=None):
    """route_combine_f16 on bfloat16 tensors."""
    return _route_combine(D, pos, weights, Y, stream, torch.bfloat16, load_library().route_combine_bf16)


def _route_combine_grad(dY, D, pos, weights, dD, dweights, stream, dtype, call):
    dev = _first(dY, "dY", dtype, 2)
    T, K = dY.shape
    k = _pos(pos, T, dev)
    R = _rows(D, "D", dtype, K, dev)
    _shaped(weights, "weights", torch.float32, (T, k), dev)
    dD = _output(dD, "dD", dtype, (R, K), dev)
    dweights = _output(dweights, "dweights", torch.float32, (T, k), dev)
    _run(dev, stream, call, dY.data_ptr(), D.data_ptr(), pos.data_ptr(), weights.data_ptr(), dD.data_ptr(),
         dweights.data_ptr(), T, k, R, K)
    return dD, dweights


def route_combine_grad_f16(dY, D, pos, weights, dD=None, dweights=None, stream=None):
    """(dD, dweights) of route_combine_f16 for dY [T,K]: dD[pos[t,j]] = weights[t,j] · dY[t] (rows that no slot has stay
    as they were) and dweights[t,j] = dY[t] · D[pos[t,j]] FP32."""
    return _route_combine_grad(dY, D, pos, weights, dD, dweights, stream, torch.float16,
                               load_library().route_combine_grad_f16)


def route_combine_grad_bf16(dY, D, pos, weights, dD=None, dweights=None, stream=None):
    """route_combine_grad_f16 on bfloat16 tensors."""
    return _route_combine_grad(dY, D, pos, weights, dD, dweights, stream, torch.bfloat16,
                               load_library().route_combine_grad_bf16)
