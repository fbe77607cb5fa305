"""Tensor entry points of the block-scaled 8-bit products and the products grouped by expert.

    quantize_fp8_rows_*(x)              (q, scale) of blocks of 1 x 128
    quantize_fp8_tiles_*(w)             (q, scale) of blocks of 128 x 128
    gemm_fp8_*(A, sA, B, sB)            D = (A scaled) · (B scaled)ᵀ
    gemm_grouped_*(X, W, offsets)       D[t] = X[t] · W[e]ᵀ for the rows t of group e
    gemm_grouped_dgrad_*(dY, W, offsets), gemm_grouped_wgrad_*(dY, X, offsets)   its gradients
    gemm_grouped_fp8_*(X, sX, W, sW, offsets)

Like the rest of the package this only marshals arguments (include/gemvtile.h
states each call's contract); the names end in the 16-bit format of the
input (quantisers) or of the output.
"""
from __future__ import annotations

import torch
from torch import Tensor
from torch._C import _cuda_getCurrentRawStream as _raw_stream

from . import BLOCK_CALLS, _check, _require, load_library

__all__ = list(BLOCK_CALLS)

FP8 = torch.float8_e4m3fn
BLOCK = 128


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


# A call's checks cost as much time as its launch if they are made one by one
# through several functions; each tensor is tested in one expression, and the
# reason is looked for only when that fails.
def _shaped(t, name, dtype, shape, dev):
    """t is a contiguous tensor of this type and shape on device number `dev`."""
    if (isinstance(t, Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous() and dev >= 0):
        return
    _require(t, name, len(shape), dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on device {dev}, got {t.device}")


def _first(t, name, dtype, ndim):
    """The device number of a call's first tensor."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous() and t.is_cuda):
        _require(t, name, ndim, dtype)
    return t.get_device()


def _output(t, name, dtype, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    _shaped(t, name, dtype, shape, dev)
    return t


def _offsets(offsets, dev):
    if _first(offsets, "offsets", torch.int32, 1) != dev:
        raise ValueError(f"offsets must be on device {dev}, got {offsets.device}")
    groups = offsets.shape[0] - 1
    if groups < 0:
        raise ValueError("offsets must have one element more than there are groups")
    return groups


def _run(dev, stream, call, *args):
    if stream is None:
        s = _raw_stream(dev)
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        status = call(*args, s)
    else:
        with torch.cuda.device(dev):
            status = call(*args, s)
    if status != 0:
        _check(status)


# ---- quantisers ----------------------------------------------------------------
def _quantize_rows(x, q, scale, stream, dtype, call):
    dev = _first(x, "x", dtype, 2)
    M, K = x.shape
    q = _output(q, "q", FP8, (M, K), dev)
    scale = _output(scale, "scale", torch.float32, (M, _blocks(K)), dev)
    _run(dev, stream, call, x.data_ptr(), q.data_ptr(), scale.data_ptr(), M, K)
    return q, scale


def quantize_fp8_rows_f16(x, q=None, scale=None, stream=None):
    """(q, scale) of x [M,K] fp16: q [M,K] float8_e4m3fn and scale [M, ceil(K/128)] FP32, one scale for every 128
    columns of a row.  K % 16 == 0.  scale = max(amax / 448, 2^-80), q the e4m3 number nearest to x / scale.  Enqueued
    on `stream` (default: the current stream), not synchronised."""
    return _quantize_rows(x, q, scale, stream, torch.float16, load_library().quantize_fp8_rows_f16)


def quantize_fp8_rows_bf16(x, q=None, scale=None, stream=None):
    """quantize_fp8_rows_f16 of a bfloat16 tensor."""
    return _quantize_rows(x, q, scale, stream, torch.bfloat16, load_library().quantize_fp8_rows_bf16)


def _quantize_tiles(x, q, scale, stream, dtype, call):
    many = isinstance(x, torch.Tensor) and x.dim() == 3
    dev = _first(x, "x", dtype, 3 if many else 2)
    *lead, N, K = x.shape
    q = _output(q, "q", FP8, (*lead, N, K), dev)
    scale = _output(scale, "scale", torch.float32, (*lead, _blocks(N), _blocks(K)), dev)
    _run(dev, stream, call, x.data_ptr(), q.data_ptr(), scale.data_ptr(), lead[0] if many else 1, N, K)
    return q, scale


def quantize_fp8_tiles_f16(x, q=None, scale=None, stream=None):
    """(q, scale) of a weight x [N,K], or of each of x [E,N,K], fp16: q of x's shape in float8_e4m3fn and scale
    [ceil(N/128), ceil(K/128)] (or [E, ...]) FP32, one for every 128 x 128.  K % 16 == 0; as quantize_fp8_rows_f16."""
    return _quantize_tiles(x, q, scale, stream, torch.float16, load_library().quantize_fp8_tiles_f16)


def quantize_fp8_tiles_bf16(x, q=None, scale=None, stream=None):
    """quantize_fp8_tiles_f16 of a bfloat16 tensor."""
    return _quantize_tiles(x, q, scale, stream, torch.bfloat16, load_library().quantize_fp8_tiles_bf16)


# ---- products --------------------------------------------------------------------
def _gemm_fp8(A, scale_A, B, scale_B, D, stream, dtype, call):
    dev = _first(A, "A", FP8, 2)
    if _first(B, "B", FP8, 2) != dev:
        raise ValueError("A and B must be on the same device")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError(f"K mismatch: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    kb = _blocks(K)
    _shaped(scale_A, "scale_A", torch.float32, (M, kb), dev)
    if _first(scale_B, "scale_B", torch.float32, 2) != dev:
        raise ValueError(f"scale_B must be on device {dev}, got {scale_B.device}")
    if scale_B.shape == (_blocks(N), kb):
        rows = BLOCK
    elif scale_B.shape == (N, kb):
        rows = 1
    else:
        raise ValueError(f"scale_B must be {[_blocks(N), kb]} (128 x 128 blocks) or {[N, kb]} (1 x 128), "
                         f"got {tuple(scale_B.shape)}")
    D = _output(D, "D", dtype, (M, N), dev)
    _run(dev, stream, call, A.data_ptr(), scale_A.data_ptr(), B.data_ptr(), scale_B.data_ptr(), D.data_ptr(), M, N, K,
         rows)
    return D


def gemm_fp8_f16(A, scale_A, B, scale_B, D=None, stream=None):
    """D = (A scaled) · (B scaled)ᵀ, rounded once to fp16.  A [M,K] and B [N,K] float8_e4m3fn, scale_A
    [M, ceil(K/128)], scale_B [ceil(N/128), ceil(K/128)] (a weight) or [N, ceil(K/128)] (both sides quantised by rows)
    FP32, D [M,N]; all contiguous, K % 16 == 0.  The product of two scales has to be a normal FP32 number (finite, 2^-126
    or more) or zero.  Enqueued on `stream` (default: the current stream), not synchronised.

    The gradients of an 8-bit product are this call again: dA = dD · B takes dD quantised by rows and Bᵀ with its
    scales transposed; dB = dDᵀ · A takes dDᵀ and Aᵀ both quantised by rows."""
    return _gemm_fp8(A, scale_A, B, scale_B, D, stream, torch.float16, load_library().gemm_fp8_f16)


def gemm_fp8_bf16(A, scale_A, B, scale_B, D=None, stream=None):
    """gemm_fp8_f16 with a bfloat16 result."""
    return _gemm_fp8(A, scale_A, B, scale_B, D, stream, torch.bfloat16, load_library().gemm_fp8_bf16)


def _weights(W, dtype, E, dev):
    """The [N, K] of one group's weights."""
    if _first(W, "W", dtype, 3) != dev:
        raise ValueError(f"W must be on device {dev}, got {W.device}")
    groups, N, K = W.shape
    if groups != E:
        raise ValueError(f"W has {groups} groups, offsets {E}")
    return N, K


def _grouped(X, W, offsets, D, stream, dtype, call):
    dev = _first(X, "X", dtype, 2)
    E = _offsets(offsets, dev)
    T, K = X.shape
    N, K2 = _weights(W, dtype, E, dev)
    if K != K2:
        raise ValueError(f"K mismatch: X is {tuple(X.shape)}, W is {tuple(W.shape)}")
    D = _output(D, "D", dtype, (T, N), dev)
    _run(dev, stream, call, X.data_ptr(), W.data_ptr(), offsets.data_ptr(), D.data_ptr(), T, N, K, E)
    return D


def gemm_grouped_f16(X, W, offsets, D=None, stream=None):
    """D[t] = X[t] · W[e]ᵀ for the rows offsets[e] <= t < offsets[e+1] of every group e; fp16.

    X [T,K] sorted by group, W [E,N,K], offsets [E+1] int32 on the device (non-decreasing, from >= 0 to <= T; read by
    the kernel, so there is no synchronisation), D [T,N]; all contiguous, K % 8 == 0, E <= 1024.  Rows of no group
    stay as they were in D, i.e. uninitialised when D is None.  Enqueued on `stream`, not synchronised."""
    return _grouped(X, W, offsets, D, stream, torch.float16, load_library().gemm_grouped_f16)


def gemm_grouped_bf16(X, W, offsets, D=None, stream=None):
    """gemm_grouped_f16 on bfloat16 tensors."""
    return _grouped(X, W, offsets, D, stream, torch.bfloat16, load_library().gemm_grouped_bf16)


def _grouped_dgrad(dY, W, offsets, dX, stream, dtype, call):
    dev = _first(dY, "dY", dtype, 2)
    E = _offsets(offsets, dev)
    T, N = dY.shape
    N2, K = _weights(W, dtype, E, dev)
    if N != N2:
        raise ValueError(f"N mismatch: dY is {tuple(dY.shape)}, W is {tuple(W.shape)}")
    dX = _output(dX, "dX", dtype, (T, K), dev)
    _run(dev, stream, call, dY.data_ptr(), W.data_ptr(), offsets.data_ptr(), dX.data_ptr(), T, N, K, E)
    return dX


def gemm_grouped_dgrad_f16(dY, W, offsets, dX=None, stream=None):
    """dX[t] = dY[t] · W[e] for the rows t of every group e: the gradient of gemm_grouped_f16 with respect to X.
    dY [T,N], W [E,N,K], dX [T,K]; N % 8 == 0 and K % 8 == 0.  Rows of no group stay as they were."""
    return _grouped_dgrad(dY, W, offsets, dX, stream, torch.float16, load_library().gemm_grouped_dgrad_f16)


def gemm_grouped_dgrad_bf16(dY, W, offsets, dX=None, stream=None):
    """gemm_grouped_dgrad_f16 on bfloat16 tensors."""
    return _grouped_dgrad(dY, W, offsets, dX, stream, torch.bfloat16, load_library().gemm_grouped_dgrad_bf16)


def _grouped_wgrad(dY, X, offsets, dW, stream, dtype, call):
    dev = _first(dY, "dY", dtype, 2)
    E = _offsets(offsets, dev)
    T, N = dY.shape
    if _first(X, "X", dtype, 2) != dev:
        raise ValueError(f"X must be on device {dev}, got {X.device}")
    T2, K = X.shape
    if T != T2:
        raise ValueError(f"T mismatch: dY is {tuple(dY.shape)}, X is {tuple(X.shape)}")
    dW = _output(dW, "dW", dtype, (E, N, K), dev)
    _run(dev, stream, call, dY.data_ptr(), X.data_ptr(), offsets.data_ptr(), dW.data_ptr(), T, N, K, E)
    return dW


def gemm_grouped_wgrad_f16(dY, X, offsets, dW=None, stream=None):
    """dW[e] = dY[rows of e]ᵀ · X[rows of e] for every group e (zeros for a group without rows): the gradient of
    gemm_grouped_f16 with respect to W.  dY [T,N], X [T,K], dW [E,N,K]; N % 8 == 0 and K % 8 == 0."""
    return _grouped_wgrad(dY, X, offsets, dW, stream, torch.float16, load_library().gemm_grouped_wgrad_f16)


def gemm_grouped_wgrad_bf16(dY, X, offsets, dW=None, stream=None):
    """gemm_grouped_wgrad_f16 on bfloat16 tensors."""
    return _grouped_wgrad(dY, X, offsets, dW, stream, torch.bfloat16, load_library().gemm_grouped_wgrad_bf16)


def _grouped_fp8(X, scale_X, W, scale_W, offsets, D, stream, dtype, call):
    dev = _first(X, "X", FP8, 2)
    E = _offsets(offsets, dev)
    T, K = X.shape
    N, K2 = _weights(W, FP8, E, dev)
    if K != K2:
        raise ValueError(f"K mismatch: X is {tuple(X.shape)}, W is {tuple(W.shape)}")
    kb = _blocks(K)
    _shaped(scale_X, "scale_X", torch.float32, (T, kb), dev)
    _shaped(scale_W, "scale_W", torch.float32, (E, _blocks(N), kb), dev)
    D = _output(D, "D", dtype, (T, N), dev)
    _run(dev, stream, call, X.data_ptr(), scale_X.data_ptr(), W.data_ptr(), scale_W.data_ptr(), offsets.data_ptr(),
         D.data_ptr(), T, N, K, E)
    return D


def gemm_grouped_fp8_f16(X, scale_X, W, scale_W, offsets, D=None, stream=None):
    """gemm_grouped_f16 on 8-bit operands: X [T,K] and W [E,N,K] float8_e4m3fn, scale_X [T, ceil(K/128)] and scale_W
    [E, ceil(N/128), ceil(K/128)] FP32 as the quantisers give them, D [T,N] fp16.  K % 16 == 0."""
    return _grouped_fp8(X, scale_X, W, scale_W, offsets, D, stream, torch.float16, load_library().gemm_grouped_fp8_f16)


def gemm_grouped_fp8_bf16(X, scale_X, W, scale_W, offsets, D=None, stream=None):
    """gemm_grouped_fp8_f16 with a bfloat16 result."""
    return _grouped_fp8(X, scale_X, W, scale_W, offsets, D, stream, torch.bfloat16,
                        load_library().gemm_grouped_fp8_bf16)
