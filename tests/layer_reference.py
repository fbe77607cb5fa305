"""Plain 64-bit references (numpy) of the 4-bit products, norms, routing and row movers, and the tolerances that their
tests use.

Tolerances.  u = 2^-24 is half a step of FP32 relative to its value; a sum of FP32 numbers in which no term goes through
more than n additions is off by at most n u S, S the sum of the absolute terms (2 u for additions that may be truncated,
as a matrix instruction's).  What is rounded to 16 bits afterwards is off by half a step of the result more.
"""
import numpy as np

from blocks_reference import rounded  # noqa: F401  (half a step, or half the smallest subnormal, on top of a slack)

U = 2.0**-24
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round16(v, fmt):
    """v (64 bits) as the nearest fp16 / bf16 numbers, ties to even, in 64 bits."""
    if fmt == "f16":
        return v.astype(np.float16).astype(np.float64)
    e = np.maximum(np.frexp(v)[1], -125)  # |v| < 2^e; numbers of this binade are 2^(e - 8) apart
    with np.errstate(invalid="ignore"):
        r = np.ldexp(np.rint(np.ldexp(v, 8 - e)), e - 8)
    return np.where(np.isfinite(v), r, v)


# ---- 4 bits ----------------------------------------------------------------------
def quantise_fp4(x):
    """(bytes, scale bytes) of x [N, K] (64 bits, finite)."""
    N, K = x.shape
    b = x.reshape(N, K // 32, 32)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -127)
    for _ in range(255):
        e = np.where(6 * np.ldexp(1.0, e) < top, e + 1, e)
    a = np.abs(np.ldexp(b, -e[..., None]))
    middle = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.searchsorted(middle, a)  # middle[code - 1] < a <= middle[code]
    tie = (code < 7) & (a == middle[np.minimum(code, 6)]) & (code % 2 == 1)
    code = (code + tie) | np.where(np.signbit(b), 8, 0)
    code = code.astype(np.uint8).reshape(N, K // 2, 2)
    return code[..., 0] | code[..., 1] << 4, (e + 127).astype(np.uint8)


def widen_fp4(q, scale):
    """The numbers that bytes and scale bytes stand for."""
    code = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, 1)


def gemv_fp4(x, q, scale, fmt):
    """The product and its tolerance.  A block's 32 terms are added by a matrix instruction, a wave's blocks by one FMA
    each, at most 16 waves' sums in a row: no term goes through more than 32 + K / 32 + 16 additions, 2 u each."""
    w = widen_fp4(q, scale)
    v, s = x @ w.T, np.abs(x) @ np.abs(w).T
    return v, rounded(v, (48 + x.shape[1] / 32) * 2 * U * s, fmt)


# ---- norm --------------------------------------------------------------------------
# The sum of squares of a row takes at most 64 additions in a lane, 6 over the wave and 16 over the waves; its relative
# error halves in the root; the quotient by C, eps, root and reciprocal are some units more, and y is two products.
NORM_ERROR = 64 * U


def rmsnorm(x, residual, weight, eps, fmt):
    """(h, r, y)."""
    h = x if residual is None else round16(x + residual, fmt)
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return h, r, h * r[:, None] * weight


def rmsnorm_grad(dy, dh, h, weight, r):
    """((dx, slack), (dweight, slack)) in 64 bits."""
    T, C = h.shape
    n = h * r[:, None]
    wdy = weight * dy
    dot, size = (wdy * n).mean(1, keepdims=True), np.abs(wdy * n).mean(1, keepdims=True)
    e = 0 if dh is None else dh
    dx = r[:, None] * (wdy - n * dot) + e
    # dot: 64 + 6 + 16 additions and three products a term; the rest is a handful of roundings of what is added.
    slack = 96 * U * r[:, None] * np.abs(n) * size + 4 * U * (r[:, None] * (np.abs(wdy) + np.abs(n * dot)) + np.abs(e))
    # dweight: a workgroup's rows (of at most 512), then 64 partial sums in a run and 8 runs; two products a term.
    dw = (dy * n).sum(0)
    return (dx, slack), (dw, (-(-T // min(T, 512)) + 76) * U * np.abs(dy * n).sum(0))


# ---- routing -----------------------------------------------------------------------
def scores(logits, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            m = logits.max(1, keepdims=True)
            p = np.where(np.isneginf(logits), 0.0, np.exp(logits - m))
            s = p.sum(1, keepdims=True)
            return p / np.where(s == 0, 1, s)
        e = np.exp(-np.abs(logits))
        return np.where(logits < 0, e, 1) / (1 + e)


def _ranked(v):
    """Indices of v [.., n] from the largest down, ties by index."""
    return np.argsort(-v, -1, kind="stable")


def topk(logits, k, bias, groups, top_groups, group_best, score, norm, scale):
    """(ids, weights) of finite or -inf logits (and -inf biases)."""
    T, E = logits.shape
    p = scores(logits, score)
    choice = logits if bias is None else p + bias
    allowed = np.ones((T, E), bool)
    if groups > 1:
        counted = (p if bias is None else choice) if group_best == 2 and E > groups else choice
        best = -np.sort(-counted.reshape(T, groups, -1), -1)
        value = best[..., :2].sum(-1) if group_best == 2 else best[..., 0]
        kept = _ranked(value)[:, :top_groups]
        allowed = np.zeros((T, groups), bool)
        np.put_along_axis(allowed, kept, True, 1)
        allowed = np.repeat(allowed, E // groups, 1)
    order = np.stack([np.lexsort((np.arange(E), -choice[t], ~allowed[t])) for t in range(T)]) if T else np.zeros((0, E), int)
    ids = order[:, :k]
    c = np.take_along_axis(p, ids, 1)
    if norm:
        if score == "sigmoid":  # ratios survive where the scores themselves leave the range
            l = np.take_along_axis(logits, ids, 1)
            ref = np.minimum(l.max(1, keepdims=True), 0)
            ref = np.where(np.isneginf(ref), 0, ref)
            c = np.exp(np.minimum(l, 0) - ref) / (1 + np.exp(-np.abs(l)))
        else:
            l = np.take_along_axis(logits, ids, 1)
            m = l.max(1, keepdims=True)
            c = np.where(np.isneginf(l), 0, np.exp(l - np.where(np.isneginf(m), 0, m)))
        s = c.sum(1, keepdims=True)
        c = c / np.where(s == 0, 1, s)
    return ids.astype(np.int32), scale * c


def topk_slack(logits, ids, weights):
    """A weight is off by the rounding of an exponential's argument (u times its size, at most the row's spread or the
    logit itself), 64 units for exponentials, sums over 1024 in a tree, quotients and the scale, and FP32's subnormals."""
    l = np.where(np.isfinite(logits), logits, 0)
    spread = l.max(1, keepdims=True) - l.min(1, keepdims=True) + np.abs(l).max(1, keepdims=True)
    return (64 + 2 * spread) * U * np.abs(weights) + 2.0**-140


def topk_grad(logits, ids, dweights, score, norm, scale):
    """(dlogits, slack): the slack is in units of the absolute terms of each difference."""
    T, E = logits.shape
    l = np.take_along_axis(logits, ids, 1)
    g = scale * dweights
    p = scores(logits, score)
    c = np.take_along_axis(p, ids, 1)
    spread = 64 + 2 * (logits.max(1, keepdims=True) - logits.min(1, keepdims=True) + np.abs(logits).max(1, keepdims=True))
    if score == "softmax" and not norm:
        full = np.zeros((T, E))
        np.put_along_axis(full, ids, g, 1)
        v = p * (full - (g * c).sum(1, keepdims=True))
        return v, spread * U * p * (np.abs(full) + np.abs(g * c).sum(1, keepdims=True)) + 2.0**-140
    if norm:
        w = topk_weights_of(l, score)
        mean, size = (g * w).sum(1, keepdims=True), np.abs(g * w).sum(1, keepdims=True)
        slope = w if score == "softmax" else w / (1 + np.exp(l))
        at, s = slope * (g - mean), slope * (np.abs(g) + size)
    else:
        at = g * c / (1 + np.exp(l))
        s = np.abs(at)
    v, slack = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(v, ids, at, 1)
    np.put_along_axis(slack, ids, spread * U * s, 1)
    return v, slack + 2.0**-140


def topk_weights_of(l, score):
    """Normalised weights of chosen logits."""
    if score == "softmax":
        c = np.exp(l - l.max(1, keepdims=True))
    else:
        c = np.exp(np.minimum(l, 0) - np.minimum(l.max(1, keepdims=True), 0)) / (1 + np.exp(-np.abs(l)))
    return c / c.sum(1, keepdims=True)


def sort_slots(ids, E):
    """(offsets, pos)."""
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < E)
    pos = np.full(flat.shape, -1, np.int32)
    slots = np.flatnonzero(valid)
    pos[slots[np.argsort(flat[slots], kind="stable")]] = np.arange(len(slots))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[valid], minlength=E))]).astype(np.int32)
    return offsets, pos.reshape(ids.shape)


# ---- rows --------------------------------------------------------------------------
def combine(D, pos, w, fmt):
    """(Y, tolerance): one FMA a term."""
    ok = (pos >= 0) & (pos < len(D))
    padded = np.concatenate([D, np.zeros((1, D.shape[1]))])
    rows = padded[np.where(ok, pos, len(D))]
    w = np.where(ok, w, 0)[..., None]
    v, s = (w * rows).sum(1), np.abs(w * rows).sum(1)
    return v, rounded(v, pos.shape[1] * U * s, fmt)


def combine_grad(dY, D, pos, w, fmt, before):
    """((dD, tolerance), (dweights, tolerance)); `before` is what dD held."""
    T, k = pos.shape
    dD, tol, dw, dtol = before.copy(), np.zeros_like(before), np.zeros((T, k)), np.zeros((T, k))
    n = 8 * -(-D.shape[1] // 2048) + 10  # terms of a lane, then 6 and 4 additions
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if 0 <= r < len(D):
                dD[r] = w[t, j] * dY[t]
                tol[r] = rounded(dD[r], U * np.abs(dD[r]), fmt)
                dw[t, j] = dY[t] @ D[r]
                dtol[t, j] = n * U * (np.abs(dY[t]) @ np.abs(D[r]))
    return (dD, tol), (dw, dtol)
