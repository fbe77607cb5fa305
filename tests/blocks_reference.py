"""Plain 64-bit references of the quantisers, the block-scaled 8-bit products and the grouped products (numpy only),
and the tolerances that their tests use.

Tolerances.  A 16-bit result is its exact value v plus the error of the sum, rounded to the nearest: half a step,
eps / 2 relative to the value, or half the smallest subnormal.  With S the sum of the absolute terms:

  16-bit products: terms are exact in FP32; n of them are added one after another (in whatever order) with at most
  2^-23 of a partial sum lost each time (2^-24 rounded, 2^-23 if a sum is truncated), so |error| <= n 2^-23 S.

  8-bit products: the terms of a block are exact; the matrix core adds up to 128 of them in a window aligned to the
  largest.  2^-10 of the block's largest term (twice what it was measured to lose) bounds that.  Scaling a block's sum
  takes two roundings and adding it one, n / 128 times.
"""
import numpy as np

HALF_STEP = {"f16": 2.0**-11, "bf16": 2.0**-8}
HALF_SUBNORMAL = {"f16": 2.0**-25, "bf16": 2.0**-134}

_E4M3 = np.array([m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)])[:-1]


def e4m3_values(bits):
    """The numbers that e4m3 bit patterns (uint8) stand for."""
    table = np.append(_E4M3, np.nan)
    v = table[bits & 0x7F]
    return np.where(bits & 0x80, -v, v)


def e4m3_bits(v):
    """The nearest e4m3 patterns of |v| <= 448 (64 bits), ties to even; the sign of zero is kept."""
    a = np.abs(v)
    at = np.searchsorted(_E4M3, a)  # _E4M3[at - 1] < a <= _E4M3[at]
    at = np.minimum(at, len(_E4M3) - 1)
    below = np.maximum(at - 1, 0)
    low, high = a - _E4M3[below], _E4M3[at] - a
    pick = np.where((low < high) | ((low == high) & (below % 2 == 0)), below, at)
    return (pick | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def quantise(x, rows):
    """(bits, scale) of x [..., R, C] (64 bits, finite): blocks of `rows` x 128."""
    *lead, R, C = x.shape
    pr, pc = -R % rows, -C % 128
    y = np.pad(x, [(0, 0)] * len(lead) + [(0, pr), (0, pc)])
    y = y.reshape(*lead, (R + pr) // rows, rows, (C + pc) // 128, 128)
    scale = np.maximum((np.abs(y).max((-3, -1)) / 448).astype(np.float32), np.float32(2.0**-80))
    q = e4m3_bits(y / scale.astype(np.float64)[..., :, None, :, None])
    return q.reshape(*lead, R + pr, C + pc)[..., :R, :C], scale


def rounded(v, slack, fmt):
    """|result - v| allowed for a result whose sum is within `slack` of v."""
    return slack + HALF_STEP[fmt] * (np.abs(v) + slack) + HALF_SUBNORMAL[fmt]


def product(a, b, fmt):
    """a · bᵀ in 64 bits and its tolerance, for 16-bit operands."""
    v, s = a @ b.T, np.abs(a) @ np.abs(b).T
    return v, rounded(v, a.shape[1] * 2.0**-23 * s, fmt)


def block_product(a, sa, b, sb, sb_rows, fmt):
    """The block-scaled product of e4m3 values (64 bits) and its tolerance."""
    M, K = a.shape
    N = b.shape[0]
    v, slack, total = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for j in range(-(-K // 128)):
        cut = slice(128 * j, 128 * (j + 1))
        scale = np.outer(sa[:, j].astype(np.float64), np.repeat(sb[:, j].astype(np.float64), sb_rows)[:N])
        v += (a[:, cut] @ b[:, cut].T) * scale
        s = (np.abs(a[:, cut]) @ np.abs(b[:, cut]).T) * scale
        # the largest term is at most the product of the rows' largest numbers, and at most the sum
        top = np.minimum(np.outer(np.abs(a[:, cut]).max(1), np.abs(b[:, cut]).max(1)) * scale, s)
        slack += 2.0**-10 * top + 2 * 2.0**-24 * s
        total += s
        slack += 2.0**-24 * total
    return v, rounded(v, slack, fmt)
