"""Products with 4-bit weights over the range of numbers and scales, beside blocks that are added in the other order, and of
matrices whose rows begin beyond 2^32 bytes."""
import numpy as np
import pytest

import layer_reference as ref
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])


@pytest.fixture(scope="module")
def env():
    return Env()


def _tolerance(x, q, s, fmt):
    """That of the sums, and for terms and sums below FP32's normal numbers half a step of 2^-150 for each of a term's
    product, a block's addition and scaling, and the rest's additions."""
    want, tol = ref.gemv_fp4(x, q, s, fmt)
    return want, tol + (2 * x.shape[1] + 64) * 2.0**-150


# exponents of x and of the scales; sums of the terms' magnitudes stay below 2^128
RANGES = {"bf16": [(100, -120), (-100, 120), (-120, 125), (60, 55), (-60, -50), (-60, -60), (120, -126), (-20, -108), (-110, -10), (0, 100)],
          "f16": [(10, -24), (-10, 12), (0, 13), (-14, 20), (8, -20), (0, -23), (0, -30)]}


@FMT
@pytest.mark.parametrize("M,N,K", [(1, 40, 1056), (6, 33, 640), (17, 100, 512), (64, 48, 384)])
def test_sizes_of_numbers_and_scales(env, M, N, K, fmt):
    r = np.random.default_rng(M + K)
    for ex, es in RANGES[fmt]:
        q = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
        s = np.clip(127 + es + r.integers(-2, 1, (N, K // 32)), 0, 254).astype(np.uint8)
        x = env.device(r.standard_normal((M, K)) * 2.0**ex, fmt)
        want, tol = _tolerance(host(x), q, s, fmt)
        got = host(env.call("gemv_fp4", fmt)(x, env.whole(q), env.whole(s)))
        top = 65504 if fmt == "f16" else 3.3895e38
        in_range = np.abs(want) + tol < top
        near(got[in_range], want[in_range], tol[in_range])


@FMT
def test_rows_beside_blocks_of_zeros(env, fmt):
    """A block of zeros has the smallest scale, and the blocks and rows beside it are added in the other order: the same
    within the sums' error, with zeros anywhere and everywhere."""
    r = np.random.default_rng(5)
    for M, N, K in ((1, 100, 2080), (8, 64, 1024), (27, 515, 1056), (64, 130, 2080)):
        w = r.standard_normal((N, K)) * 0.05
        x = env.device(r.standard_normal((M, K)), fmt)
        for share in (0.01, 0.3, 1.0):
            w[np.repeat(r.random((N, K // 32)) < share, 32, 1)] = 0
            q, s = env.call("quantize_fp4", fmt)(env.device(w, fmt))
            want, tol = _tolerance(host(x), host(q), host(s), fmt)
            got = host(env.call("gemv_fp4", fmt)(x, q, s))
            near(got, want, tol)
        assert not got.any()


def test_weights_beyond_32_bits(env):
    """A matrix of 2^25 rows: those at its end begin beyond 2^32 bytes, the last outputs beyond 2^25 numbers."""
    t = env.torch
    N, K = 1 << 25, 288
    W = t.zeros(N, K // 2, dtype=t.uint8, device="cuda")
    s = t.full((N, K // 32), 127, dtype=t.uint8, device="cuda")
    r = np.random.default_rng(6)
    rows = np.concatenate([np.arange(20), N // 2 + np.arange(20), N - 40 + np.arange(40)])
    q = r.integers(0, 256, (len(rows), K // 2), dtype=np.uint8)
    W[env.whole(rows)] = env.whole(q)
    x = env.device(r.standard_normal((3, K)), "bf16")
    y = env.gt.gemv_fp4_bf16(x, W, s)
    want, tol = ref.gemv_fp4(host(x), q, np.full((len(rows), K // 32), 127, np.uint8), "bf16")
    near(host(y[:, env.whole(rows)]), want, tol)
    assert int((y != 0).sum()) <= 3 * len(rows)


def test_quantiser_beyond_32_bits(env):
    """Blocks beyond 2^32 bytes of x, and beyond 2^31 numbers."""
    t = env.torch
    N, K = 600000, 4096
    x = t.zeros(N, K, dtype=t.float16, device="cuda")
    r = np.random.default_rng(7)
    rows = np.concatenate([np.arange(3), N // 2 + np.arange(3), N - 3 + np.arange(3)])
    v = r.standard_normal((9, K))
    x[env.whole(rows)] = env.device(v, "f16")
    q, s = env.gt.quantize_fp4_f16(x)
    want_q, want_s = ref.quantise_fp4(host(env.device(v, "f16")))
    np.testing.assert_array_equal(q[env.whole(rows)].cpu().numpy(), want_q)
    np.testing.assert_array_equal(s[env.whole(rows)].cpu().numpy(), want_s)
    assert int(q.count_nonzero()) == np.count_nonzero(want_q) and int(s.count_nonzero()) == np.count_nonzero(want_s)
