"""The 4-bit quantiser, bit for bit, and the product of a few rows with 4-bit weights, against 64-bit references."""
import numpy as np
import pytest

import layer_reference as ref
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])


@pytest.fixture(scope="module")
def env():
    return Env()


def _check_quantiser(env, x, fmt):
    t = env.device(x, fmt)
    q, s = env.call("quantize_fp4", fmt)(t)
    want_q, want_s = ref.quantise_fp4(host(t))
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


@FMT
@pytest.mark.parametrize("shape", [(1, 32), (1, 96), (3, 160), (33, 1056), (129, 4096)])
def test_quantiser(env, shape, fmt):
    _check_quantiser(env, np.random.default_rng(1).standard_normal(shape) * 0.05, fmt)


@FMT
def test_quantiser_every_pattern(env, fmt):
    """All finite 16-bit patterns, 16 to a block beside numbers that set the block's scale, in several ratios."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    t = env.torch.from_numpy(bits.view(np.int16)).view(env.types[fmt]).double().numpy()
    v = t[np.isfinite(t)].reshape(-1, 16)
    _check_quantiser(env, np.concatenate([v, v * 0.37], 1), fmt)
    small = v[np.abs(v).max(1) < 1e3]
    _check_quantiser(env, np.concatenate([small, small[:, ::-1] * 3], 1), fmt)


@FMT
def test_quantiser_ties(env, fmt):
    """Numbers exactly between two of the format's, next to such, and scales at the border of 6."""
    steps = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for top in (6.0, 6.0 * (1 + 2.0**-7), 4.0, 3.0, 5.0):
        for shift in (1.0, 1 + 2.0**-7, 1 - 2.0**-8):
            for scale in (1.0, 2.0**-9):
                v = np.concatenate([steps * shift, -steps * shift, [0.0, -0.0, top]]) * scale
                rows.append(np.concatenate([v, np.zeros(32 - len(v))]))
    _check_quantiser(env, np.stack(rows), fmt)


def test_quantiser_not_finite_and_zero(env):
    x = np.random.default_rng(2).standard_normal((4, 96))
    x[2] = 0.0
    x[3] = 2.0**-133
    want = env.gt.quantize_fp4_bf16(env.device(x, "bf16"))
    assert host(want[1])[2].max() == 0 and host(want[0])[2].max() == 0
    x[0, 40] = np.inf
    x[1, 95] = np.nan
    q, s = env.gt.quantize_fp4_bf16(env.device(x, "bf16"))
    q, s, wq, ws = (host(t).copy() for t in (q, s, *want))
    assert s[0, 1] == 255 and s[1, 2] == 255 and not q[0, 16:32].any() and not q[1, 32:].any()
    for a, b in ((q, wq), (s, ws)):
        w = a.shape[1] // 3
        a[0, w : 2 * w] = b[0, w : 2 * w]
        a[1, 2 * w :] = b[1, 2 * w :]
        np.testing.assert_array_equal(a, b)


def test_quantiser_of_experts(env):
    x = env.device(np.random.default_rng(3).standard_normal((3, 5, 64)), "f16")
    q, s = env.gt.quantize_fp4_f16(x)
    assert q.shape == (3, 5, 32) and s.shape == (3, 5, 2)
    flat = env.gt.quantize_fp4_f16(x.reshape(15, 64))
    assert env.torch.equal(q.reshape(15, 32), flat[0]) and env.torch.equal(s.reshape(15, 2), flat[1])


def _weights(r, N, K, low=110, high=130):
    return r.integers(0, 256, (N, K // 2), dtype=np.uint8), r.integers(low, high, (N, K // 32)).astype(np.uint8)


SHAPES = [(1, 1, 32), (1, 16, 128), (1, 17, 160), (2, 15, 64), (3, 33, 96), (4, 300, 1024), (5, 40, 4128), (15, 31, 224), (16, 100, 512),
          (17, 47, 2080), (27, 515, 1056), (32, 64, 256), (33, 65, 1056), (48, 70, 320), (64, 130, 2080), (65, 50, 256), (200, 33, 160),
          (1, 1000, 14336), (1, 5000, 96), (1, 9000, 544), (7, 8200, 288), (40, 4200, 160),
          # each number of rows of x and of W that a workgroup has, and scales past one segment of 8192 or 16384 columns
          *((M, N, 160) for M in (1, 5, 9, 20, 32, 40, 64) for N in (4100, 8200, 12290)), (3, 16400, 64), (12, 16400, 64),
          (17, 2080, 96), (9, 2080, 96), (17, 2752, 64), (81, 1360, 96), (25, 6160, 64), (33, 6160, 64), (73, 3090, 64),
          (2, 20, 16416), (1, 35, 33024), (13, 33, 20000), (70, 18, 16512), (18, 8210, 8224)]


@FMT
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemv(env, M, N, K, fmt):
    r = np.random.default_rng(M * 7 + N + K)
    q, s = _weights(r, N, K)
    x = env.device(r.standard_normal((M, K)), fmt)
    y = env.torch.full((M + 2, N), 7.0, dtype=env.types[fmt], device="cuda")
    got = env.call("gemv_fp4", fmt)(x, env.whole(q), env.whole(s), y[1 : M + 1])
    want, tol = ref.gemv_fp4(host(x), q, s, fmt)
    near(host(got), want, tol)
    assert (y[[0, -1]] == 7).all()
    if M == 1:
        one = env.call("gemv_fp4", fmt)(x[0], env.whole(q), env.whole(s))
        assert one.shape == (N,) and env.torch.equal(one, got[0])


@pytest.mark.parametrize("K", [96, 160, 16416])
def test_gemv_of_one_of_several_matrices(env, K):
    """Weights and scales of one expert: scales that begin at any byte."""
    r = np.random.default_rng(K)
    q, s = _weights(r, 3 * 5, K)
    x = env.device(r.standard_normal((2, K)), "bf16")
    tq, ts = env.whole(q).reshape(3, 5, -1), env.whole(s).reshape(3, 5, -1)
    for e in range(3):
        want, tol = ref.gemv_fp4(host(x), q[5 * e : 5 * e + 5], s[5 * e : 5 * e + 5], "bf16")
        near(host(env.gt.gemv_fp4_bf16(x, tq[e], ts[e])), want, tol)


@FMT
def test_gemv_mixed_scales(env, fmt):
    """Chunks in which a few blocks have scales that 16-bit numbers do not hold, among others, for every block of rows."""
    r = np.random.default_rng(8)
    for M, N, K in ((1, 40, 1056), (6, 33, 640), (14, 50, 1024), (30, 40, 512), (64, 48, 384), (50, 300, 256)):
        q, s = _weights(r, N, K, 118, 124)
        s[r.random(s.shape) < 0.05] = 20
        s[r.random(s.shape) < 0.02] = 0
        if fmt == "bf16":
            s[r.random(s.shape) < 0.002] = 230
        x = env.device(r.standard_normal((M, K)), fmt)
        want, tol = ref.gemv_fp4(host(x), q, s, fmt)
        near(host(env.call("gemv_fp4", fmt)(x, env.whole(q), env.whole(s))), want, tol)


@FMT
def test_gemv_of_quantised_weights(env, fmt):
    r = np.random.default_rng(5)
    w = env.device(r.standard_normal((200, 416)) * 0.05, fmt)
    x = env.device(r.standard_normal((6, 416)), fmt)
    q, s = env.call("quantize_fp4", fmt)(w)
    want, tol = ref.gemv_fp4(host(x), host(q), host(s), fmt)
    near(host(env.call("gemv_fp4", fmt)(x, q, s)), want, tol)
    # what 4 bits cost: a number is off by at most half of the widest step (2 of 6) of its block's scale
    widest = np.repeat(np.ldexp(1.0, host(s).astype(int) - 127), 32, 1)
    near(ref.widen_fp4(host(q), host(s)), host(w), widest)


@FMT
def test_gemv_every_number_and_scale(env, fmt):
    """One-hot rows read single numbers: every code in every place of a block, and scales over the whole range."""
    K = 224
    q = np.zeros((16, K // 2), np.uint8)
    codes = (np.arange(16)[:, None] + np.arange(K)[None] * 3) % 16
    q = (codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)
    for low in range(0, 256, 7):
        s = np.minimum(low + np.arange(7), 255).astype(np.uint8)[None].repeat(16, 0)
        x = env.device(np.eye(K), fmt)
        got = host(env.call("gemv_fp4", fmt)(x, env.whole(q), env.whole(s)))
        v = ref.widen_fp4(q, s)
        blocks = np.repeat(s == 255, 32, 1)
        # every other block of a row adds 0 * its numbers: a NaN scale anywhere makes the whole row NaN
        v = np.where(blocks.any(1, keepdims=True), np.nan, v).T
        with np.errstate(over="ignore"):
            want = ref.round16(v, fmt)
            want = np.where(np.abs(want) > (65504 if fmt == "f16" else 3.39e38), np.copysign(np.inf, want), want)
        near(got, want, 0)


@FMT
def test_gemv_not_finite(env, fmt):
    """An infinity or a NaN in a row of x gives what the sum gives; other rows, and what lies behind the rows, do not matter."""
    r = np.random.default_rng(6)
    M, N, K = 5, 37, 160
    q, s = _weights(r, N, K)
    x = r.standard_normal((M + 1, K))
    clean = host(env.call("gemv_fp4", fmt)(env.device(x, fmt)[:M], env.whole(q), env.whole(s)))
    x[1, 130] = np.inf
    x[3, 7] = np.nan
    x[M] = np.nan
    t = env.device(x, fmt)
    got = host(env.call("gemv_fp4", fmt)(t[:M], env.whole(q), env.whole(s)))
    np.testing.assert_array_equal(got[[0, 2, 4]], clean[[0, 2, 4]])
    assert np.isnan(got[3]).all()
    w = ref.widen_fp4(q, s)[:, 130]
    np.testing.assert_array_equal(got[1], np.where(w == 0, np.nan, np.copysign(np.inf, w)))


def test_gemv_empty(env):
    t = env.torch
    w, s = t.zeros(5, 0, dtype=t.uint8, device="cuda"), t.zeros(5, 0, dtype=t.uint8, device="cuda")
    y = t.full((3, 5), 7.0, device="cuda").half()
    assert (env.gt.gemv_fp4_f16(t.zeros(3, 0, device="cuda").half(), w, s, y) == 0).all()
    assert env.gt.gemv_fp4_f16(t.zeros(0, 32, device="cuda").half(), t.zeros(5, 16, dtype=t.uint8, device="cuda"),
                               t.zeros(5, 1, dtype=t.uint8, device="cuda")).shape == (0, 5)


def test_refusals(env):
    t = env.torch
    x = t.zeros(2, 64, device="cuda").half()
    w, s = t.zeros(5, 32, dtype=t.uint8, device="cuda"), t.zeros(5, 2, dtype=t.uint8, device="cuda")
    for bad in ((x[:, :32].contiguous(), w, s), (x, w, s[:, :1].contiguous()), (x, w[:4], s), (x.t(), w, s)):
        with pytest.raises(ValueError):
            env.gt.gemv_fp4_f16(*bad)
    with pytest.raises(TypeError):
        env.gt.gemv_fp4_bf16(x, w, s)
    with pytest.raises(ValueError, match="multiple of 32"):
        env.gt.quantize_fp4_f16(t.zeros(2, 48, device="cuda").half())
    with pytest.raises(env.gt.GemvTileError):
        env.gt.gemv_fp4_f16(t.zeros(132, device="cuda").half()[4:].reshape(2, 64), w, s)
