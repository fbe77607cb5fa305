"""Rows to their experts and back, and the gradients, against 64-bit references."""
import numpy as np
import pytest

import layer_reference as ref
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])

# tokens, slots of each, columns
SHAPES = [(1, 1, 8), (1, 8, 16), (3, 5, 24), (27, 8, 2048), (5, 3, 2056), (130, 2, 136), (17, 4, 4096), (4, 32, 1000), (3, 7, 16384), (700, 6, 64)]


@pytest.fixture(scope="module")
def env():
    return Env()


def _pos(r, T, k, R, drop=0.2):
    """Different rows of 0 .. R - 1 for the slots, some of them outside."""
    pos = np.full(T * k, -1, np.int64)
    some = r.permutation(T * k)[: min(R, T * k)]
    pos[some] = r.permutation(R)[: len(some)]
    away = r.random(T * k) < drop
    pos[away] = r.choice([-1, -(1 << 31), R, (1 << 31) - 1], away.sum())
    return pos.reshape(T, k).astype(np.int32)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "fp8"])
@pytest.mark.parametrize("T,k,K", SHAPES)
def test_gather(env, T, k, K, fmt):
    t = env.torch
    K = -(-K // 16) * 16
    r = np.random.default_rng(T + K)
    R = T * k + 3
    pos = _pos(r, T, k, R)
    x = t.from_numpy(r.standard_normal((T, K))).cuda()
    x = x.to(t.float8_e4m3fn) if fmt == "fp8" else x.to(env.types[fmt])
    raw = t.uint8 if fmt == "fp8" else t.int16
    out = t.full((R, K), 7.0, device="cuda").to(x.dtype)
    want = host(out.view(raw)).copy()
    ok = (pos >= 0) & (pos < R)
    want[pos[ok]] = host(x.view(raw))[np.nonzero(ok)[0]]
    if fmt == "fp8":
        s = t.from_numpy(r.random((T, -(-K // 128)))).cuda().float()
        scales = t.full((R, s.shape[1]), 7.0, device="cuda")
        got, got_s = env.gt.route_gather_fp8(x, s, env.whole(pos), out, scales)
        want_s = np.full(scales.shape, 7.0)
        want_s[pos[ok]] = host(s)[np.nonzero(ok)[0]]
        np.testing.assert_array_equal(host(got_s), want_s)
    else:
        got = env.call("route_gather", fmt)(x, env.whole(pos), out)
    np.testing.assert_array_equal(host(got.view(raw)), want)


@FMT
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,K", SHAPES)
def test_combine(env, T, k, K, weighted, fmt):
    r = np.random.default_rng(T + K + 1)
    R = T * k + 2
    pos = _pos(r, T, k, R)
    D = env.device(r.standard_normal((R, K)), fmt)
    unused = np.setdiff1d(np.arange(R), pos)
    D[env.whole(unused)] = float("nan")
    w = r.random((T, k)) if weighted else np.ones((T, k))
    tw = env.device(w)
    y = env.torch.full((T + 2, K), 7.0, device="cuda").to(env.types[fmt])
    got = env.call("route_combine", fmt)(D, env.whole(pos), tw if weighted else None, y[1 : T + 1])
    d = host(D)
    d[unused] = 0
    want, tol = ref.combine(d, pos, host(tw), fmt)
    near(host(got), want, tol)
    assert (y[[0, -1]] == 7).all()


@FMT
@pytest.mark.parametrize("T,k,K", SHAPES)
def test_combine_gradient(env, T, k, K, fmt):
    r = np.random.default_rng(T + K + 2)
    R = T * k + 2
    pos = _pos(r, T, k, R)
    D, dY = env.device(r.standard_normal((R, K)), fmt), env.device(r.standard_normal((T, K)) * 0.1, fmt)
    w = env.device(r.random((T, k)))
    dD = env.torch.full((R, K), 7.0, device="cuda").to(env.types[fmt])
    before = host(dD)
    got, got_w = env.call("route_combine_grad", fmt)(dY, D, env.whole(pos), w, dD)
    (want, tol), (want_w, tol_w) = ref.combine_grad(host(dY), host(D), pos, host(w), fmt, before)
    near(host(got), want, tol)
    near(host(got_w), want_w, tol_w)


@pytest.mark.parametrize("T,k,K", [(900, 9, 256), (333, 4, 512), (50, 2, 520), (1001, 3, 128), (67, 5, 56)])
def test_tokens_of_a_wave_apart(env, T, k, K):
    """The gradients of tokens that share a wave or a workgroup, a NaN in some of them."""
    test_combine_gradient(env, T, k, K, "bf16")
    t = env.torch
    r = np.random.default_rng(T)
    pos = env.whole(_pos(r, T, k, T * k, 0.0))
    D, dY, w = env.device(r.standard_normal((T * k, K)), "f16"), env.device(r.standard_normal((T, K)), "f16"), env.device(r.random((T, k)))
    dD, dw = env.gt.route_combine_grad_f16(dY, D, pos, w)
    bad = [0, 3, 33, T - 1]
    keep = [i for i in range(T) if i not in bad]
    dY[bad, 1] = float("nan")
    dD2, dw2 = env.gt.route_combine_grad_f16(dY, D, pos, w)
    at = pos[keep].flatten().long()
    assert t.equal(dD2[at], dD[at]) and t.equal(dw2[keep], dw[keep]) and t.isnan(dw2[bad]).all()


def test_nothing(env):
    t = env.torch
    pos = t.zeros(3, 2, dtype=t.int32, device="cuda")
    none = t.empty(0, 16, device="cuda").half()
    y = t.full((3, 16), 7.0, device="cuda").half()
    assert not env.gt.route_combine_f16(none, pos, None, y).any()
    w = t.ones(3, 2, device="cuda")
    dD, dw = env.gt.route_combine_grad_f16(y, none, pos, w)
    assert dD.shape == (0, 16) and not dw.any()
    assert env.gt.route_gather_f16(y, pos, none).shape == (0, 16)
    e = t.empty(3, 0, device="cuda").half()
    dD, dw = env.gt.route_combine_grad_f16(e, t.empty(6, 0, device="cuda").half(), pos, w)
    assert not dw.any()
    assert env.gt.route_combine_f16(none, pos[:0]).shape == (0, 16)


def test_offsets_past_32_bits(env):
    """Rows whose first element lies beyond 2^32 bytes."""
    t = env.torch
    K, R = 16384, 140000
    D = t.empty(R, K, dtype=t.bfloat16, device="cuda")
    x = t.randn(3, K, device="cuda").bfloat16()
    pos = t.tensor([[R - 1, 5], [131073, R - 2], [7, 131071]], dtype=t.int32, device="cuda")
    env.gt.route_gather_bf16(x, pos, D)
    for i in range(3):
        for j in range(2):
            assert t.equal(D[pos[i, j]], x[i])
    y = env.gt.route_combine_bf16(D, pos, t.tensor([[0.5, 0.25]] * 3, device="cuda"))
    assert t.equal(y, (x.float() * 0.75).bfloat16())
    dD, dw = env.gt.route_combine_grad_bf16(x, D, pos, t.full((3, 2), 2.0, device="cuda"), D.clone())
    assert t.equal(dD[R - 1], x[0] * 2) and t.equal(dD[131071], x[2] * 2)
    n = (x.double() ** 2).sum(1, keepdim=True)
    assert ((dw.double() - n).abs() <= n * (8 * 8 + 10) * 2.0**-24).all()


def test_refusals(env):
    t = env.torch
    x, pos = t.zeros(3, 16, device="cuda").half(), t.zeros(3, 2, dtype=t.int32, device="cuda")
    w = t.zeros(3, 2, device="cuda")
    for bad in (lambda: env.gt.route_gather_f16(x, pos[:2]), lambda: env.gt.route_gather_f16(x, pos, x[:, :8].contiguous()),
                lambda: env.gt.route_combine_f16(x, pos, w[:2]), lambda: env.gt.route_combine_grad_f16(x, x[:, :8].contiguous(), pos, w),
                lambda: env.gt.route_combine_f16(x, pos, w, x[:2]), lambda: env.gt.route_gather_f16(x.t(), pos)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        env.gt.route_combine_f16(x, pos.long())
    with pytest.raises(env.gt.GemvTileError, match="UNSUPPORTED"):
        env.gt.route_gather_f16(t.zeros(3, 12, device="cuda").half(), pos)
    with pytest.raises(env.gt.GemvTileError, match="UNSUPPORTED"):
        env.gt.route_gather_f16(x, t.zeros(3, 33, dtype=t.int32, device="cuda"))
