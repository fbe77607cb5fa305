"""The norms and their gradients against 64-bit references."""
import numpy as np
import pytest

import layer_reference as ref
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])
EPS = 1e-5

# rows, columns: every launch shape, ragged ends of it, more rows than workgroups
SHAPES = [(1, 16), (3, 144), (5, 512), (2, 528), (4, 1024), (3, 1040), (7, 2048), (2, 2064), (3, 4096), (1, 4112), (2, 8192), (2, 8208),
          (1, 16384), (2, 16400), (1, 32768), (2100, 48), (17000, 128), (4100, 272)]


@pytest.fixture(scope="module")
def env():
    return Env()


def _inputs(env, T, C, fmt, seed=1):
    r = np.random.default_rng(seed + T + C)
    x, res = r.standard_normal((T, C)), r.standard_normal((T, C))
    x[:, r.integers(C, size=max(1, C // 100))] *= 12
    return env.device(x, fmt), env.device(res, fmt), env.device(1 + 0.1 * r.standard_normal(C), fmt)


def _check_fp8(q, scale, y):
    """e4m3 numbers and scales that stand for y (64 bits), whose FP32 value is off by NORM_ERROR."""
    T, C = y.shape
    blocks = np.pad(y, ((0, 0), (0, -C % 128))).reshape(T, -1, 128)
    want = np.maximum(np.abs(blocks).max(-1) / 448, 2.0**-80)
    near(scale, want, (ref.NORM_ERROR + 4 * ref.U) * want)
    s = np.repeat(scale, 128, 1)[:, :C]
    # half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6) around y / scale, itself a few units of FP32 off
    near(q * s, y, (2.0**-4 + 2 * ref.NORM_ERROR) * np.abs(y) + 2.0**-10 * s * (1 + 2.0**-10))


@FMT
@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("T,C", SHAPES)
def test_rmsnorm(env, T, C, with_residual, fmt):
    x, res, w = _inputs(env, T, C, fmt)
    if not with_residual:
        res = None
    rstd = env.torch.empty(T, device="cuda")
    y, h = env.call("rmsnorm", fmt)(x, w, res, EPS, rstd=rstd)
    want_h, want_r, want_y = ref.rmsnorm(host(x), None if res is None else host(res), host(w), EPS, fmt)
    np.testing.assert_array_equal(host(h), want_h)
    near(host(rstd), want_r, ref.NORM_ERROR * want_r)
    near(host(y), want_y, ref.rounded(want_y, ref.NORM_ERROR * np.abs(want_y), fmt))
    y8 = env.torch.empty_like(y)
    rstd8 = env.torch.empty_like(rstd)
    q, scale, h8 = env.call("rmsnorm_fp8", fmt)(x, w, res, EPS, y=y8, rstd=rstd8)
    assert env.torch.equal(h8, h) and env.torch.equal(y8, y) and env.torch.equal(rstd8, rstd)
    _check_fp8(q.float().cpu().double().numpy(), host(scale), want_y)
    again = env.call("rmsnorm_fp8", fmt)(x, w, res, EPS)
    assert env.torch.equal(again[0].view(env.torch.uint8), q.view(env.torch.uint8)) and env.torch.equal(again[1], scale)


@FMT
def test_columns_of_eight(env, fmt):
    for C in (8, 24, 1000):
        x, res, w = _inputs(env, 3, C, fmt)
        y, h = env.call("rmsnorm", fmt)(x, w, res, EPS)
        want_h, _, want_y = ref.rmsnorm(host(x), host(res), host(w), EPS, fmt)
        np.testing.assert_array_equal(host(h), want_h)
        near(host(y), want_y, ref.rounded(want_y, ref.NORM_ERROR * np.abs(want_y), fmt))


@FMT
@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(env, which, fmt):
    x, res, w = _inputs(env, 2500, 272, fmt)
    y, h = env.call("rmsnorm", fmt)(x, w, res, EPS)
    x2, res2 = x.clone(), res.clone()
    into = x2 if which == "x" else res2
    y2, h2 = env.call("rmsnorm", fmt)(x2, w, res2, EPS, h=into)
    assert h2 is into and env.torch.equal(h2, h) and env.torch.equal(y2, y)


def test_rows_apart(env):
    """A row with an infinity or a NaN, or of zeros, changes no other; nothing outside the outputs is written."""
    t = env.torch
    x, res, w = _inputs(env, 40, 272, "bf16")
    want = env.gt.rmsnorm_fp8_bf16(x, w, res, EPS)
    want_y = env.gt.rmsnorm_bf16(x, w, res, EPS)[0]
    x[3, 100], x[7, 271], x[9] = float("inf"), float("nan"), 0
    res[9] = 0
    q = t.full((42, 272), 7.0, device="cuda").to(t.float8_e4m3fn)
    s = t.full((42, 3), 7.0, device="cuda")
    h = t.full((42, 272), 7.0, device="cuda").bfloat16()
    y = t.full((42, 272), 7.0, device="cuda").bfloat16()
    env.gt.rmsnorm_fp8_bf16(x, w, res, EPS, h=h[1:41], q=q[1:41], scale=s[1:41], y=y[1:41])
    keep = [i for i in range(40) if i not in (3, 7, 9)]
    assert t.equal(q.view(t.uint8)[1:41][keep], want[0].view(t.uint8)[keep]) and t.equal(s[1:41][keep], want[1][keep])
    assert t.equal(h[1:41][keep], want[2][keep]) and t.equal(y[1:41][keep], want_y[keep])
    for out in (q.float(), s, h, y):
        assert (out[[0, 41]] == 7).all()
    assert not y[10].any() and not q[10].float().any() and (s[10] == 2.0**-80).all()
    assert t.isnan(s[8]).all() and t.isnan(y[8]).all()
    assert t.isnan(y[4, 100]) and t.isnan(s[4, 0])  # inf * 0


@FMT
@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("T,C", SHAPES + [(6, 8), (520, 24), (1300, 1040)])
def test_gradient(env, T, C, with_dh, fmt):
    h, dh, w = _inputs(env, T, C, fmt, seed=9)
    dy = env.device(np.random.default_rng(3).standard_normal((T, C)) * 0.1, fmt)
    rstd = env.torch.empty(T, device="cuda")
    env.call("rmsnorm", fmt)(h, w, None, EPS, rstd=rstd)
    space = env.gt.alloc_rmsnorm_grad_workspace(h).fill_(255)
    dx, dw = env.call("rmsnorm_grad", fmt)(dy, h, w, rstd, dh if with_dh else None, workspace=space)
    (want, slack), (want_w, slack_w) = ref.rmsnorm_grad(host(dy), host(dh) if with_dh else None, host(h), host(w), host(rstd))
    near(host(dx), want, ref.rounded(want, slack, fmt))
    near(host(dw), want_w, slack_w + 2.0**-149)
    again = env.call("rmsnorm_grad", fmt)(dy, h, w, rstd, dh if with_dh else None, workspace=space)
    assert env.torch.equal(again[0], dx) and env.torch.equal(again[1], dw)


# rows of every launch shape, several to a wave or a workgroup, and more of them than workgroups take at once
MANY = [(20000, 64), (33, 56), (20, 136), (70, 256), (5000, 512), (9, 528), (2600, 1024), (2100, 1536), (530, 2048), (600, 5120), (300, 8192),
        (270, 16384), (3, 16392), (259, 20480), (2, 24576), (258, 24584), (257, 32768)]


@pytest.mark.parametrize("T,C", MANY)
def test_many_rows(env, T, C):
    x, res, w = _inputs(env, T, C, "bf16")
    rstd = env.torch.empty(T, device="cuda")
    y, h = env.gt.rmsnorm_bf16(x, w, res, EPS, rstd=rstd)
    want_h, want_r, want_y = ref.rmsnorm(host(x), host(res), host(w), EPS, "bf16")
    np.testing.assert_array_equal(host(h), want_h)
    near(host(rstd), want_r, ref.NORM_ERROR * want_r)
    near(host(y), want_y, ref.rounded(want_y, ref.NORM_ERROR * np.abs(want_y), "bf16"))
    if C % 16 == 0:
        q, scale, _ = env.gt.rmsnorm_fp8_bf16(x, w, res, EPS)
        _check_fp8(q.float().cpu().double().numpy(), host(scale), want_y)
    dx, dw = env.gt.rmsnorm_grad_bf16(res, h, w, rstd, x, workspace=env.gt.alloc_rmsnorm_grad_workspace(h).fill_(255))
    (want, slack), (want_w, slack_w) = ref.rmsnorm_grad(host(res), host(x), host(h), host(w), host(rstd))
    near(host(dx), want, ref.rounded(want, slack, "bf16"))
    near(host(dw), want_w, slack_w + 2.0**-149)


@pytest.mark.parametrize("C", [8, 64, 128, 256, 512, 1024, 1536])
def test_rows_of_a_wave_apart(env, C):
    """A NaN in a row changes neither output nor gradient of those beside it in a wave or a workgroup."""
    t = env.torch
    x, res, w = _inputs(env, 70, C, "f16")
    rstd = t.empty(70, device="cuda")
    y, h = env.gt.rmsnorm_f16(x, w, res, EPS, rstd=rstd)
    space = env.gt.alloc_rmsnorm_grad_workspace(h)
    dx, _ = env.gt.rmsnorm_grad_f16(res, h, w, rstd, x, workspace=space)
    bad = [0, 5, 33, 69]
    keep = [i for i in range(70) if i not in bad]
    h2, rstd2 = h.clone(), rstd.clone()
    h2[bad, -1], rstd2[bad] = float("nan"), float("nan")
    y2, _ = env.gt.rmsnorm_f16(h2, w, None, EPS)
    dx2, _ = env.gt.rmsnorm_grad_f16(res, h2, w, rstd2, x, workspace=space)
    assert t.equal(y2[keep], y[keep]) and t.equal(dx2[keep], dx[keep])
    assert t.isnan(y2[bad]).all() and t.isnan(dx2[bad]).all()
    if C % 16 == 0:
        q, s, _ = env.gt.rmsnorm_fp8_f16(h, w, None, EPS)
        q2, s2, _ = env.gt.rmsnorm_fp8_f16(h2, w, None, EPS)
        assert t.equal(q2.view(t.uint8)[keep], q.view(t.uint8)[keep]) and t.equal(s2[keep], s[keep]) and t.isnan(s2[bad]).all()


@pytest.mark.parametrize("T,C", [(1, 8), (2, 2048), (2, 4112), (1, 24584), (5, 64), (3, 4096)])
def test_gradient_into_given(env, T, C):
    """dweight at any 4-byte alignment, and nothing around it."""
    t = env.torch
    h, dy, w = _inputs(env, T, C, "bf16")
    rstd = t.rand(T, device="cuda") + 0.5
    space = env.gt.alloc_rmsnorm_grad_workspace(h)
    want = env.gt.rmsnorm_grad_bf16(dy, h, w, rstd, workspace=space)
    for at in (1, 2, 3):
        dw = t.full((C + 8,), 7.0, device="cuda")
        dx, got = env.gt.rmsnorm_grad_bf16(dy, h, w, rstd, dweight=dw[at : at + C], workspace=space)
        assert t.equal(got, want[1]) and t.equal(dx, want[0]) and (dw[:at] == 7).all() and (dw[at + C :] == 7).all()


def test_gradient_of_no_rows(env):
    t = env.torch
    e = t.empty(0, 64, device="cuda").half()
    dw = t.full((64,), 7.0, device="cuda")
    dx, got = env.gt.rmsnorm_grad_f16(e, e, t.ones(64, device="cuda").half(), t.empty(0, device="cuda"), dweight=dw)
    assert dx.shape == (0, 64) and got is dw and not dw.any()


def test_refusals(env):
    t = env.torch
    x, w = t.zeros(3, 64, device="cuda").half(), t.zeros(64, device="cuda").half()
    for bad in (lambda: env.gt.rmsnorm_f16(x, w[:32]), lambda: env.gt.rmsnorm_f16(x, w, x[:2]),
                lambda: env.gt.rmsnorm_f16(x, w, h=x), lambda: env.gt.rmsnorm_f16(x[:, ::2], w[:32])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        env.gt.rmsnorm_bf16(x, w)
    with pytest.raises(env.gt.GemvTileError, match="UNSUPPORTED"):
        env.gt.rmsnorm_fp8_f16(x[:, :24].contiguous(), w[:24].contiguous())
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.rmsnorm_f16(x, w, None, -1.0)
    r = t.zeros(3, device="cuda")
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.rmsnorm_grad_f16(x, x, w, r)
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.rmsnorm_grad_f16(x, x, w, r, workspace=t.zeros(700, dtype=t.uint8, device="cuda"))
    with pytest.raises(TypeError):
        env.gt.rmsnorm_grad_f16(x, x, w, r, workspace=t.zeros(4096))
