"""The 8-bit norm's numbers one by one: each e4m3 number is that nearest to y / scale, with y worked out in 64 bits and
the scale that came with it, and scales and rstd are the FP32 numbers nearest to the real ones.

Where two e4m3 numbers are about equally near, the kernel's quotient in 48 bits and the reference's in 53 may fall on
different sides: y / scale is off by 2^-49 for the lower half of rd / scale, some 2^-52 for rd and for the quotient, and
some 2^-52 here, less than 2^-47 in all; either number is right within 2^-45 of the middle.  An FP32 number nearest to a
value that is off by some 2^-52 is within half a step, 2^-24 of the value (or 2^-150), and that."""
import numpy as np
import pytest

import layer_reference as ref
from blocks_reference import e4m3_bits, e4m3_values
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])
NEAREST = 2.0**-24 * (1 + 2.0**-20)
EITHER = 2.0**-45
EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    return Env()


def _check(env, h, weight, fmt, eps=EPS):
    """Numbers, scales and rstd of the norm of h (on the device) against 64 bits; how many numbers lie within 2^-24 of the
    middle between two."""
    T, C = h.shape
    rstd = env.torch.empty(T, device="cuda")
    q, scale, _ = env.call("rmsnorm_fp8", fmt)(h, weight, None, eps, rstd=rstd)
    v = host(h)
    r = 1 / np.sqrt((v * v).sum(1) / C + eps)
    y = v * r[:, None] * host(weight)
    assert ((np.abs(host(rstd) - r) <= NEAREST * r + 2.0**-150) | (np.isinf(host(rstd)) & (r >= 2.0**128 * (1 - 2.0**-25)))).all()
    blocks = np.pad(y, ((0, 0), (0, -C % 128))).reshape(T, -1, 128)
    want = np.maximum(np.abs(blocks).max(-1) / 448, 2.0**-80)
    assert (np.abs(host(scale) - want) <= NEAREST * want).all()
    real = y / np.repeat(host(scale), 128, 1)[:, :C]
    bits = q.view(env.torch.uint8).cpu().numpy()
    most = np.minimum(np.abs(real), 448.0)
    either = [e4m3_bits(np.copysign(np.minimum(most * f, 448.0), real)) for f in (1 - EITHER, 1, 1 + EITHER)]
    wrong = np.argwhere((bits != either[0]) & (bits != either[1]) & (bits != either[2]))
    assert not len(wrong), (f"{len(wrong)} of {bits.size} are not the nearest; first at {tuple(wrong[0])}: "
                            f"{e4m3_values(bits)[tuple(wrong[0])]} for {real[tuple(wrong[0])]!r}")
    return (e4m3_bits(most * (1 - 2.0**-24)) != e4m3_bits(np.minimum(most * (1 + 2.0**-24), 448.0))).sum()


@FMT
@pytest.mark.parametrize("T,C", [(4800, 688), (300, 4096), (9, 20480)])
def test_numbers(env, T, C, fmt):
    r = np.random.default_rng(C)
    h = r.standard_normal((T, C))
    h[:, r.integers(C, size=max(1, C // 200))] *= 12
    _check(env, env.device(h, fmt), env.device(1 + 0.1 * r.standard_normal(C), fmt), fmt)


@FMT
@pytest.mark.parametrize("T,C", [(500, 64), (500, 128), (400, 256), (300, 512), (300, 1024), (200, 1536), (200, 2048), (100, 4096), (60, 8192)])
def test_numbers_next_to_the_middle(env, T, C, fmt):
    """Each block's largest number is 1.75, or 448 / 256, and all others are such middles over 256; a block's columns have
    one weight.  y / scale is then off the middle by what the scale's rounding to FP32 is off, less than 2^-24 to either
    side."""
    h, weight = _between(C, T)
    between = _check(env, env.device(h, fmt), env.device(weight, fmt), fmt)
    assert between >= 0.9 * T * C


def _between(C, T):
    r = np.random.default_rng(C + 1)
    h = r.integers(8, 16, (T, C)) * 2 + 1.0  # 17 to 31: five bits, between two numbers of four
    h = h * np.ldexp(1.0, r.integers(-12, -4, (T, C))) * r.choice([-1, 1], (T, C))
    h = np.where(np.abs(h) < 1.75, h, h / 4)
    h[:, ::128] = 1.75
    return h, np.repeat(r.integers(128, 256, -(-C // 128)) / 128, 128)[:C]  # weights of eight bits


@pytest.mark.parametrize("C", [64, 256, 1536, 4096])
def test_numbers_next_to_the_middle_of_every_size(env, C):
    """The same with rows and weights of bf16's whole range: r / scale has its 48 bits wherever they lie."""
    h, weight = _between(C, 300)
    for eh, ew in ((60, 40), (60, 50), (60, 60), (100, 10), (0, 90), (0, 110), (0, 125), (120, -20), (-100, 0), (-100, 100), (-60, -10), (-120, 120)):
        hd, wd = env.device(np.ldexp(h, eh), "bf16"), env.device(np.ldexp(weight, ew), "bf16")
        assert _check(env, hd, wd, "bf16", 0.0) >= 0.9 * 300 * C


@FMT
@pytest.mark.parametrize("C", [64, 272, 4096])
def test_signs_of_zeros(env, C, fmt):
    """Zeros, and numbers too small beside the block's largest, keep their signs."""
    r = np.random.default_rng(C)
    h = r.standard_normal((200, C)) * r.choice([0.0, 2.0**-13, 1.0], (200, C))
    h = h * r.choice([-1, 1], (200, C))
    _check(env, env.device(h, fmt), env.device(1 + 0.1 * r.standard_normal(C), fmt), fmt)
    q = env.call("rmsnorm_fp8", fmt)(env.device(h, fmt), env.device(np.ones(C), fmt), None, EPS)[0]
    signs = q.view(env.torch.uint8).cpu().numpy() >> 7
    np.testing.assert_array_equal(signs, np.signbit(h))


@FMT
@pytest.mark.parametrize("eps", [1e-6, 1e-5, 0.1])
@pytest.mark.parametrize("size", [0.1, 1.0, 3.0])
def test_eps_counts(env, size, eps, fmt):
    """Rows whose mean square is about eps: half of what r is off by comes from eps, whole in 64 bits."""
    r = np.random.default_rng(7)
    h = r.standard_normal((2000, 1024)) * size * eps**0.5
    _check(env, env.device(h, fmt), env.device(1 + 0.1 * r.standard_normal(1024), fmt), fmt, eps)


def test_eps_of_no_fp32_number(env):
    """An eps below FP32's range is not zero: a row of zeros has zeros, not NaN."""
    t = env.torch
    x, rstd = t.zeros(3, 256, device="cuda").bfloat16(), t.empty(3, device="cuda")
    y, _ = env.gt.rmsnorm_bf16(x, t.ones(256, device="cuda").bfloat16(), None, 1e-60, rstd=rstd)
    assert not y.any() and (np.abs(host(rstd) - 1e30) <= NEAREST * 1e30).all()


def _check_y(env, h, weight, fmt, eps):
    """y in 16 bits: r, h r and y take an FP32 rounding each (half a step of an h r below 2^-126 is 2^-150), then the one to
    16 bits; none makes y infinite below the type's largest."""
    y, _ = env.call("rmsnorm", fmt)(h, weight, None, eps)
    v = host(h)
    want = v * (1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)) * host(weight)
    tol = ref.rounded(want, 3 * ref.U * np.abs(want) + 2.0**-150 * (1 + np.abs(host(weight))), fmt)
    big = np.abs(want) >= 2.0**128 * (1 - 2.0**-9)  # what bf16 rounds to an infinity
    near(host(y)[~big], want[~big], tol[~big])
    assert (host(y)[big] == np.copysign(np.inf, want[big])).all()


def test_one_number_far_beyond_the_others(env):
    """weight h beyond FP32 where y is not: one h of 2^127 with a weight of 2 in a row of 4096 makes y 128."""
    t = env.torch
    h = t.randn(2, 4096, device="cuda", generator=t.Generator("cuda").manual_seed(1)).bfloat16()
    h[1, 300] = 2.0**127
    w = t.full((4096,), 2.0, device="cuda").bfloat16()
    q, scale, _ = env.gt.rmsnorm_fp8_bf16(h, w, None, EPS)
    assert q[1, 300].float() * scale[1, 2] == 128 and t.isfinite(scale).all() and t.isfinite(q.float()).all()
    assert env.gt.rmsnorm_bf16(h, w, None, EPS)[0][1, 300] == 128
    _check(env, h, w, "bf16")


@pytest.mark.parametrize("C", [16, 128, 272, 1024, 2048, 4096, 20480])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_the_whole_range_of_bf16(env, C, eps):
    """Rows of every size from bf16's subnormals to its largest numbers, with weights of every size: what is between h and
    y does not leave its range where y is in it."""
    r = np.random.default_rng(C)
    e = np.arange(-130, 127, 4)
    h = r.standard_normal((len(e), C)) * np.ldexp(1.0, e)[:, None]
    h = np.clip(h, -2.0**127, 2.0**127)
    h[::3, C // 2] = np.ldexp(1.0, 126)
    h[1::3, : C // 4] = np.ldexp(1.5, -133)
    for weight in (r.standard_normal(C), r.standard_normal(C) * np.ldexp(1.0, r.integers(-100, 100, C)), r.standard_normal(C) * 2.0**120):
        hd, wd = env.device(h, "bf16"), env.device(weight, "bf16")
        live = (host(hd) != 0).any(1)  # a row of zeros over an eps of 0 is NaN
        hd = hd[env.whole(np.flatnonzero(live))].contiguous()
        _check(env, hd, wd, "bf16", eps)
        _check_y(env, hd, wd, "bf16", eps)


@FMT
def test_roots_beyond_fp32(env, fmt):
    """Rows of zeros, and small ones, over an eps whose root FP32 does not hold."""
    r = np.random.default_rng(3)
    h = r.standard_normal((6, 272)) * 2.0**-20
    h[::2] = 0
    hd, wd = env.device(h, fmt), env.device(r.standard_normal(272), fmt)
    for eps in (1e-100, 1e-300, 1e200):
        _check(env, hd, wd, fmt, eps)
        _check_y(env, hd, wd, fmt, eps)
    assert not host(env.call("rmsnorm", fmt)(hd, wd, None, 1e-100)[0])[::2].any()


@FMT
def test_rows_that_are_not_finite_beside_others(env, fmt):
    """A row with an infinity has zeros elsewhere and NaN in its block; one of zeros over an eps of 0, and one with a NaN,
    are NaN; rows beside them, in a wave or not, do not change."""
    t = env.torch
    r = np.random.default_rng(4)
    for C in (64, 272, 4096):
        h, w = r.standard_normal((40, C)), env.device(1 + 0.1 * r.standard_normal(C), fmt)
        clean = env.call("rmsnorm_fp8", fmt)(env.device(h, fmt), w, None, 0.0)
        y = env.call("rmsnorm", fmt)(env.device(h, fmt), w, None, 0.0)[0]
        h[3, 5], h[8], h[30, C - 1] = np.inf, 0, np.nan
        keep = [i for i in range(40) if i not in (3, 8, 30)]
        hd = env.device(h, fmt)
        q, s, _ = env.call("rmsnorm_fp8", fmt)(hd, w, None, 0.0)
        y2 = env.call("rmsnorm", fmt)(hd, w, None, 0.0)[0]
        assert t.equal(q.view(t.uint8)[keep], clean[0].view(t.uint8)[keep]) and t.equal(s[keep], clean[1][keep]) and t.equal(y2[keep], y[keep])
        assert t.isnan(y2[[8, 30]]).all() and t.isnan(s[[8, 30]]).all()
        assert t.isnan(y2[3, 5]) and not y2[3, :5].any() and not y2[3, 6:].any()
        assert t.isnan(s[3, 0]) and (s[3, 1:] == 2.0**-80).all() and not q[3, 128:].float().any()
