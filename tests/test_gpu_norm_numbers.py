"""The 8-bit norm's numbers one by one: each e4m3 number is that nearest to y / scale, with y worked out in 64 bits and
the scale that came with it, and scales and rstd are the FP32 numbers nearest to the real ones.

Where two e4m3 numbers are about equally near, the kernel's quotient in 48 bits and the reference's in 53 may fall on
different sides: y / scale is off by 2^-49 for the lower half of rd / scale, some 2^-52 for rd and for the quotient, and
some 2^-52 here, less than 2^-47 in all; either number is right within 2^-45 of the middle.  An FP32 number nearest to a
value that is off by some 2^-52 is within half a step, 2^-24 of the value, and that."""
import numpy as np
import pytest

from blocks_reference import e4m3_bits, e4m3_values
from layer_env import Env, host

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
    assert (np.abs(host(rstd) - r) <= NEAREST * r).all()
    blocks = np.pad(y, ((0, 0), (0, -C % 128))).reshape(T, -1, 128)
    want = np.maximum(np.abs(blocks).max(-1) / 448, 2.0**-80)
    assert (np.abs(host(scale) - want) <= NEAREST * want).all()
    real = y / np.repeat(host(scale), 128, 1)[:, :C]
    bits = q.view(env.torch.uint8).cpu().numpy()
    most = np.minimum(np.abs(real), 448.0)
    near = [e4m3_bits(np.copysign(np.minimum(most * f, 448.0), real)) for f in (1 - EITHER, 1, 1 + EITHER)]
    wrong = np.argwhere((bits != near[0]) & (bits != near[1]) & (bits != near[2]))
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
    r = np.random.default_rng(C + 1)
    h = r.integers(8, 16, (T, C)) * 2 + 1.0  # 17 to 31: five bits, between two numbers of four
    h = h * np.ldexp(1.0, r.integers(-12, -4, (T, C))) * r.choice([-1, 1], (T, C))
    h = np.where(np.abs(h) < 1.75, h, h / 4)
    h[:, ::128] = 1.75
    weight = np.repeat(r.integers(128, 256, -(-C // 128)) / 128, 128)[:C]  # eight bits
    near = _check(env, env.device(h, fmt), env.device(weight, fmt), fmt)
    assert near >= 0.9 * T * C


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
