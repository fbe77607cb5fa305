"""What the norm's gradient writes of its workspace, and its rows beyond 2^32 bytes."""
import numpy as np
import pytest

from layer_env import Env, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return Env()


@pytest.mark.parametrize("T", [1, 2, 3, 33, 70, 600, 20000])
@pytest.mark.parametrize("C", [8, 64, 128, 256, 512, 1024, 1536, 2048, 4096, 8192, 16384, 24576, 32768])
def test_nothing_behind_the_workspace(env, T, C):
    """A workspace of just the bytes asked for, for every launch: nothing behind it is written, and where it lies does not
    matter."""
    if T * C > 1 << 25:
        T = (1 << 25) // C
    t = env.torch
    g = t.Generator("cuda").manual_seed(T + C)
    h, dy = (t.randn(T, C, device="cuda", generator=g).bfloat16() for _ in range(2))
    w, rstd = t.randn(C, device="cuda", generator=g).bfloat16(), t.rand(T, device="cuda", generator=g)
    need = env.gt.load_library().gemvtile_rmsnorm_grad_workspace(T, C)
    room = t.full((need + 4096,), 0xA5, dtype=t.uint8, device="cuda")
    want = env.gt.rmsnorm_grad_bf16(dy, h, w, rstd, workspace=env.gt.alloc_rmsnorm_grad_workspace(h))
    got = env.gt.rmsnorm_grad_bf16(dy, h, w, rstd, workspace=room[2048 : 2048 + need])
    assert (room[:2048] == 0xA5).all() and (room[2048 + need :] == 0xA5).all()
    assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.rmsnorm_grad_bf16(dy, h, w, rstd, workspace=room[2048 : 2048 + need - 1])


def test_rows_beyond_32_bits(env):
    """A norm and its gradient of rows beyond 2^32 bytes, those at both ends and in the middle checked."""
    t = env.torch
    T, C = 600000, 4096
    rows = t.tensor([0, 1, 262143, 262144, 524287, 524288, T - 1], device="cuda")
    few = env.device(np.random.default_rng(1).standard_normal((len(rows), C)), "bf16")
    x = t.zeros(T, C, dtype=t.bfloat16, device="cuda")
    x[rows] = few
    w = env.device(np.random.default_rng(2).standard_normal(C), "bf16")
    rstd = t.empty(T, device="cuda")
    q, s, h = env.gt.rmsnorm_fp8_bf16(x, w, x, 1e-5, rstd=rstd)
    want_r = t.empty(len(rows), device="cuda")
    want_q, want_s, want_h = env.gt.rmsnorm_fp8_bf16(few, w, few, 1e-5, rstd=want_r)
    assert t.equal(q[rows].view(t.uint8), want_q.view(t.uint8)) and t.equal(s[rows], want_s) and t.equal(h[rows], want_h)
    assert t.equal(rstd[rows], want_r) and int(h.count_nonzero()) == int(want_h.count_nonzero())
    # the zeros of the other rows have the weights' signs
    assert int((q.view(t.uint8) & 0x7F).count_nonzero()) == int((want_q.view(t.uint8) & 0x7F).count_nonzero())
    del q, x
    dx, dw = env.gt.rmsnorm_grad_bf16(h, h, w, rstd, workspace=env.gt.alloc_rmsnorm_grad_workspace(h))
    want_dx, want_dw = env.gt.rmsnorm_grad_bf16(want_h, want_h, w, want_r, workspace=env.gt.alloc_rmsnorm_grad_workspace(want_h))
    assert t.equal(dx[rows], want_dx) and int(dx.count_nonzero()) == int(want_dx.count_nonzero())
    # sums of the same seven terms and zeros, in another order
    n = (want_h.double() ** 2 * want_r[:, None].double()).sum(0)
    assert (np.abs(host(dw) - host(want_dw)) <= 2 * 9 * 2.0**-24 * host(n)).all()
