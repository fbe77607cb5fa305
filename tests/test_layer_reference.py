"""The 64-bit references' gradients against differences of the references' forward (numpy only)."""
import numpy as np
import pytest

import layer_reference as ref

STEP = 1e-6
# A central difference of a function with third derivatives of a few units is off by STEP^2, and by the rounding of its
# two values (2^-53 of some units each) over STEP.
NEAR = 1e-8


def _differences(f, x):
    """d f(x) / d x for a scalar f."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += STEP
        down[i] -= STEP
        g[i] = (f(up) - f(down)) / (2 * STEP)
    return g


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_topk_grad(score, norm):
    r = np.random.default_rng(1)
    logits, g = r.standard_normal((3, 7)), r.standard_normal((3, 2))
    ids, _ = ref.topk(logits, 2, None, 1, 1, 1, score, norm, 2.5)

    def f(l):
        p = ref.scores(l, score)
        c = np.take_along_axis(p, ids, 1)
        return (g * 2.5 * (c / c.sum(1, keepdims=True) if norm else c)).sum()

    got, slack = ref.topk_grad(logits, ids, g, score, norm, 2.5)
    np.testing.assert_allclose(got, _differences(f, logits), rtol=0, atol=NEAR)
    assert (slack >= 0).all()


def test_rmsnorm_grad():
    r = np.random.default_rng(2)
    h, w, dy, dh = r.standard_normal((3, 6)), r.standard_normal(6), r.standard_normal((3, 6)), r.standard_normal((3, 6))

    def f(h, w):
        return (dy * h / np.sqrt((h * h).mean(1, keepdims=True) + 0.1) * w).sum() + (dh * h).sum()

    (dx, _), (dw, _) = ref.rmsnorm_grad(dy, dh, h, w, 1 / np.sqrt((h * h).mean(1) + 0.1))
    np.testing.assert_allclose(dx, _differences(lambda v: f(v, w), h), rtol=0, atol=NEAR)
    np.testing.assert_allclose(dw, _differences(lambda v: f(h, v), w), rtol=0, atol=NEAR)


def test_combine_grad():
    r = np.random.default_rng(3)
    pos = np.array([[2, 0], [-1, 3], [1, 9]])
    D, w, dY = r.standard_normal((5, 4)), r.standard_normal((3, 2)), r.standard_normal((3, 4))
    (dD, _), (dw, _) = ref.combine_grad(dY, D, pos, w, "f16", np.zeros_like(D))
    np.testing.assert_allclose(dD, _differences(lambda v: (dY * ref.combine(v, pos, w, "f16")[0]).sum(), D), rtol=0, atol=NEAR)
    np.testing.assert_allclose(dw, _differences(lambda v: (dY * ref.combine(D, pos, v, "f16")[0]).sum(), w), rtol=0, atol=NEAR)


def test_round16():
    r = np.random.default_rng(4)
    import torch

    v = np.concatenate([r.standard_normal(1000) * 2.0 ** r.integers(-30, 14, 1000), [0.0, -0.0, 1 + 2.0**-8, 1 + 3 * 2.0**-8, 2.0**-134]])
    f = v.astype(np.float32)  # what torch rounds from
    for fmt, t in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        np.testing.assert_array_equal(ref.round16(f.astype(np.float64), fmt), torch.from_numpy(f).to(t).double().numpy())
