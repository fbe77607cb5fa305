"""The choice of experts at the limits of its contract: logits that are not finite beside a bias or in groups, decisions
next to FP32's error with many experts, biases and rows at every place, repeated calls."""
import numpy as np
import pytest

import layer_reference as ref
from layer_env import Env, host, near

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16", "f32"])
INF = float("inf")


@pytest.fixture(scope="module")
def env():
    return Env()


@FMT
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("E", [4, 48, 64, 256, 600])
def test_a_softmax_of_an_infinite_logit(env, E, norm, fmt):
    """A softmax with an infinite or a NaN logit is NaN: so are the token's weights, chosen or not, with a bias every choice
    (the lowest experts are taken), and without one every group's sum (the lowest groups)."""
    t = env.torch
    r = np.random.default_rng(E)
    T, k, groups, top = 7, 3 if E > 4 else 1, 4, 2
    l, bias = r.standard_normal((T, E)), env.device(r.standard_normal(E) * 0.1)
    clean = env.device(l, fmt)
    l[1, E - 1], l[3, E // 2], l[5, E - 1], l[5, 0] = INF, np.nan, INF, -INF
    d = env.device(l, fmt)
    topk = env.call("route_topk", fmt)
    size = E // groups
    for b, g, n, best in ((bias, 1, 1, 1), (bias, groups, top, 1), (bias, groups, top, 2), (None, groups, top, 2), (None, groups, groups, 2)):
        ids, w = topk(d, k, b, g, n, best, "softmax", norm)
        want_ids, want_w = topk(clean, k, b, g, n, best, "softmax", norm)
        assert t.isnan(w[[1, 3, 5]]).all()
        assert t.equal(ids[::2][[0, 1, 3]], want_ids[::2][[0, 1, 3]]) and t.equal(w[::2][[0, 1, 3]], want_w[::2][[0, 1, 3]])
        for row in (1, 3, 5):
            if b is not None:
                assert ids[row].tolist() == list(range(k))
            else:
                kept = np.where(np.isnan(l[row]), -INF, host(d)[row])[: size * n] if size > 1 else None
                if kept is not None:
                    assert ids[row].tolist() == np.argsort(-kept, kind="stable")[:k].tolist()


@FMT
def test_a_sigmoid_of_an_infinite_logit(env, fmt):
    """A sigmoid of an infinite logit is 1 or 0."""
    r = np.random.default_rng(1)
    l = r.standard_normal((6, 64))
    l[1, 60], l[2, [3, 50]], l[3, 10:] = INF, INF, -INF
    finite = np.where(np.isposinf(l), 60000.0, l)  # 1 as well
    for bias in (None, env.device(r.standard_normal(64) * 0.1)):
        for norm in (True, False):
            for groups, top, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
                ids, w = env.call("route_topk", fmt)(env.device(l, fmt), 6, bias, groups, top, best, "sigmoid", norm)
                want_ids, want_w = env.call("route_topk", fmt)(env.device(finite, fmt), 6, bias, groups, top, best, "sigmoid", norm)
                assert env.torch.equal(ids, want_ids) and env.torch.equal(w, want_w)


@FMT
@pytest.mark.parametrize("T,E,k", [(9, 64, 8), (70, 256, 14), (5, 600, 32)])
def test_gradient_of_an_id_that_stands_twice(env, T, E, k, fmt):
    """Ids of a token are different; where one stands more than once in spite of that, one of its places counts for it, the
    same one in every call, and other experts and tokens are as they are."""
    t = env.torch
    r = np.random.default_rng(E)
    l, g = env.device(r.standard_normal((T, E)), fmt), env.device(r.standard_normal((T, k)))
    ids, _ = env.call("route_topk", fmt)(l, k, None, 1, 1, 1, "sigmoid", False)
    grad = env.call("route_topk_grad", fmt)
    want = grad(l, ids, g, "sigmoid", False)
    twice = ids.clone()
    twice[2, 1], twice[2, 2] = ids[2, 0], ids[2, 0]
    single = []
    for j in range(3):
        only = t.full_like(ids, -1)
        only[2, j] = ids[2, 0]
        single.append(grad(l, only, g, "sigmoid", False)[2, int(ids[2, 0])].item())
    got = grad(l, twice, g, "sigmoid", False)
    for _ in range(20):
        assert t.equal(grad(l, twice, g, "sigmoid", False), got)
    assert got[2, int(ids[2, 0])].item() in single and not got[2, ids[2, 1:3].long()].any()
    got[2, ids[2, :3].long()] = want[2, ids[2, :3].long()]
    assert t.equal(got, want)


@pytest.mark.parametrize("E", [64, 256, 512, 1024])
def test_decisions_beside_the_error_of_a_large_sum(env, E):
    """One logit on top and all others as far below as makes a softmax's sum most uncertain, with biases that bring their
    choices within a few units of FP32 of the one on top, and of one another."""
    r = np.random.default_rng(E)
    below = {64: 2.9, 256: 4.1, 512: 4.8, 1024: 5.44}[E]
    T = 250
    l = -below + r.standard_normal((T, E)) * 2.0**-12
    l[:, 0] = r.standard_normal(T) * 2.0**-14
    logits = env.device(l)
    p = ref.scores(host(logits), "softmax")
    bias = env.device(np.where(np.arange(E) == 0, 0, p[:, :1].mean() - p.mean(0)) + r.integers(-24, 25, E) * 2.0**-27)
    for k, groups, top, best in ((3, 1, 1, 1), (12, 1, 1, 1), (6, 8, 3, 1), (6, 8, 3, 2), (1, 16, 1, 2)):
        ids, w = env.gt.route_topk_f32(logits, k, bias, groups, top, best, "softmax", True)
        want_ids, want_w = ref.topk(host(logits), k, host(bias), groups, top, best, "softmax", 1, 1.0)
        np.testing.assert_array_equal(host(ids), want_ids)
        near(host(w), want_w, ref.topk_slack(host(logits), want_ids, want_w))
    ids = env.gt.route_topk_f32(logits, 6, None, 8, 3, 2, "softmax", True)[0]
    np.testing.assert_array_equal(host(ids), ref.topk(host(logits), 6, None, 8, 3, 2, "softmax", 1, 1.0)[0])


@FMT
@pytest.mark.parametrize("E", [16, 64, 250, 256, 512, 1024])
def test_a_bias_at_any_place(env, E, fmt):
    """A bias that is only 4-byte aligned."""
    r = np.random.default_rng(E)
    l, b = env.device(r.standard_normal((40, E)), fmt), env.device(r.standard_normal(E) * 0.1)
    want = env.call("route_topk", fmt)(l, 6, b, 2, 1, 2, "sigmoid")
    for at in (1, 2, 3):
        there = env.torch.full((E + 8,), 9.0, device="cuda")
        there[at : at + E] = b
        got = env.call("route_topk", fmt)(l, 6, there[at : at + E], 2, 1, 2, "sigmoid")
        assert env.torch.equal(got[0], want[0]) and env.torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt,T,E", [("f32", 1100000, 1024), ("bf16", 4300000, 512)])
def test_tokens_beyond_32_bits(env, fmt, T, E):
    """Logits and gradients beyond 2^32 bytes."""
    t = env.torch
    l = t.zeros(T, E, dtype=env.types[fmt], device="cuda")
    rows = t.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    r = np.random.default_rng(8)
    few = env.device(r.standard_normal((5, E)), fmt)
    l[rows] = few
    ids, w = env.call("route_topk", fmt)(l, 8)
    want_ids, want_w = env.call("route_topk", fmt)(few, 8)
    assert t.equal(ids[rows], want_ids) and t.equal(w[rows], want_w)
    other = t.ones(T, dtype=t.bool, device="cuda")
    other[rows] = False
    assert (ids[other] == t.arange(8, device="cuda")).all() and (w[other] == 0.125).all()
    g = t.zeros(T, 8, device="cuda")
    g[rows] = env.device(r.standard_normal((5, 8)))
    d = env.call("route_topk_grad", fmt)(l, ids, g)
    assert t.equal(d[rows], env.call("route_topk_grad", fmt)(few, want_ids, g[rows]))
    assert int(d.count_nonzero()) == int(d[rows].count_nonzero())
