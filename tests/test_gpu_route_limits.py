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
