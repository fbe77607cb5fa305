"""The choice of experts, its gradient and the sort of the slots against 64-bit references."""
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


def _check(env, logits, fmt, k, bias=None, groups=1, top_groups=1, group_best=1, score="softmax", norm=1, scale=1.0):
    l = env.device(logits, fmt)
    b = None if bias is None else env.device(bias)
    ids, w = env.call("route_topk", fmt)(l, k, b, groups, top_groups, group_best, score, norm, scale)
    want_ids, want_w = ref.topk(host(l), k, None if b is None else host(b), groups, top_groups, group_best, score, norm, scale)
    np.testing.assert_array_equal(host(ids), want_ids)
    near(host(w), want_w, ref.topk_slack(host(l), want_ids, want_w))


# tokens, experts, k, groups, top groups
SHAPES = [(1, 1, 1, 1, 1), (5, 2, 2, 1, 1), (3, 7, 3, 1, 1), (9, 8, 2, 4, 2), (33, 64, 8, 1, 1), (4, 64, 6, 8, 3), (7, 60, 4, 6, 2), (6, 65, 8, 5, 2),
          (5, 100, 7, 10, 4), (130, 128, 8, 1, 1), (3, 160, 6, 8, 3), (70, 256, 8, 8, 4), (2, 255, 9, 1, 1), (3, 384, 8, 64, 9),
          (4, 512, 22, 16, 3), (3, 1000, 32, 1, 1), (5, 1024, 8, 32, 1), (2, 1024, 32, 64, 2)]


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups", SHAPES)
def test_topk(env, T, E, k, groups, top_groups, score, fmt):
    r = np.random.default_rng(T + E + k)
    logits, bias = r.standard_normal((T, E)) * 1.5, r.standard_normal(E) * 0.05
    for norm in (0, 1):
        for b in (None, bias, np.zeros(E)):
            for best in (1, 2) if groups > 1 else (1,):
                _check(env, logits, fmt, k, b, groups, top_groups, best, score, norm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(env, score):
    r = np.random.default_rng(2)
    _check(env, r.standard_normal((3000, 256)), "bf16", 8, r.standard_normal(256) * 0.05, 8, 4, 2, score, 1, 2.5)
    _check(env, r.standard_normal((3001, 96)), "f32", 4, r.standard_normal(96) * 0.05, 1, 1, 1, score, 0)


@FMT
@pytest.mark.parametrize("bias", [False, True])
def test_ties(env, bias, fmt):
    """Few different logits and biases: ties everywhere, in the choice and between groups."""
    r = np.random.default_rng(3)
    for T, E, k, groups, top in ((50, 64, 8, 1, 1), (50, 64, 8, 8, 3), (20, 200, 16, 4, 2), (1, 1024, 32, 64, 4)):
        logits = r.integers(-1, 2, (T, E)) * 0.5
        for best in (1, 2):
            _check(env, logits, fmt, k, r.integers(0, 2, E) * 0.25 if bias else None, groups, top, best, "sigmoid")
    _check(env, np.zeros((3, 40)), fmt, 5, np.zeros(40) if bias else None, 8, 2, 2)
    _check(env, np.where(r.integers(0, 2, (9, 40)) > 0, 0.0, -0.0), fmt, 5, np.zeros(40) if bias else None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_closer_than_fp32_tells(env, score):
    """Logits a unit or so of FP32 apart with biases that all but undo it: FP32 sums tie or swap, 64 bits decide."""
    r = np.random.default_rng(4)
    T, E = 200, 64
    base = r.standard_normal((T, 1))
    logits = (base + r.integers(-40, 41, (T, E)) * 2.0**-24).astype(np.float32).astype(np.float64)
    bias = (r.integers(-2, 3, E) * 2.0**-24).astype(np.float32).astype(np.float64)
    _check(env, logits, "f32", 8, bias, 1, 1, 1, score)
    _check(env, logits, "f32", 8, bias, 8, 3, 2, score)
    _check(env, logits, "f32", 8, None, 8, 3, 2, score)
    _check(env, logits, "f32", 8, bias + 1000.0, 8, 3, 1, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_far_apart(env, score):
    """Biases that spread the choices over many times the scores' range: clusters a few units of FP32 wide, whole units
    below the largest choice and beside numbers far below them, with and without a large offset."""
    r = np.random.default_rng(9)
    T, E = 400, 128
    for offset in (0.0, 37.0, -900.0):
        for down in (1.0, 2.0, 2.0 + 2.0**-20, 5.0, 16.0):
            logits = np.where(r.random((T, E)) < 0.5, 0.0, r.integers(-20, 21, (T, E)) * 2.0**-22).astype(np.float32).astype(np.float64)
            bias = offset - down + r.integers(-6, 7, E) * 2.0**-22
            bias[r.permutation(E)[:4]] = offset
            bias[r.permutation(E)[:60]] -= 50.0
            bias = bias.astype(np.float32).astype(np.float64)
            for k in (3, 6, 12, 20):
                _check(env, logits, "f32", k, bias, 1, 1, 1, score)
            _check(env, logits, "f32", 6, bias, 8, 3, 2, score)
            _check(env, logits, "bf16", 6, bias, 4, 2, 1, score)
    logits = r.standard_normal((T, E)) * 30
    logits[:, ::3] = np.round(logits[:, ::3])
    _check(env, logits, "f32", 14, None, 1, 1, 1, score)
    _check(env, logits, "f32", 30, None, 8, 4, 1, score)


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(env, score, fmt):
    """-inf, and the type's lowest number, for experts that are not to be chosen; rows that have too few others, or none."""
    r = np.random.default_rng(5)
    low = {"f16": -65504.0, "bf16": -3.3895313892515355e38, "f32": -3.4028234663852886e38}[fmt]
    for mask in (-INF, low):
        logits = r.standard_normal((12, 48))
        logits[:, r.permutation(48)[:30]] = mask
        logits[3, 5:] = mask
        logits[4] = mask
        for norm in (0, 1):
            _check(env, logits, fmt, 6, None, 1, 1, 1, score, norm)
            _check(env, logits, fmt, 6, None, 6, 2, 1, score, norm)
            _check(env, logits, fmt, 6, r.standard_normal(48) * 0.05, 6, 2, 2, score, norm)
    bias = np.where(np.arange(48) % 3 == 0, -INF, 0.1)
    _check(env, r.standard_normal((12, 48)), fmt, 6, bias, 1, 1, 1, score)


@FMT
def test_far_logits(env, fmt):
    """Scores that leave FP32's range keep their ratios where they are normalised."""
    r = np.random.default_rng(6)
    logits = r.standard_normal((20, 16)) * 3 - 150
    logits[10:] += 300
    for score in ("softmax", "sigmoid"):
        _check(env, logits, fmt, 4, None, 1, 1, 1, score, 1)


@FMT
def test_not_finite(env, fmt):
    """NaN ranks last and spreads as the formula has it; ids are always different experts; other tokens do not change."""
    r = np.random.default_rng(7)
    logits = r.standard_normal((6, 64))
    clean = [env.call("route_topk", fmt)(env.device(logits, fmt), 4, score=s) for s in ("softmax", "sigmoid")]
    logits[1, 10], logits[3] = np.nan, np.nan
    logits[4, [5, 9]] = INF
    l = env.device(logits, fmt)
    for (cid, cw), score in zip(clean, ("softmax", "sigmoid")):
        ids, w = env.call("route_topk", fmt)(l, 4, score=score)
        assert env.torch.equal(ids[[0, 2, 5]], cid[[0, 2, 5]]) and env.torch.equal(w[[0, 2, 5]], cw[[0, 2, 5]])
        assert 10 not in ids[1].tolist() and ids[3].tolist() == [0, 1, 2, 3] and ids[4, :2].tolist() == [5, 9]
        assert env.torch.isnan(w[3]).all()
        if score == "softmax":
            assert env.torch.isnan(w[[1, 4]]).all()
        else:
            assert not env.torch.isnan(w[[1, 4]]).any()
        for bias in (None, env.device(r.standard_normal(64) * 0.1)):
            for groups, top, best in ((1, 1, 1), (8, 2, 2)):
                ids = host(env.call("route_topk", fmt)(l, 16, bias, groups, top, best, score)[0])
                assert ((ids >= 0) & (ids < 64)).all() and all(len(set(row)) == 16 for row in ids)


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_bias(env, score, fmt):
    """An expert whose bias is NaN ranks below all others, far ones and those with a bias of -inf too, in the choice and in
    its group; its weight is that of its score."""
    r = np.random.default_rng(10)
    for E, groups, top in ((4, 1, 1), (48, 6, 2), (60, 5, 4), (600, 4, 1)):
        logits = r.standard_normal((9, E))
        for others in (0.1, -200.0, -INF):
            bias = np.full(E, others)
            bias[r.permutation(E)[: E // 4]] = 0.2
            bias[r.permutation(E)[: E // 2]] = np.nan
            bias[0] = np.nan
            for k in (3, min(E // groups * top, 13)):
                _check(env, logits, fmt, k, bias, 1, 1, 1, score)
                if groups > 1:
                    _check(env, logits, fmt, k, bias, groups, top, 1, score)
                    _check(env, logits, fmt, k, bias, groups, top, 2, score)
    _check(env, logits, fmt, 5, np.full(E, np.nan), 4, 2, 2, score)


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (9, 64, 8), (4, 100, 6), (130, 128, 6), (3, 255, 8), (6, 512, 32), (3, 1000, 9), (2, 1024, 8)])
def test_gradient(env, T, E, k, score, fmt):
    r = np.random.default_rng(T + E)
    l = env.device(r.standard_normal((T, E)) * 1.5, fmt)
    g = env.device(r.standard_normal((T, k)))
    for norm in (0, 1):
        ids, _ = env.call("route_topk", fmt)(l, k, score=score, norm=norm, scale=2.5)
        out = env.torch.full((T, E), 7.0, device="cuda").to(env.types[fmt])
        got = env.call("route_topk_grad", fmt)(l, ids, g, score, norm, 2.5, out)
        want, slack = ref.topk_grad(host(l), host(ids).astype(np.int64), host(g), score, norm, 2.5)
        near(host(got), want, ref.rounded(want, slack, fmt) if fmt != "f32" else slack)


def test_gradient_far_masked_and_left_out(env):
    t = env.torch
    r = np.random.default_rng(8)
    l = r.standard_normal((6, 40))
    l[1] -= 200
    l[2, 6:] = -INF
    l[3] = -INF
    logits = env.device(l)
    g = env.device(r.standard_normal((6, 4)))
    for score in ("softmax", "sigmoid"):
        for norm in (False, True):
            ids, _ = env.gt.route_topk_f32(logits, 4, score=score, norm=norm)
            d = env.gt.route_topk_grad_f32(logits, ids, g, score, norm)
            assert t.isfinite(d).all() and not d[3].any() and not d[2, 6:].any()
            live = [0, 1, 2, 4, 5]
            want, slack = ref.topk_grad(np.where(np.isinf(l), -1e4, host(logits))[live], host(ids)[live].astype(np.int64), host(g)[live],
                                        score, int(norm), 1.0)
            near(host(d)[live], want, np.where(np.isinf(l[live]), 0, slack))
            ids2 = ids.clone()
            ids2[:, 1], ids2[0, 2] = -1, 40
            d2 = env.gt.route_topk_grad_f32(logits[:1].contiguous(), ids2[:1, [0, 3]].contiguous(), g[:1, [0, 3]].contiguous(), score, norm)
            assert t.equal(env.gt.route_topk_grad_f32(logits, ids2, g, score, norm)[:1], d2)


# ---- sort ------------------------------------------------------------------------
def _sort(env, ids, E, **kw):
    T, k = ids.shape
    space = env.gt.alloc_route_sort_workspace(T, E, k, "cuda").fill_(255)
    offsets, pos = env.gt.route_sort(env.whole(ids), E, workspace=space, **kw)
    want_offsets, want_pos = ref.sort_slots(ids, E)
    np.testing.assert_array_equal(host(offsets), want_offsets)
    np.testing.assert_array_equal(host(pos), want_pos)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (27, 8, 64), (63, 1, 3), (65, 3, 1000), (255, 8, 256), (256, 8, 1024), (257, 8, 1024), (513, 8, 1024),
                                   (4097, 1, 17), (9000, 8, 256), (16384, 8, 256), (40000, 6, 1024), (300000, 1, 2)])
def test_sort(env, T, k, E):
    r = np.random.default_rng(T + E)
    _sort(env, r.integers(0, E, (T, k)).astype(np.int32), E)
    _sort(env, np.minimum(r.geometric(min(0.9, 3 / E), (T, k)) - 1, E - 1).astype(np.int32), E)
    _sort(env, np.full((T, k), E - 1, np.int32), E)


@pytest.mark.parametrize("T", [40, 5000])
def test_sort_of_some_experts(env, T):
    """Ids below 0 and from E on (experts of another card) get no row."""
    r = np.random.default_rng(T)
    _sort(env, r.integers(-3, 40, (T, 4)).astype(np.int32), 32)
    _sort(env, r.choice(np.array([-(1 << 31), -1, 5, 31, 32, (1 << 31) - 1], np.int32), (T, 4)), 32)
    _sort(env, np.full((T, 4), -1, np.int32), 32)


def test_sort_into_given_and_of_nothing(env):
    t = env.torch
    pos = t.full((12, 2), 77, dtype=t.int32, device="cuda")
    offsets = t.full((6,), 77, dtype=t.int32, device="cuda")
    ids = np.random.default_rng(1).integers(0, 3, (10, 2)).astype(np.int32)
    _sort(env, ids, 3, offsets=offsets[1:5], pos=pos[1:11])
    assert (pos[[0, 11]] == 77).all() and (offsets[[0, 5]] == 77).all()
    got, none = env.gt.route_sort(t.empty(0, 2, dtype=t.int32, device="cuda"), 4, offsets[:5])
    assert not got.any() and none.shape == (0, 2)


def test_refusals(env):
    t = env.torch
    l = t.zeros(3, 16, device="cuda")
    with pytest.raises(ValueError, match="score"):
        env.gt.route_topk_f32(l, 2, score="tanh")
    with pytest.raises(ValueError, match="k must be"):
        env.gt.route_topk_f32(l, 17)
    with pytest.raises(ValueError, match="bias"):
        env.gt.route_topk_f32(l, 2, l[0, :8].contiguous())
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.route_topk_f32(l, 8, None, 4, 1)
    with pytest.raises(env.gt.GemvTileError, match="UNSUPPORTED"):
        env.gt.route_topk_f32(t.zeros(2, 1100, device="cuda"), 2)
    with pytest.raises(TypeError):
        env.gt.route_topk_f16(l, 2)
    ids = t.zeros(1025, 2, dtype=t.int32, device="cuda")
    with pytest.raises(env.gt.GemvTileError, match="INVALID"):
        env.gt.route_sort(ids, 4)
    with pytest.raises(ValueError):
        env.gt.route_topk_grad_f32(l, ids, l)
    with pytest.raises(TypeError):
        env.gt.route_sort(ids.long(), 4)
