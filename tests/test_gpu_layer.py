"""The operators around the products run together with them, as a model runs them: a mixture of experts forwards and
backwards in 16 bits and forwards in 8, a decode step on 4-bit weights; eager, on another stream and in a graph."""
import numpy as np
import pytest

import layer_reference as ref
from blocks_reference import HALF_STEP
from layer_env import Env, host

pytestmark = pytest.mark.gpu
T, K, N, E, TOP = 90, 256, 320, 16, 4
EPS = 1e-5


@pytest.fixture(scope="module")
def env():
    return Env()


def _model(env, fmt, tokens=T):
    r = np.random.default_rng(11)
    return {name: env.device(v, fmt) for name, v in {
        "x": r.standard_normal((tokens, K)), "residual": r.standard_normal((tokens, K)), "gain": 1 + 0.1 * r.standard_normal(K),
        "router": r.standard_normal((E, K)) * K**-0.5, "up": r.standard_normal((E, N, K)) * K**-0.5,
        "down": r.standard_normal((E, K, N)) * N**-0.5, "dY": r.standard_normal((tokens, K)) * 0.1}.items()}


def _forward(env, m, fmt, space):
    """Everything that the backward pass needs, by name."""
    gt, t = env.gt, env.torch
    rstd = t.empty(m["x"].shape[0], device="cuda")
    y, h = env.call("rmsnorm", fmt)(m["x"], m["gain"], m["residual"], EPS, rstd=rstd)
    logits = env.call("gemm", fmt)(y, m["router"])
    ids, w = env.call("route_topk", fmt)(logits, TOP)
    offsets, pos = gt.route_sort(ids, E, workspace=space)
    xs = env.call("route_gather", fmt)(y, pos)
    up = env.call("gemm_grouped", fmt)(xs, m["up"], offsets)
    down = env.call("gemm_grouped", fmt)(up, m["down"], offsets)
    out = env.call("route_combine", fmt)(down, pos, w)
    return dict(rstd=rstd, y=y, h=h, logits=logits, ids=ids, w=w, offsets=offsets, pos=pos, xs=xs, up=up, down=down, out=out)


def _backward(env, m, f, fmt, space):
    d_down, dw = env.call("route_combine_grad", fmt)(m["dY"], f["down"], f["pos"], f["w"])
    d_up = env.call("gemm_grouped_dgrad", fmt)(d_down, m["down"], f["offsets"])
    g_down = env.call("gemm_grouped_wgrad", fmt)(d_down, f["up"], f["offsets"])
    d_xs = env.call("gemm_grouped_dgrad", fmt)(d_up, m["up"], f["offsets"])
    g_up = env.call("gemm_grouped_wgrad", fmt)(d_up, f["xs"], f["offsets"])
    d_y = env.call("route_combine", fmt)(d_xs, f["pos"])
    d_logits = env.call("route_topk_grad", fmt)(f["logits"], f["ids"], dw)
    dx, g_gain = env.call("rmsnorm_grad", fmt)(d_y, f["h"], m["gain"], f["rstd"], m["dY"], workspace=space)
    return dict(dw=dw, d_logits=d_logits, d_y=d_y, dx=dx, g_gain=g_gain, g_up=g_up, g_down=g_down)


def _reference(env, m, ids):
    """The same layer in 64 bits with autograd on the CPU (the experts' part of the gradient of y alone, as above)."""
    t = env.torch
    d = {k: v.detach().cpu().double() for k, v in m.items()}
    for k in ("gain", "up", "down"):
        d[k].requires_grad_()
    h = (d["x"] + d["residual"]).to(m["x"].dtype).double().requires_grad_()
    y = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * d["gain"]
    y.retain_grad()
    logits = (y.detach() @ d["router"].t()).requires_grad_()
    w = t.softmax(logits.gather(1, ids), 1)
    out = t.zeros(*h.shape, dtype=t.float64)
    for j in range(TOP):
        for e in range(E):
            rows = (ids[:, j] == e).nonzero()[:, 0]
            if len(rows):
                out = out.index_add(0, rows, w[rows, j, None] * (y[rows] @ d["up"][e].t() @ d["down"][e].t()))
    ((out + h) * d["dY"]).sum().backward()
    return dict(out=out, d_logits=logits.grad, d_y=y.grad, dx=h.grad, g_gain=d["gain"].grad, g_up=d["up"].grad, g_down=d["down"].grad)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_mixture_of_experts(env, fmt):
    """Each of a result's at most 8 roundings to 16 bits on the way is off by half a step of the intermediate; they add up
    at random, so that 8 half steps of the root mean square bound the root mean square of the error."""
    m = _model(env, fmt)
    f = _forward(env, m, fmt, None)
    b = _backward(env, m, f, fmt, env.gt.alloc_rmsnorm_grad_workspace(f["h"]))
    ids = f["ids"].cpu().long()
    want = _reference(env, m, ids)
    for name, got in {"out": f["out"], **{k: b[k] for k in want if k != "out"}}.items():
        w = want[name].detach().numpy()
        error = np.sqrt(np.mean((host(got) - w) ** 2)) / np.sqrt(np.mean(w**2))
        assert error <= 8 * HALF_STEP[fmt], (name, error)
    counts = np.bincount(ids.numpy().reshape(-1), minlength=E)
    np.testing.assert_array_equal(host(f["offsets"]), np.concatenate([[0], np.cumsum(counts)]))


def test_in_8_bits(env):
    """Norm, gather and grouped product in 8 bits against the same numbers widened."""
    m = _model(env, "bf16")
    gt, t = env.gt, env.torch
    y = t.empty_like(m["x"])
    q, s, h = gt.rmsnorm_fp8_bf16(m["x"], m["gain"], m["residual"], EPS, y=y)
    ids, w = gt.route_topk_bf16(gt.gemm_bf16(y, m["router"]), TOP, score="sigmoid", scale=2.5)
    offsets, pos = gt.route_sort(ids, E)
    xs, ss = gt.route_gather_fp8(q, s, pos)
    wq, ws = gt.quantize_fp8_tiles_bf16(m["up"])
    d = gt.gemm_grouped_fp8_bf16(xs, ss, wq, ws, offsets)
    a = host(q.float()) * np.repeat(host(s), 128, 1)
    scale = np.repeat(np.repeat(host(ws), 128, 1)[:, :N], 128, 2)[:, :, :K]
    b = host(wq.float()) * scale
    got, at = host(d), host(pos)
    for i in range(T):
        for j in range(TOP):
            e = int(ids[i, j])
            want, terms = a[i] @ b[e].T, np.abs(a[i]) @ np.abs(b[e]).T
            assert (np.abs(got[at[i, j]] - want) <= HALF_STEP["bf16"] * np.abs(want) + 2.0**-10 * terms).all()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_decode_on_4_bits(env, fmt):
    """One token and a few through a norm and a 4-bit projection."""
    m = _model(env, fmt)
    wq, ws = env.call("quantize_fp4", fmt)(m["up"][0])
    for tokens in (1, 5):
        y, _ = env.call("rmsnorm", fmt)(m["x"][:tokens].contiguous(), m["gain"], m["residual"][:tokens].contiguous(), EPS)
        got = env.call("gemv_fp4", fmt)(y, wq, ws)
        want, tol = ref.gemv_fp4(host(y), host(wq), host(ws), fmt)
        assert (np.abs(host(got) - want) <= tol).all()


def _everything(env, m, fmt, sort_space, norm_space):
    f = _forward(env, m, fmt, sort_space)
    b = _backward(env, m, f, fmt, norm_space)
    q, s, _ = env.call("rmsnorm_fp8", fmt)(m["x"], m["gain"], m["residual"], EPS)
    xs, ss = env.gt.route_gather_fp8(q, s, f["pos"])
    wq, ws = env.call("quantize_fp4", fmt)(m["up"])
    y4 = env.call("gemv_fp4", fmt)(f["y"][:20].contiguous(), wq[1], ws[1])
    return {**f, **b, "q": q.view(env.torch.uint8), "s": s, "xs8": xs.view(env.torch.uint8), "ss": ss, "wq": wq, "ws": ws, "y4": y4}


def _same(env, a, b):
    for k in a:
        assert env.torch.equal(a[k].view(env.torch.uint8), b[k].view(env.torch.uint8)), k


@pytest.mark.parametrize("tokens", [40, 1100])
def test_graph_and_stream(env, tokens):
    """Captured and replayed with new inputs, eager work in between, and on a stream of its own: bit for bit the eager
    results.  1100 tokens sort in two launches with a workspace."""
    t = env.torch
    m = _model(env, "bf16", tokens)
    sort_space = env.gt.alloc_route_sort_workspace(tokens, E, TOP, "cuda")
    norm_space = env.gt.alloc_rmsnorm_grad_workspace(m["x"])
    want = _everything(env, m, "bf16", sort_space, norm_space)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        got = _everything(env, m, "bf16", sort_space, norm_space)
    side.synchronize()
    _same(env, want, got)
    own = [env.gt.alloc_route_sort_workspace(tokens, E, TOP, "cuda"), env.gt.alloc_rmsnorm_grad_workspace(m["x"])]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        held = _everything(env, m, "bf16", *own)
    for seed in range(3):
        g = t.Generator("cuda").manual_seed(seed)
        for name in ("x", "residual", "dY"):
            m[name].copy_(t.randn(m[name].shape, device="cuda", generator=g))
        for v in own:
            v.fill_(255)
        want = _everything(env, m, "bf16", sort_space, norm_space)
        graph.replay()
        t.cuda.synchronize()
        _same(env, want, held)
