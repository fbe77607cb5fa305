"""How exactly the streamed 8-bit products add a block's 128 terms: in FP32, beside terms that cancel.

Tolerance: terms are exact; n of them are added one after another in FP32 with at most 2^-23 of a partial sum lost each
time, so |error| <= n 2^-23 S for a sum S of their absolute values; a block's sum is scaled with two roundings and added
with one; then the result is rounded to 16 bits (blocks_reference.rounded)."""
import numpy as np
import pytest

from blocks_reference import e4m3_values, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import gemv_tile_pipelined_amd as gt

    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    gt.load_library()
    return torch, gt


def _cancelling(torch, seed, M, N, K):
    """Operands whose blocks hold 448 x 448 and 448 x -448, at places that change, and small terms."""
    g = np.random.default_rng(seed)
    a, b = g.uniform(0.5, 2, (M, K)), g.uniform(0.5, 2, (N, K))
    for k0 in range(0, K, 128):
        i, j = k0 + g.permutation(min(128, K - k0))[:2]
        a[:, i] = a[:, j] = b[:, i] = 448
        b[:, j] = -448
    q = [torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn) for v in (a, b)]
    return q, [e4m3_values(t.view(torch.uint8).numpy()) for t in q]


def _want(a, sa, b, sb, fmt):
    """The product and its tolerance: sa [M, blocks], sb [N, blocks] in 64 bits."""
    v, slack, total = 0.0, 0.0, 0.0
    for k in range(0, a.shape[1], 128):
        cut, scale = slice(k, k + 128), np.outer(sa[:, k // 128], sb[:, k // 128])
        s = (np.abs(a[:, cut]) @ np.abs(b[:, cut]).T) * scale
        v = v + (a[:, cut] @ b[:, cut].T) * scale
        total = total + s
        slack = slack + a[:, cut].shape[1] * 2.0**-23 * s + 2 * 2.0**-24 * s + 2.0**-24 * total
    return v, rounded(v, slack, fmt)


def _check(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, worst {np.abs(got - want)[bad].max()}"


SHAPES = [(1, 300, 400), (1, 17, 4112), (2, 1, 16), (3, 2998, 272), (4, 130, 2064)]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense(env, M, N, K, rows):
    torch, gt = env
    (A, B), (a, b) = _cancelling(torch, M, M, N, K)
    g = np.random.default_rng(N)
    kb = -(-K // 128)
    sa = np.exp2(g.uniform(-3, 0, (M, kb))).astype(np.float32)
    sb = np.exp2(g.uniform(-3, 0, (-(-N // rows), kb))).astype(np.float32)
    fmt = "bf16" if M % 2 else "f16"
    D = getattr(gt, f"gemm_fp8_{fmt}")(*[t.cuda() for t in (A, torch.from_numpy(sa), B, torch.from_numpy(sb))])
    _check(D.double().cpu().numpy(), *_want(a, sa.astype(float), b, sb.astype(float).repeat(rows, 0)[:N], fmt))


@pytest.mark.parametrize("sizes,N,blocks", [([1, 0, 2, 1], 130, 1), ([9, 3] * 40, 1040, 2), ([0, 17, 0, 1] * 30, 1000, 2)])
def test_grouped(env, sizes, N, blocks):
    torch, gt = env
    T, E, K = sum(sizes), len(sizes), 400
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_stream_blocks("fp8", T, N, K, E, cus) == blocks
    (X, W), (x, w) = _cancelling(torch, E, T, E * N, K)
    g = np.random.default_rng(T)
    sx = np.exp2(g.uniform(-3, 0, (T, 4))).astype(np.float32)
    sw = np.exp2(g.uniform(-3, 0, (E, -(-N // 128), 4))).astype(np.float32)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    D = gt.gemm_grouped_fp8_f16(*[t.cuda() for t in (X, torch.from_numpy(sx), W.view(E, N, K), torch.from_numpy(sw),
                                                     torch.from_numpy(off))]).double().cpu().numpy()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if sizes[e]:
            _check(D[r], *_want(x[r], sx[r].astype(float), w[e * N : (e + 1) * N], sw[e].astype(float).repeat(128, 0)[:N], "f16"))
