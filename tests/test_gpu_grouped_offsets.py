"""Offsets that are not non-decreasing or leave the rows: what each row of the output holds.

A group owns the rows from its offset, kept within 0 .. T, to the next one's, kept within its own first row .. T.  Rows that
one group owns are that group's product, elements of rows that several own are one of theirs, and rows of no group stay as
they were."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import gemv_tile_pipelined_amd as gt

    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    gt.load_library()
    return torch, gt


def _owned(offsets, T):
    first = [min(max(o, 0), T) for o in offsets]
    return [(a, max(a, b)) for a, b in zip(first[:-1], first[1:])]


MARK = 0.5


def _product(env, op, offsets, T, N, K, kind):
    """Ones times a weight of e + 1 in group e: rows of group e hold (terms of the sum) * (e + 1), exactly."""
    torch, gt = env
    E = len(offsets) - 1
    assert gt.grouped_plan(op, T, N, K, E, 256)[0] == kind
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    W = torch.arange(1, E + 1, device="cuda").half().view(E, 1, 1).expand(E, N, K).contiguous()
    out = torch.full((3, T, K if op == "dgrad" else N), MARK, device="cuda").half()
    X = torch.ones(T, N if op == "dgrad" else K, device="cuda").half()
    if op == "fp8":
        e4m3, kb = torch.float8_e4m3fn, -(-K // 128)
        gt.gemm_grouped_fp8_f16(X.to(e4m3), torch.ones(T, kb, device="cuda"), W.to(e4m3),
                                torch.ones(E, -(-N // 128), kb, device="cuda"), off, out[1])
    else:
        (gt.gemm_grouped_dgrad_f16 if op == "dgrad" else gt.gemm_grouped_f16)(X, W, off, out[1])
    torch.cuda.synchronize()
    assert (out[0] == MARK).all() and (out[2] == MARK).all(), "outside of the output"
    terms, owned, rows = (N if op == "dgrad" else K), _owned(offsets, T), out[1]
    right = torch.zeros_like(rows, dtype=torch.bool)
    free = torch.ones(T, 1, dtype=torch.bool, device="cuda")
    for e, (a, b) in enumerate(owned):
        right[a:b] |= rows[a:b] == terms * (e + 1)
        free[a:b] = False
    right |= free & (rows == MARK)
    assert right.all(), f"rows {(~right).any(1).nonzero().flatten().tolist()[:20]} of {owned}"


def _wild(T):
    return [-7, 2, 1, 4, 1 << 30, T + 5, -(1 << 31)]


@pytest.mark.parametrize("op,T,kind", [("forward", 5, "deep"), ("fp8", 5, "deep"), ("forward", 4, "stream"), ("fp8", 4, "stream"),
                                       ("dgrad", 5, "tiled"), ("forward", 400, "deep"), ("fp8", 400, "deep"),
                                       ("dgrad", 400, "tiled")])
def test_few_tiles(env, op, T, kind):
    _product(env, op, _wild(T), T, 32, 48, kind)


TILES = [_wild(3000), [2000, 0, 2900, 100, 3000, 50, 3000], [3000] * 7, [0, 3000, 0, 3000, 0, 3000, 0],
         [0, 900, 700, 1400, 1300, 3000, 2999]]
IDS = ["wild", "back", "none", "all", "overlapping"]


@pytest.mark.parametrize("op", ["forward", "dgrad", "fp8"])
@pytest.mark.parametrize("offsets", TILES, ids=IDS)
def test_many_tiles(env, op, offsets):
    _product(env, op, offsets, 3000, 48 if op == "dgrad" else 4096, 4096 if op == "dgrad" else 48, "tiled")


@pytest.mark.parametrize("T,N,K,offsets", [(5, 32, 48, _wild(5)), (400, 32, 48, _wild(400))]
                         + [(3000, 2048, 1032, o) for o in TILES] + [(3000, 264, 272, o) for o in TILES])
def test_weight_gradient(env, T, N, K, offsets):
    """A group's gradient of ones is the number of its rows, whatever other groups own them too."""
    torch, gt = env
    E = len(offsets) - 1
    out = torch.full((3, E, N, K), MARK, device="cuda").half()
    gt.gemm_grouped_wgrad_f16(torch.ones(T, N, device="cuda").half(), torch.ones(T, K, device="cuda").half(),
                              torch.tensor(offsets, dtype=torch.int32, device="cuda"), out[1])
    torch.cuda.synchronize()
    assert (out[0] == MARK).all() and (out[2] == MARK).all(), "outside of the output"
    for e, (a, b) in enumerate(_owned(offsets, T)):
        assert (out[1, e] == float(np.float16(b - a))).all(), (e, a, b)
