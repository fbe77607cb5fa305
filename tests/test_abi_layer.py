"""The argument checks of the operators around the products, on the CPU: every refusal comes before any HIP call."""
import os

import pytest

import gemv_tile_pipelined_amd as gt

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # a 16-byte aligned address; never dereferenced by these calls
FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gt.LIBRARY_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return gt.load_library()


def _pointers(f, n, rest, needed, align):
    """NULL for a needed pointer is invalid, a misaligned one unsupported; `align` by pointer."""
    for i in range(n):
        args = [None if j == i else P for j in range(n)]
        if i in needed:
            assert f(*args, *rest, None) == INVALID, i
        if align[i] > 1:
            assert f(*[P + align[i] // 2 if j == i else P for j in range(n)], *rest, None) == UNSUPPORTED, i


@FMT
def test_quantize_fp4(lib, fmt):
    f = getattr(lib, f"quantize_fp4_{fmt}")
    assert f(None, None, None, 0, 32, None) == OK and f(None, None, None, 4, 0, None) == OK
    assert f(P, P, P, -1, 32, None) == INVALID and f(P, P, P, 1, -32, None) == INVALID
    _pointers(f, 3, (4, 32), {0, 1, 2}, (16, 16, 1))
    assert f(P, P, P, 4, 48, None) == UNSUPPORTED
    assert f(P, P, P, (1 << 31) - 1, 64, None) == UNSUPPORTED
    assert f(P, P, P, 1 << 60, 1 << 60, None) == UNSUPPORTED


@FMT
def test_gemv_fp4(lib, fmt):
    f = getattr(lib, f"gemv_fp4_{fmt}")
    assert f(*[None] * 4, 0, 4, 32, None) == OK and f(*[None] * 4, 4, 0, 32, None) == OK
    for sizes in ((-1, 4, 32), (4, -1, 32), (4, 4, -32)):
        assert f(*[P] * 4, *sizes, None) == INVALID
    _pointers(f, 4, (1, 4, 32), {0, 1, 2, 3}, (16, 16, 1, 2))
    assert f(None, None, None, None, 1, 4, 0, None) == INVALID
    for sizes in ((1, 4, 48), ((1 << 19) + 1, 4, 32), (1, (1 << 25) + 1, 32), (1, 4, 4194304)):
        assert f(*[P] * 4, *sizes, None) == UNSUPPORTED


@FMT
def test_rmsnorm(lib, fmt):
    f = getattr(lib, f"rmsnorm_{fmt}")
    assert f(*[None] * 6, 0, 16, 0.0, None) == OK and f(*[None] * 6, 4, 0, 0.0, None) == OK
    for bad in ((-1, 16, 0.0), (4, -16, 0.0), (4, 16, -1e-6), (4, 16, float("nan"))):
        assert f(*[P] * 6, *bad, None) == INVALID
    # x, residual, weight, h, y, rstd: residual and h come together
    _pointers(f, 6, (4, 16, 1e-6), {0, 1, 2, 3, 4}, (16, 16, 16, 16, 16, 4))
    assert f(*[P] * 6, 4, 12, 1e-6, None) == UNSUPPORTED
    assert f(*[P] * 6, 4, 32776, 1e-6, None) == UNSUPPORTED
    assert f(*[P] * 6, (1 << 31) - 511, 16, 1e-6, None) == UNSUPPORTED


@FMT
def test_rmsnorm_fp8(lib, fmt):
    f = getattr(lib, f"rmsnorm_fp8_{fmt}")
    assert f(*[None] * 8, 0, 16, 0.0, None) == OK
    # x, residual, weight, h, y, q, scale, rstd
    _pointers(f, 8, (4, 16, 1e-6), {0, 1, 2, 3, 5, 6}, (16, 16, 16, 16, 16, 16, 4, 4))
    assert f(*[P] * 8, 4, 24, 1e-6, None) == UNSUPPORTED


@FMT
def test_rmsnorm_grad(lib, fmt):
    f = getattr(lib, f"rmsnorm_grad_{fmt}")
    need = lib.gemvtile_rmsnorm_grad_workspace(4, 16)
    assert need == 4 * 4 * 16 and lib.gemvtile_rmsnorm_grad_workspace(1 << 20, 4096) == 4 * 512 * 4096
    assert lib.gemvtile_rmsnorm_grad_workspace(0, 16) == 0 == lib.gemvtile_rmsnorm_grad_workspace(4, 1 << 20)
    assert f(*[None] * 7, 4, 0, None, 0, None) == OK
    for bad in ((-1, 16), (4, -16)):
        assert f(*[P] * 7, *bad, P, need, None) == INVALID
    assert f(*[P] * 7, 4, 16, P, -1, None) == INVALID
    assert f(*[P] * 7, 4, 16, P, need - 1, None) == INVALID and f(*[P] * 7, 4, 16, None, need, None) == INVALID
    assert f(*[P] * 7, 4, 16, P + 8, need, None) == UNSUPPORTED
    # dy, dh, h, weight, rstd, dx, dweight
    _pointers(f, 7, (4, 16, P, need), {0, 2, 3, 4, 5, 6}, (16, 16, 16, 16, 4, 16, 4))
    assert f(*[None] * 6, None, 0, 16, None, 0, None) == INVALID
    assert f(*[P] * 7, 4, 12, P, 1 << 20, None) == UNSUPPORTED


TOPK = {"T": 4, "E": 16, "k": 2, "groups": 4, "top_groups": 2, "group_best": 2, "score": 1, "norm": 1, "scale": 1.0}


@pytest.mark.parametrize("fmt", ["f16", "bf16", "f32"])
def test_route_topk(lib, fmt):
    f = getattr(lib, f"route_topk_{fmt}")

    def call(pointers=(P, P, P, P), **change):
        return f(*pointers, *{**TOPK, **change}.values(), None)

    assert call((None,) * 4, T=0) == OK
    for bad in ({"T": -1}, {"E": 0}, {"k": 0}, {"k": 17, "top_groups": 4}, {"k": 9}, {"groups": 0}, {"groups": 3}, {"top_groups": 0},
                {"top_groups": 5}, {"group_best": 0}, {"group_best": 3}, {"score": 2}, {"score": -1}, {"norm": 2}):
        assert call(**bad) == INVALID, bad
    for i in (0, 2, 3):
        assert call(tuple(None if j == i else P for j in range(4))) == INVALID
    for i, off in ((0, 8), (1, 2), (2, 2), (3, 2)):
        assert call(tuple(P + off if j == i else P for j in range(4))) == UNSUPPORTED
    for bad in ({"E": 1028}, {"T": 1 << 26}, {"E": 128, "groups": 128, "k": 1}, {"E": 64, "groups": 1, "top_groups": 1, "k": 33}):
        assert call(**bad) == UNSUPPORTED, bad


@pytest.mark.parametrize("fmt", ["f16", "bf16", "f32"])
def test_route_topk_grad(lib, fmt):
    f = getattr(lib, f"route_topk_grad_{fmt}")
    good = (4, 16, 2, 0, 1, 1.0)
    assert f(*[None] * 4, 0, *good[1:], None) == OK
    for i, bad in ((0, -1), (1, 0), (2, 0), (2, 17), (3, 2), (4, 2)):
        assert f(*[P] * 4, *[bad if j == i else g for j, g in enumerate(good)], None) == INVALID
    _pointers(f, 4, good, {0, 1, 2, 3}, (16, 4, 4, 16))
    for i, bad in ((0, 1 << 26), (1, 1025)):
        assert f(*[P] * 4, *[bad if j == i else g for j, g in enumerate(good)], None) == UNSUPPORTED


def test_route_sort(lib):
    f = lib.route_sort
    space = lib.gemvtile_route_sort_workspace
    assert space(256, 8, 64) == 0 and space(257, 8, 64) == 4 * 5 * 64 and space(1 << 20, 8, 256) == 4 * 128 * 256
    assert space(-1, 8, 64) == space(8, 0, 64) == space(8, 8, 0) == space(1 << 31, 8, 64) == 0
    for sizes in ((-1, 2, 4), (4, 0, 4), (4, 2, 0)):
        assert f(P, P, P, *sizes, None, 0, None) == INVALID
    for i in range(3):
        assert f(*[None if j == i else P for j in range(3)], 4, 2, 4, None, 0, None) == INVALID
        assert f(*[P + 2 if j == i else P for j in range(3)], 4, 2, 4, None, 0, None) == UNSUPPORTED
    assert f(None, None, None, 0, 2, 4, None, 0, None) == INVALID
    assert f(P, P, P, 4, 2, 4, None, -1, None) == INVALID
    assert f(P, P, P, 4096, 8, 64, None, 0, None) == INVALID
    need = space(4096, 8, 64)
    assert f(P, P, P, 4096, 8, 64, P, need - 1, None) == INVALID
    assert f(P, P, P, 4096, 8, 64, P + 4, need, None) == UNSUPPORTED
    assert f(P, P, P, 4, 2, 1025, None, 0, None) == UNSUPPORTED
    assert f(P, P, P, 1 << 30, 2, 4, P, 1 << 30, None) == UNSUPPORTED


ROWS = (4, 2, 8, 32)  # T, k, R, K


def _row_sizes(f, n, step):
    for i, bad in ((0, -1), (1, 0), (2, -1), (3, -32)):
        assert f(*[P] * n, *[bad if j == i else g for j, g in enumerate(ROWS)], None) == INVALID
    for i, bad in ((0, 1 << 24), (1, 33), (2, 1 << 31), (3, (1 << 20) + 32), (3, 32 + step // 2)):
        assert f(*[P] * n, *[bad if j == i else g for j, g in enumerate(ROWS)], None) == UNSUPPORTED


def test_route_gather(lib):
    for fmt in ("f16", "bf16"):
        f = getattr(lib, f"route_gather_{fmt}")
        for sizes in ((0, 2, 8, 32), (4, 2, 0, 32), (4, 2, 8, 0)):
            assert f(*[None] * 3, *sizes, None) == OK
        _row_sizes(f, 3, 8)
        _pointers(f, 3, ROWS, {0, 1, 2}, (16, 4, 16))
    f = lib.route_gather_fp8
    assert f(*[None] * 5, 0, 2, 8, 32, None) == OK
    _row_sizes(f, 5, 16)
    _pointers(f, 5, ROWS, {0, 1, 2, 3, 4}, (16, 4, 4, 16, 4))


@FMT
def test_route_combine(lib, fmt):
    f = getattr(lib, f"route_combine_{fmt}")
    assert f(*[None] * 4, 0, 2, 8, 32, None) == OK and f(*[None] * 4, 4, 2, 8, 0, None) == OK
    _row_sizes(f, 4, 8)
    _pointers(f, 4, ROWS, {0, 1, 3}, (16, 4, 4, 16))
    f = getattr(lib, f"route_combine_grad_{fmt}")
    assert f(*[None] * 6, 0, 2, 8, 32, None) == OK
    _row_sizes(f, 6, 8)
    _pointers(f, 6, ROWS, {0, 1, 2, 3, 4, 5}, (16, 16, 4, 4, 16, 4))


def test_tensor_checks():
    """Types, shapes and devices are checked before the library is called; a CPU tensor is refused."""
    import torch

    x, i = torch.zeros(4, 32).half(), torch.zeros(4, 2, dtype=torch.int32)
    b = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        gt.quantize_fp4_f16(x)
    with pytest.raises(TypeError, match="x must be"):
        gt.quantize_fp4_bf16(x)
    with pytest.raises(TypeError, match="torch.Tensor"):
        gt.gemv_fp4_f16([1.0], b, b)
    for f in (lambda: gt.gemv_fp4_f16(x, b, b), lambda: gt.rmsnorm_f16(x, x[0]), lambda: gt.rmsnorm_fp8_f16(x, x[0]),
              lambda: gt.rmsnorm_grad_f16(x, x, x[0], x[0]), lambda: gt.route_topk_f16(x, 2), lambda: gt.route_sort(i, 4),
              lambda: gt.route_topk_grad_f16(x, i, x), lambda: gt.route_gather_f16(x, i), lambda: gt.route_combine_f16(x, i),
              lambda: gt.route_combine_grad_f16(x, x, i, x)):
        with pytest.raises(ValueError, match="device tensor"):
            f()


def test_tensor_calls_are_listed():
    assert set(gt.LAYER_CALLS) <= set(gt.EXPORTED_SYMBOLS)
    assert set(gt.LAYER_NAMES) <= set(gt.__all__) and set(gt.LAYER_NAMES) <= set(dir(gt)) and "layer" in dir(gt)
    assert sorted(gt.layer.__all__) == sorted(gt.LAYER_NAMES)
