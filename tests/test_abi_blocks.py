"""The argument checks of the 8-bit and grouped entry points, and the host side of the groups' units, on the CPU: every
refusal comes before any HIP call."""
import itertools
import os
import random

import pytest

import gemv_tile_pipelined_amd as gt

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # a 16-byte aligned address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gt.LIBRARY_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return gt.load_library()


FMT = pytest.mark.parametrize("fmt", ["f16", "bf16"])


@FMT
def test_quantize_rows(lib, fmt):
    f = getattr(lib, f"quantize_fp8_rows_{fmt}")
    assert f(None, None, None, 0, 16, None) == OK
    assert f(None, None, None, 4, 0, None) == OK
    assert f(P, P, P, -1, 16, None) == INVALID and f(P, P, P, 1, -16, None) == INVALID
    for bad in range(3):
        assert f(*[None if i == bad else P for i in range(3)], 4, 16, None) == INVALID
    assert f(P, P, P, 4, 24, None) == UNSUPPORTED
    for bad, off in ((0, 8), (1, 8), (2, 2)):
        assert f(*[P + off if i == bad else P for i in range(3)], 4, 16, None) == UNSUPPORTED
    assert f(P, P, P, (1 << 29) - 31, 16, None) == UNSUPPORTED
    assert f(P, P, P, 1 << 60, 1 << 60, None) == UNSUPPORTED


@FMT
def test_quantize_tiles(lib, fmt):
    f = getattr(lib, f"quantize_fp8_tiles_{fmt}")
    for sizes in ((0, 4, 16), (4, 0, 16), (4, 4, 0)):
        assert f(None, None, None, *sizes, None) == OK
    for sizes in ((-1, 4, 16), (4, -1, 16), (4, 4, -16)):
        assert f(P, P, P, *sizes, None) == INVALID
    for bad in range(3):
        assert f(*[None if i == bad else P for i in range(3)], 1, 4, 16, None) == INVALID
    assert f(P, P, P, 1, 4, 8, None) == UNSUPPORTED
    assert f(P, P + 8, P, 1, 4, 16, None) == UNSUPPORTED
    assert f(P, P, P, 1 << 23, 4, 16, None) == UNSUPPORTED
    assert f(P, P, P, 1 << 60, 1 << 60, 1 << 60, None) == UNSUPPORTED


@FMT
def test_gemm_fp8(lib, fmt):
    f = getattr(lib, f"gemm_fp8_{fmt}")
    assert f(*[None] * 5, 0, 4, 16, 128, None) == OK and f(*[None] * 5, 4, 0, 16, 1, None) == OK
    for sizes in ((-1, 4, 16), (4, -1, 16), (4, 4, -16)):
        assert f(*[P] * 5, *sizes, 128, None) == INVALID
    for rows in (0, -1, 2, 64, 127, 256):
        assert f(*[P] * 5, 4, 4, 16, rows, None) == INVALID
    for bad in range(5):
        assert f(*[None if i == bad else P for i in range(5)], 4, 4, 16, 128, None) == INVALID
    assert f(*[P] * 5, 4, 4, 24, 128, None) == UNSUPPORTED
    assert f(*[P] * 5, (1 << 25) + 1, 4, 16, 128, None) == UNSUPPORTED
    assert f(*[P] * 5, 4, (1 << 25) + 1, 16, 128, None) == UNSUPPORTED
    assert f(*[P] * 5, 4, 4, 4194304, 128, None) == UNSUPPORTED
    for bad, off in ((0, 8), (1, 2), (2, 4), (3, 1), (4, 1)):
        assert f(*[P + off if i == bad else P for i in range(5)], 4, 4, 16, 128, None) == UNSUPPORTED


GROUPED = [("gemm_grouped", 4), ("gemm_grouped_dgrad", 4), ("gemm_grouped_wgrad", 4), ("gemm_grouped_fp8", 6)]


@FMT
@pytest.mark.parametrize("name,n", GROUPED)
def test_grouped(lib, name, n, fmt):
    f = getattr(lib, f"{name}_{fmt}")
    aligned = (32, 32)  # N, K
    assert f(*[None] * n, 8, *aligned, 0, None) == OK
    nothing = {"gemm_grouped": [(0, 32, 32), (8, 0, 32)], "gemm_grouped_fp8": [(0, 32, 32), (8, 0, 32)],
               "gemm_grouped_dgrad": [(0, 32, 32), (8, 32, 0)], "gemm_grouped_wgrad": [(8, 0, 32), (8, 32, 0)]}
    for sizes in nothing[name]:
        assert f(*[None] * n, *sizes, 2, None) == OK
    for sizes in ((-1, 32, 32, 2), (8, -1, 32, 2), (8, 32, -32, 2), (8, 32, 32, -1)):
        assert f(*[P] * n, *sizes, None) == INVALID
    for bad in range(n):
        assert f(*[None if i == bad else P for i in range(n)], 8, *aligned, 2, None) == INVALID
        assert f(*[P + 1 if i == bad else P for i in range(n)], 8, *aligned, 2, None) == UNSUPPORTED
    assert f(*[P] * n, 8, 32, 40 if n == 6 else 36, 2, None) == UNSUPPORTED
    if name in ("gemm_grouped_dgrad", "gemm_grouped_wgrad"):
        assert f(*[P] * n, 8, 36, 32, 2, None) == UNSUPPORTED
    assert f(*[P] * n, 8, *aligned, 1025, None) == UNSUPPORTED
    assert f(*[P] * n, 1 << 31, *aligned, 2, None) == UNSUPPORTED
    assert f(*[P] * n, 8, (1 << 20) + 16, 32, 2, None) == UNSUPPORTED
    assert f(*[P] * n, 8, 32, (1 << 20) + 16, 2, None) == UNSUPPORTED
    if name == "gemm_grouped_wgrad":
        assert f(*[P] * n, 8, 1 << 20, 1 << 20, 1, None) == UNSUPPORTED


def test_tensor_checks():
    """Types, shapes and devices are checked before the library is called; a CPU tensor is refused."""
    import torch

    q = torch.zeros(4, 16).to(torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device tensor"):
        gt.gemm_fp8_f16(q, s, q, s)
    with pytest.raises(TypeError, match="A must be"):
        gt.gemm_fp8_f16(s, s, q, s)
    with pytest.raises(ValueError, match="device tensor"):
        gt.quantize_fp8_rows_f16(torch.zeros(4, 16).half())
    with pytest.raises(TypeError, match="x must be"):
        gt.quantize_fp8_rows_f16(torch.zeros(4, 16))
    with pytest.raises(TypeError, match="torch.Tensor"):
        gt.quantize_fp8_tiles_bf16([1.0])
    for f in (gt.gemm_grouped_f16, gt.gemm_grouped_dgrad_f16, gt.gemm_grouped_wgrad_f16):
        with pytest.raises(ValueError, match="device tensor"):
            f(torch.zeros(4, 16).half(), torch.zeros(1, 16, 16).half(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        gt.gemm_grouped_fp8_bf16(q, s, q[None], s[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(AttributeError):
        gt.gemm_fp4_f16


def _units(offsets, T, rows):
    """Every unit, from the definition."""
    out = []
    for e in range(len(offsets) - 1):
        low = min(max(offsets[e], 0), T)
        high = min(max(offsets[e + 1], low), T)
        out += [(e, t, min(t + rows, high)) for t in range(low, high, rows)]
    return out


def test_units_cover_every_groups_rows(lib):
    r = random.Random(1)
    for _ in range(200):
        E, T, rows = r.choice((1, 2, 5, 64, 65, 1024)), r.randint(0, 600), r.choice((1, 16, 64, 128, 256))
        cuts = sorted(r.randint(0, T) for _ in range(E + 1))
        want = _units(cuts, T, rows)
        got = []
        for u in itertools.count():
            unit = gt.group_unit(cuts, T, rows, u)
            if unit is None:
                break
            got.append(unit[:3])
            assert len(want) <= unit[3], "more units than the launch allows for"
        assert got == want


def test_units_of_unsound_offsets_stay_inside(lib):
    r = random.Random(2)
    for _ in range(300):
        T = r.randint(1, 100)
        cuts = [r.choice((r.randint(-5, T + 5), -(1 << 31), (1 << 31) - 1)) for _ in range(r.randint(2, 9))]
        want = _units(cuts, T, 16)
        for u, unit in enumerate(want):
            e, low, high = gt.group_unit(cuts, T, 16, u)[:3]
            assert (e, low, high) == unit and 0 <= low < high <= T
        assert gt.group_unit(cuts, T, 16, len(want)) is None


def test_unit_bound_is_reached():
    """As many groups of one row as there can be, the rest in one: the launch allows for exactly that many units."""
    for E, T, rows in ((1, 1, 16), (3, 100, 16), (8, 5, 64), (16, 8200, 256), (1024, 4000, 16)):
        some = min(E, T)
        cuts = [0] + [T - some + 1 + i for i in range(some)] + [T] * (E - some)
        assert len(_units(cuts, T, rows)) == gt.group_unit(cuts, T, rows, 0)[3]


def test_grouped_plan(lib):
    assert gt.grouped_plan("forward", 32, 2048, 2048, 64, 256) == ("stream", 16, 16)
    assert gt.grouped_plan("fp8", 8, 4096, 2048, 64, 256) == ("stream", 16, 16)
    for op in gt.GROUPED_OPS:
        kind, rows, cols = gt.grouped_plan(op, 16384, 4096, 4096, 32, 256)
        assert (kind, rows, cols) == ("tiled", 256, 256)
    assert gt.grouped_plan("fp8", 512, 2048, 4096, 8, 256) == ("deep", 128, 64)
    assert gt.grouped_plan("forward", 24, 2048, 2048, 8, 256) == ("deep", 32, 64)
    assert gt.grouped_plan("forward", 4, 2048, 2048, 8, 256) == ("stream", 16, 16)
    # a streamed grid that would not fit is tiled instead
    assert gt.grouped_plan("forward", 4000, 1 << 20, 64, 500, 256)[0] == "tiled"
    for bad in (("forward", 0, 16, 16, 1, 256), ("wgrad", 8, 12, 16, 1, 256), ("fp8", 8, 16, 24, 1, 256),
                ("forward", 8, 16, 16, 1025, 256)):
        with pytest.raises(gt.GemvTileError):
            gt.grouped_plan(*bad)
