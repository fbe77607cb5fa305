"""Products grouped by expert against a 64-bit reference (tolerances: blocks_reference.py): forward, both gradients,
16-bit and 8-bit, groups of no rows, one row and many, rows of no group, and every tile and unit size."""
import numpy as np
import pytest

from blocks_reference import block_product, e4m3_values, product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import gemv_tile_pipelined_amd as gt

    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    gt.load_library()
    return torch, gt


def _half(torch, seed, shape, fmt, scale=1.0):
    v = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale
    return torch.from_numpy(v).to(torch.float16 if fmt == "f16" else torch.bfloat16)


def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def _check(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.abs(got - want)[bad].max()}"


def _run(env, op, fmt, sizes, N, K, first=0, pad=0, untouched=True):
    """One product; rows of no group have to keep what the output held."""
    torch, gt = env
    off = _offsets(sizes, first)
    T, E = int(off[-1]) + pad, len(sizes)
    cuda = lambda t: t.cuda()  # noqa: E731
    offsets = torch.from_numpy(off).cuda()
    mark = 0.40625
    if op == "wgrad":
        dY, X = _half(torch, 1, (T, N), fmt, 0.1), _half(torch, 2, (T, K), fmt)
        out = torch.full((E, N, K), mark).to(X.dtype).cuda()
        getattr(gt, f"gemm_grouped_wgrad_{fmt}")(cuda(dY), cuda(X), offsets, out)
        got, dY, X = out.double().cpu().numpy(), dY.double().numpy(), X.double().numpy()
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            _check(got[e], *product(dY[rows].T, X[rows].T, fmt), f"group {e}")
        return
    cols = K if op == "dgrad" else N
    out = torch.full((T, cols), mark).to(torch.float16 if fmt == "f16" else torch.bfloat16).cuda()
    if op == "fp8":
        g = np.random.default_rng(3)
        X = torch.from_numpy(np.clip(g.standard_normal((T, K)) * 60, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
        W = torch.from_numpy(np.clip(g.standard_normal((E, N, K)) * 60, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
        kb = -(-K // 128)
        sX = np.exp2(g.uniform(-9, -6, (T, kb))).astype(np.float32)
        sW = np.exp2(g.uniform(-9, -6, (E, -(-N // 128), kb))).astype(np.float32)
        getattr(gt, f"gemm_grouped_fp8_{fmt}")(cuda(X), torch.from_numpy(sX).cuda(), cuda(W), torch.from_numpy(sW).cuda(),
                                               offsets, out)
        x, w = (e4m3_values(v.view(torch.uint8).numpy()) for v in (X, W))
    else:
        X, W = _half(torch, 4, (T, N if op == "dgrad" else K), fmt), _half(torch, 5, (E, N, K), fmt, 0.1)
        name = "gemm_grouped_dgrad" if op == "dgrad" else "gemm_grouped"
        getattr(gt, f"{name}_{fmt}")(cuda(X), cuda(W), offsets, out)
        x, w = X.double().numpy(), W.double().numpy()
    got = out.double().cpu().numpy()
    assert (got[: off[0]] == mark).all() and (got[off[-1] :] == mark).all(), "rows of no group were written"
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        if op == "fp8":
            want = block_product(x[rows], sX[rows], w[e], sW[e], 128, fmt)
        else:
            want = product(x[rows], w[e].T if op == "dgrad" else w[e], fmt)
        _check(got[rows], *want, f"group {e}")


FEW = [[1], [0, 1, 0], [3, 0, 16, 17, 0, 1], [0] * 70 + [2] + [0] * 60 + [5, 1], [15] * 9, [40, 0, 2], [33, 64, 1],
       [1] * 300]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", FEW, ids=lambda s: f"{len(s)}groups{sum(s)}rows")
@pytest.mark.parametrize("N,K", [(130, 72), (16, 264), (1, 8), (100, 1032)])
def test_forward_few_rows(env, sizes, N, K, fmt):
    _run(env, "forward", fmt, sizes, N, K, pad=3)


@pytest.mark.parametrize("sizes", FEW, ids=lambda s: f"{len(s)}groups{sum(s)}rows")
@pytest.mark.parametrize("N,K", [(130, 144), (16, 272), (1, 16), (260, 2064)])
def test_fp8_few_rows(env, sizes, N, K):
    _run(env, "fp8", "bf16" if K % 32 else "f16", sizes, N, K, first=2, pad=1)


MANY = [[300], [129, 0, 257], [0, 1, 500, 0, 64], [70] * 5, [256, 128], [0, 0, 400, 1, 1, 1]]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("sizes", MANY, ids=lambda s: f"{len(s)}groups{sum(s)}rows")
@pytest.mark.parametrize("N,K", [(136, 72), (264, 520), (8, 8), (40, 1032)])
def test_many_rows(env, op, sizes, N, K, fmt):
    _run(env, op, fmt, sizes, N, K, first=5, pad=7)


@pytest.mark.parametrize("sizes", MANY, ids=lambda s: f"{len(s)}groups{sum(s)}rows")
@pytest.mark.parametrize("N,K", [(131, 144), (264, 528), (1, 16), (40, 1040)])
def test_fp8_many_rows(env, sizes, N, K):
    _run(env, "fp8", "bf16" if N % 2 else "f16", sizes, N, K, pad=2)


@pytest.mark.parametrize("op", ["dgrad", "wgrad"])
@pytest.mark.parametrize("sizes", [[1], [0, 0], [1, 0, 2, 0, 9, 63, 65]], ids=["1row", "0rows", "few"])
def test_gradients_of_few_rows(env, op, sizes):
    _run(env, op, "bf16", sizes, 72, 200, pad=1)


def test_forward_odd_columns_in_tiles(env):
    """Rows of the output that are not 16-byte aligned leave element by element."""
    _run(env, "forward", "f16", [300, 17], 261, 136)


def _tiles(op, sizes, N, K):
    """256 x 256 tiles of a product's output."""
    down = len(sizes) * -(-N // 256) if op == "wgrad" else sum(-(-n // 256) for n in sizes)
    return down * -(-(K if op in ("dgrad", "wgrad") else N) // 256)


# 256 x 256 tiles on 256 workgroups: a last round that is not whole and not cut into quarters, alone and after a whole
# one; whole rounds only; quarters after a whole round, and quarters alone.  Remainders of more and fewer than 128 rows.
ROUNDS = {
    "one": ([900, 1100, 1000], 4000, 136),
    "whole": ([700, 1, 1024, 0, 1800], 4090, 72),
    "whole and quarters": ([2560, 5, 0, 2000, 130], 4000, 72),
    "two": ([2560, 1500, 0, 3000, 130], 3900, 72),
}


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("kind", list(ROUNDS))
def test_rounds_of_tiles(env, op, kind):
    torch, gt = env
    sizes, N, K = ROUNDS[kind]
    if op == "dgrad":
        N, K = K, N - N % 8
    if op == "wgrad":
        sizes = [70, 0, 1, 130]
        N, K = {"one": (2296, 1104), "whole": (2048, 2048), "whole and quarters": (2304, 2048), "two": (3584, 2048)}[kind]
    whole, left = divmod(_tiles(op, sizes, N, K), torch.cuda.get_device_properties(0).multi_processor_count)
    assert {"one": whole == 0 and left > 128, "whole": whole >= 1 and left == 0,
            "whole and quarters": whole >= 1 and 0 < left <= 128, "two": whole >= 1 and left > 128}[kind], (whole, left)
    assert gt.grouped_plan(op, sum(sizes), N, K, len(sizes), 256) == ("tiled", 256, 256)
    _run(env, op, "f16", sizes, N, K)


# Last units of no more than 128 rows, enough of them that they are set apart: after a whole round and 16 tiles more.
APART = [1024, 100, 1300, 0, 1, 1790, 128, 64, 129, 127, 3, 90, 50]


@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_short_units_set_apart(env, op):
    torch, gt = env
    N, K = (4000, 136) if op == "forward" else (136, 4000)
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
    across = -(-4000 // 256)
    light = sum(0 < n % 256 <= 128 for n in APART)
    heavy = sum(-(-n // 256) for n in APART) - light
    assert light * across > 128 and heavy * across == 256 + 16
    assert gt.grouped_plan(op, sum(APART), N, K, len(APART), 256) == ("tiled", 256, 256)
    _run(env, op, "bf16", APART, N, K)


# The smaller tiles, and a plan that expected more rows in each group than there are.
SMALL = [("forward", (256, 128), [700, 1, 1300, 0], 2501, 200), ("forward", (128, 128), [1200, 300], 1501, 264),
         ("dgrad", (256, 128), [800, 0, 1200], 200, 2504), ("dgrad", (128, 128), [200, 90], 264, 304),
         ("wgrad", (256, 128), [60, 100, 3, 1, 0, 70, 66], 1000, 1032), ("wgrad", (128, 128), [200, 90], 264, 304)]


@pytest.mark.parametrize("op,tile,sizes,N,K", SMALL)
def test_smaller_tiles(env, op, tile, sizes, N, K):
    torch, gt = env
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_plan(op, sum(sizes), N, K, len(sizes), cus) == ("tiled", *tile)
    _run(env, op, "bf16", sizes, N, K)


@pytest.mark.parametrize("tile,sizes,N,K", [(256, [900, 1100, 1000], 4000, 272), (256, [900, 5, 1100, 0, 2600], 4091, 144),
                                            (128, [700, 1, 1300, 0], 1497, 400)])
def test_fp8_tiles(env, tile, sizes, N, K):
    torch, gt = env
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_plan("fp8", sum(sizes), N, K, len(sizes), cus) == ("tiled", tile, tile)
    _run(env, "fp8", "bf16", sizes, N, K)


# No more tiles than CUs, of each of the sizes that there are for that; the last has more units than were expected.
DEEP = [((32, 32), [9, 0, 40, 1, 64], 1000, 2064), ((32, 64), [20, 33, 0, 50, 1, 70], 2011, 176),
        ((64, 64), [100, 0, 65, 200, 1], 1900, 1040), ((128, 64), [400, 129, 0, 1, 300], 1698, 144),
        ((64, 64), [1] * 30 + [800], 397, 48)]


@pytest.mark.parametrize("op", ["forward", "fp8"])
@pytest.mark.parametrize("tile,sizes,N,K", DEEP)
def test_few_tiles(env, op, tile, sizes, N, K):
    torch, gt = env
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_plan(op, sum(sizes) + 9, N, K, len(sizes), cus) == ("deep", *tile)
    for fmt in ("f16", "bf16"):
        _run(env, op, fmt, sizes, N, K, first=6, pad=3)


# Enough tiles for the tiled kernels: columns and depths that end inside a tile, rows before and behind the groups.
@pytest.mark.parametrize("op", ["forward", "fp8"])
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [[0, 129, 1, 0, 1500, 257], [1887], [70] * 27], ids=["uneven", "one", "even"])
@pytest.mark.parametrize("N,K", [(1501, 80), (1640, 1040), (1498, 16)])
def test_many_tiles(env, op, fmt, sizes, N, K):
    torch, gt = env
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_plan(op, sum(sizes) + 10, N, K, len(sizes), cus)[0] == "tiled"
    _run(env, op, fmt, sizes, N, K, first=3, pad=7)


@pytest.mark.parametrize("op", ["forward", "fp8"])
def test_most_groups_in_tiles(env, op):
    torch, gt = env
    sizes = [9] * 1000 + [0] * 22 + [130, 1]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert gt.grouped_plan(op, sum(sizes), 24, 48, 1024, cus)[0] == "tiled"
    _run(env, op, "f16", sizes, 24, 48)


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad", "fp8"])
def test_most_groups(env, op):
    sizes = [0] * 1024
    sizes[0], sizes[511], sizes[1023] = 3, 70, 1
    _run(env, op, "f16", sizes, 16, 32, pad=1)


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad", "fp8"])
@pytest.mark.parametrize("rows", [5, 400])
def test_offsets_out_of_order_stay_inside(env, op, rows):
    """Offsets that break the rules give wrong rows, but nothing outside the output changes, and groups whose own
    offsets are sound are right if no other group claims their rows."""
    torch, gt = env
    T, N, K = rows, 32, 48
    bad = torch.tensor([-7, 2, 1, 4, 1 << 30, T + 5, -(1 << 31)], dtype=torch.int32, device="cuda")
    E = 6
    guard = lambda *s: torch.full((3, *s), 0.5, device="cuda").half()  # noqa: E731
    if op == "fp8":
        X, W = torch.ones(T, K, device="cuda").to(torch.float8_e4m3fn), torch.ones(E, N, K, device="cuda").to(torch.float8_e4m3fn)
        out = guard(T, N)
        gt.gemm_grouped_fp8_f16(X, torch.ones(T, 1, device="cuda"), W, torch.ones(E, 1, 1, device="cuda"), bad, out[1])
    elif op == "wgrad":
        out = guard(E, N, K)
        gt.gemm_grouped_wgrad_f16(torch.ones(T, N, device="cuda").half(), torch.ones(T, K, device="cuda").half(), bad, out[1])
    else:
        out = guard(T, N if op == "forward" else K)
        call = gt.gemm_grouped_f16 if op == "forward" else gt.gemm_grouped_dgrad_f16
        call(torch.ones(T, K if op == "forward" else N, device="cuda").half(), torch.ones(E, N, K, device="cuda").half(), bad, out[1])
    torch.cuda.synchronize()
    assert (out[0] == 0.5).all() and (out[2] == 0.5).all()


@pytest.mark.parametrize("op", ["forward", "dgrad", "fp8"])
@pytest.mark.parametrize("bad", [[-7, 2, 1, 4, 1 << 30, 3005, -(1 << 31)], [2000, 0, 2900, 100, 3000, 50, 3000], [3000] * 7,
                                 [0, 3000, 0, 3000, 0, 3000, 0]], ids=["wild", "back", "none", "all"])
def test_offsets_out_of_order_in_tiles(env, op, bad):
    torch, gt = env
    T, E, N, K = 3000, 6, 4096, 48
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    out = torch.full((3, T, K if op == "dgrad" else N), 0.5, device="cuda").half()
    if op == "fp8":
        e4m3 = torch.float8_e4m3fn
        gt.gemm_grouped_fp8_f16(one(T, K).to(e4m3), one(T, 1), one(E, N, K).to(e4m3), one(E, N // 128, 1), offsets, out[1])
    elif op == "dgrad":
        gt.gemm_grouped_dgrad_f16(one(T, N).half(), one(E, N, K).half(), offsets, out[1])
    else:
        assert gt.grouped_plan(op, T, N, K, E, 256)[0] == "tiled"
        gt.gemm_grouped_f16(one(T, K).half(), one(E, N, K).half(), offsets, out[1])
    torch.cuda.synchronize()
    assert (out[0] == 0.5).all() and (out[2] == 0.5).all()
    assert ((out[1] == 0.5) | (out[1] == (N if op == "dgrad" else K))).all()


@pytest.mark.parametrize("op", ["forward", "fp8"])
@pytest.mark.parametrize("sizes", [[9, 40, 1, 64], [1] * 4, [700, 1300, 500, 3]], ids=["deep", "streamed", "tiled"])
def test_two_calls_at_once(env, op, sizes):
    """Two streams run the same product on different inputs, unordered."""
    torch, gt = env
    off, T, E, N, K = torch.from_numpy(_offsets(sizes)).cuda(), sum(sizes), len(sizes), 2048, 528
    X, W = (_half(torch, i, s, "f16", 0.3).cuda() for i, s in enumerate(((2, T, K), (2, E, N, K))))
    if op == "fp8":
        ops = [(*gt.quantize_fp8_rows_f16(X[i]), *gt.quantize_fp8_tiles_f16(W[i])) for i in range(2)]
        call = gt.gemm_grouped_fp8_f16
    else:
        ops, call = [(X[i], W[i]) for i in range(2)], gt.gemm_grouped_f16
    alone = [call(*o, off) for o in ops]
    outs = [[torch.empty_like(alone[i]) for _ in range(4)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(4):
        for i in range(2):
            call(*ops[i], off, outs[i][k], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[i]) for i in range(2) for o in outs[i])


# Operands and outputs of more than 2^32 bytes: what lies at their ends.
FAR = [("forward", 540700, 3, 16, 4096), ("forward", 540700, 3, 4096, 16), ("dgrad", 540700, 3, 16, 4096),
       ("dgrad", 540700, 3, 4096, 16), ("wgrad", 540700, 3, 4096, 16), ("wgrad", 540700, 3, 16, 4096),
       ("fp8", 540700, 3, 16, 8192), ("fp8", 540700, 3, 4096, 16),
       ("forward", 300, 70, 8192, 4096), ("forward", 900, 70, 8192, 4096), ("dgrad", 90, 70, 8192, 4096),
       ("wgrad", 90, 70, 8192, 4096), ("fp8", 300, 70, 8192, 8192), ("fp8", 900, 70, 8192, 8192)]


@pytest.mark.parametrize("op,T,E,N,K", FAR)
def test_past_32_bits(env, op, T, E, N, K):
    torch, gt = env
    sizes = [0] * E
    sizes[-1] = min(T, 700)
    sizes[0] = T - sizes[-1]
    off = _offsets(sizes)
    offsets = torch.from_numpy(off).cuda()

    def many(seed, rows, cols, scale=1.0):  # a few thousand rows, over and over
        base = _half(torch, seed, (min(rows, 4099), cols), "f16", scale).cuda()
        return base.repeat(-(-rows // len(base)), 1)[:rows].contiguous()

    left = many(1, T, N if op in ("dgrad", "wgrad") else K)
    if op == "wgrad":
        right = many(2, T, K, 0.05)
        dW = gt.gemm_grouped_wgrad_f16(left, right, offsets)
        assert E < 4 or not dW[1:-1].any()
        rows = slice(off[-2], off[-1])
        dY, X = (t[rows].double().cpu().numpy() for t in (left, right))
        _check(dW[-1].double().cpu().numpy(), *product(dY.T, X.T, "f16"), "last group")
        return
    weights = many(3, E * N, K, 0.05).view(E, N, K)
    if op == "fp8":
        left, weights = left.to(torch.float8_e4m3fn), weights.to(torch.float8_e4m3fn)
        kb = -(-K // 128)
        sX = many(4, T, kb).float().abs() + 0.25
        sW = many(5, E * -(-N // 128), kb).float().abs().view(E, -1, kb) + 0.25
        D = gt.gemm_grouped_fp8_f16(left, sX, weights, sW, offsets)
    else:
        D = (gt.gemm_grouped_dgrad_f16 if op == "dgrad" else gt.gemm_grouped_f16)(left, weights, offsets)
    for e, rows in ((0, slice(max(off[1] - 70, 0), off[1])), (E - 1, slice(max(T - 70, off[-2]), T))):
        if rows.start == rows.stop:
            continue
        got = D[rows].double().cpu().numpy()
        if op == "fp8":
            x, w = (e4m3_values(t.view(torch.uint8).cpu().numpy()) for t in (left[rows], weights[e]))
            want = block_product(x, sX[rows].cpu().numpy(), w, sW[e].cpu().numpy(), 128, "f16")
        else:
            a, b = left[rows].double().cpu().numpy(), weights[e].double().cpu().numpy()
            want = product(a, b.T if op == "dgrad" else b, "f16")
        _check(got, *want, f"group {e}")


@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_sum_over_nothing(env, op):
    torch, gt = env
    offsets = torch.tensor([0, 2, 100], dtype=torch.int32, device="cuda")
    z = lambda *s: torch.empty(*s, device="cuda").half()  # noqa: E731
    out = torch.full((103, 24), 5.0, device="cuda").half()
    if op == "forward":
        gt.gemm_grouped_f16(z(103, 0), z(2, 24, 0), offsets, out)
    else:
        gt.gemm_grouped_dgrad_f16(z(103, 0), z(2, 0, 24), offsets, out)
    assert (out[:100] == 0).all() and (out[100:] == 5).all()
    assert (gt.gemm_grouped_wgrad_f16(z(0, 16), z(0, 24), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                      torch.ones(2, 16, 24, device="cuda").half()) == 0).all()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_gradients_against_differences(env, fmt):
    """A step of one element of X or W changes the sum of D * dY by the gradient's element times the step."""
    torch, gt = env
    sizes, N, K = [70, 0, 3], 48, 40
    T, E = sum(sizes), len(sizes)
    offsets = torch.from_numpy(_offsets(sizes)).cuda()
    X, W, dY = _half(torch, 1, (T, K), fmt).cuda(), _half(torch, 2, (E, N, K), fmt).cuda(), _half(torch, 3, (T, N), fmt).cuda()
    dX = getattr(gt, f"gemm_grouped_dgrad_{fmt}")(dY, W, offsets).double()
    dW = getattr(gt, f"gemm_grouped_wgrad_{fmt}")(dY, X, offsets).double()
    half_step = 2.0**-11 if fmt == "f16" else 2.0**-8

    def loss(x, w):
        total = 0.0
        for e in range(E):
            rows = slice(sum(sizes[:e]), sum(sizes[: e + 1]))
            total += float(((x[rows] @ w[e].t().contiguous()) * dY[rows].double()).sum())
        return total

    x, w = X.double(), W.double()
    for at in [(0, 0), (69, 39), (72, 5), (33, 17)]:
        up = x.clone()
        up[at] += 1.0  # the loss is linear in each operand: any step is exact
        diff = loss(up, w) - loss(x, w)
        # the sum's error (N terms) and the rounding of the result; 1e-9 for the difference's own
        assert abs(float(dX[at]) - diff) <= half_step * abs(diff) + N * 2.0**-23 * 100 + 1e-9
    for at in [(0, 0, 0), (0, 47, 39), (1, 3, 3), (2, 20, 11)]:
        up = w.clone()
        up[at] += 1.0
        diff = loss(x, up) - loss(x, w)
        assert abs(float(dW[at]) - diff) <= half_step * abs(diff) + 70 * 2.0**-23 * 200 + 1e-9


def test_a_layer_of_experts(env):
    """As a mixture layer uses them: a router's choice sorts the tokens, two grouped products with an activation
    between, and the gradients of a loss; against the same layer run token by token in 64 bits, with the 16-bit
    roundings of the values between the products made alike."""
    torch, gt = env
    g = torch.Generator().manual_seed(11)
    tokens, top, E, C, H = 150, 2, 6, 72, 136
    x = torch.randn(tokens, C, generator=g).bfloat16().cuda()
    w1 = (torch.randn(E, H, C, generator=g) * C**-0.5).bfloat16().cuda()
    w2 = (torch.randn(E, C, H, generator=g) * H**-0.5).bfloat16().cuda()
    choice = torch.randn(tokens, E, generator=g).cuda()
    choice[:, 4] = -100.0  # an expert that nobody chooses
    expert = choice.topk(top).indices.reshape(-1)
    order = expert.argsort(stable=True)
    token = order // top
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(expert, minlength=E).cumsum(0)
    rows = x[token].contiguous()
    h = gt.gemm_grouped_bf16(rows, w1, offsets)
    a = torch.relu(h)
    y = gt.gemm_grouped_bf16(a, w2, offsets)
    dy = torch.randn(tokens * top, C, generator=g).bfloat16().cuda()
    da = gt.gemm_grouped_dgrad_bf16(dy, w2, offsets)
    dw2 = gt.gemm_grouped_wgrad_bf16(dy, a, offsets)
    dh = torch.where(h > 0, da, torch.zeros_like(da))
    dx = gt.gemm_grouped_dgrad_bf16(dh, w1, offsets)
    dw1 = gt.gemm_grouped_wgrad_bf16(dh, rows, offsets)
    cut = offsets.tolist()
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    for e in range(E):
        r = slice(cut[e], cut[e + 1])
        for got, want in ((h[r], product(n(rows[r]), n(w1[e]), "bf16")), (y[r], product(n(a[r]), n(w2[e]), "bf16")),
                          (da[r], product(n(dy[r]), n(w2[e]).T, "bf16")), (dx[r], product(n(dh[r]), n(w1[e]).T, "bf16")),
                          (dw2[e], product(n(dy[r]).T, n(a[r]).T, "bf16")), (dw1[e], product(n(dh[r]).T, n(rows[r]).T, "bf16"))):
            _check(n(got), *want, f"expert {e}")
    assert cut[4] == cut[5] and not dw1[4].any() and not dw2[4].any()


@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad", "fp8"])
@pytest.mark.parametrize("rows", [12, 400])
def test_streams_and_graph(env, op, rows):
    """Replayed from a graph with other offsets and inputs each time, eager work between; and on another stream."""
    torch, gt = env
    T, N, K, E = rows, 136, 144, 5
    g = torch.Generator().manual_seed(2)
    t = lambda *s: torch.randn(*s, generator=g).half().cuda()  # noqa: E731
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    if op == "fp8":
        (W, sW), X = gt.quantize_fp8_tiles_f16(t(E, N, K)), t(T, K)
        q, s = gt.quantize_fp8_rows_f16(X)
        D = torch.zeros(T, N, device="cuda").half()

        def call(out=None, stream=None):
            gt.quantize_fp8_rows_f16(X, q, s, stream=stream)
            return gt.gemm_grouped_fp8_f16(q, s, W, sW, offsets, out, stream=stream)
    elif op == "wgrad":
        X, dY = t(T, K), t(T, N)
        D = torch.zeros(E, N, K, device="cuda").half()

        def call(out=None, stream=None):
            return gt.gemm_grouped_wgrad_f16(dY, X, offsets, out, stream=stream)
    else:
        X, W = t(T, K if op == "forward" else N), t(E, N, K)
        D = torch.zeros(T, N if op == "forward" else K, device="cuda").half()
        f = gt.gemm_grouped_f16 if op == "forward" else gt.gemm_grouped_dgrad_f16

        def call(out=None, stream=None):
            return f(X, W, offsets, out, stream=stream)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(D)
    side = torch.cuda.Stream()
    for seed in range(3):
        r = np.random.default_rng(seed)
        offsets.copy_(torch.from_numpy(_offsets(r.multinomial(T, np.ones(E) / E))))
        X.copy_(torch.from_numpy(r.standard_normal(X.shape).astype(np.float32)))
        eager = call(torch.zeros_like(D))
        side.wait_stream(torch.cuda.current_stream())
        other = call(torch.zeros_like(D), side)
        torch.cuda.current_stream().wait_stream(side)
        D.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, eager) and torch.equal(other, eager)
