"""Block-scaled 8-bit products against a 64-bit reference (tolerances: blocks_reference.py)."""
import numpy as np
import pytest

from blocks_reference import block_product, e4m3_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import gemv_tile_pipelined_amd as gt

    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    gt.load_library()
    return torch, gt


def _operand(torch, seed, R, K, rows, spread=1.0):
    """(tensors, values, scales): e4m3 numbers of every magnitude and scales over a few powers of two."""
    g = np.random.default_rng(seed)
    v = np.clip(g.standard_normal((R, K)) * 60 * spread, -448, 448).astype(np.float32)
    q = torch.from_numpy(v).to(torch.float8_e4m3fn)
    s = np.exp2(g.uniform(-9, -5, (-(-R // rows), -(-K // 128)))).astype(np.float32)
    return (q.cuda(), torch.from_numpy(s).cuda()), e4m3_values(q.view(torch.uint8).numpy()), s


def _check(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, worst {np.abs(got - want)[bad].max()}"


def _run(env, M, N, K, fmt, sb_rows):
    torch, gt = env
    (A, sA), a, sa = _operand(torch, M * 7 + N, M, K, 1)
    (B, sB), b, sb = _operand(torch, N * 11 + K, N, K, sb_rows)
    D = getattr(gt, f"gemm_fp8_{fmt}")(A, sA, B, sB)
    want, tol = block_product(a, sa, b, sb, sb_rows, fmt)
    _check(D.double().cpu().numpy(), want, tol)


# One row to a few blocks of rows (streamed up to 4), columns around the blocks of 16 and 128, K from a part of a
# scale block to several; the last ones have more tiles of 32 x 32, 32 x 64, 64 x 64 and 128 x 64 than there are CUs.
SHAPES = [(1, 1, 16), (1, 130, 128), (1, 300, 2064), (2, 16, 144), (16, 129, 400), (17, 100, 1040), (33, 257, 112),
          (48, 15, 4112), (64, 300, 272), (65, 129, 144), (65, 1, 16), (130, 7, 256), (200, 300, 400), (513, 260, 1040),
          (300, 1000, 4112), (3, 33, 272), (4, 70, 4112), (5, 63, 2064), (31, 97, 1936), (100, 3001, 400), (97, 2998, 2192),
          (200, 3000, 400), (130, 3063, 1168), (500, 3000, 400), (391, 3001, 912), (1100, 3001, 272)]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weight_tiles(env, M, N, K, fmt):
    _run(env, M, N, K, fmt, 128)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_both_by_rows(env, M, N, K):
    _run(env, M, N, K, "bf16" if N % 2 else "f16", 1)


@pytest.mark.parametrize("M,N,K,sb_rows", [(3500, 3601, 272, 128), (3300, 4000, 528, 1), (4100, 3345, 16, 128)])
def test_large_tiles(env, M, N, K, sb_rows):
    _run(env, M, N, K, "bf16", sb_rows)


@pytest.mark.parametrize("M,N,K", [(540700, 16, 8192), (540700, 4096, 16), (30, 540700, 8192), (3, 540700, 8192)])
def test_past_32_bits(env, M, N, K):
    """Operands and outputs of more than 2^32 bytes: what lies at their ends."""
    torch, gt = env

    def many(seed, rows):
        (q, s), _, _ = _operand(torch, seed, min(rows, 4099), K, 1)
        again = lambda t: t.repeat(-(-rows // len(t)), 1)[:rows].contiguous()  # noqa: E731
        return again(q.view(torch.uint8)).view(q.dtype), again(s)

    (A, sA), (B, sB) = many(1, M), many(2, N)
    sB = sB[::128].contiguous()
    D = gt.gemm_fp8_f16(A, sA, B, sB)
    m, n = max(M - 70, 0), max(N - 70, 0) // 128 * 128
    a, b = (e4m3_values(t.view(torch.uint8).cpu().numpy()) for t in (A[m:], B[n:]))
    want = block_product(a, sA[m:].cpu().numpy(), b, sB[n // 128 :].cpu().numpy(), 128, "f16")
    _check(D[m:, n:].double().cpu().numpy(), *want)


@pytest.mark.parametrize("M,N,K", [(5, 40, 4096), (300, 260, 4096), (3500, 3600, 256)])
def test_integers_are_exact(env, M, N, K):
    """Small integers and scales of powers of two: every partial sum is a number of the format."""
    torch, gt = env
    g = np.random.default_rng(5)
    a, b = (g.integers(-2, 3, s).astype(np.float32) for s in ((M, K), (N, K)))
    sa = np.exp2(g.integers(-1, 2, (M, 1)).repeat(-(-K // 128), 1)).astype(np.float32)
    sb = np.full((-(-N // 128), -(-K // 128)), 0.5, np.float32)
    dev = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    D = gt.gemm_fp8_f16(dev[0].to(torch.float8_e4m3fn), dev[1], dev[2].to(torch.float8_e4m3fn), dev[3])
    want = (dev[0].double() @ dev[2].double().t().contiguous() * dev[1][:, :1].double() * 0.5).half()
    assert torch.equal(D, want)


@pytest.mark.parametrize("M", [3, 200])
def test_k_zero_and_nothing_to_do(env, M):
    torch, gt = env
    e = lambda *s: torch.empty(*s, device="cuda", dtype=torch.float8_e4m3fn)  # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    D = gt.gemm_fp8_bf16(e(M, 0), f(M, 0), e(33, 0), f(1, 0), torch.full((M, 33), 5.0, device="cuda").bfloat16())
    assert (D == 0).all()
    assert gt.gemm_fp8_bf16(e(0, 16), f(0, 1), e(33, 16), f(1, 1)).shape == (0, 33)
    assert gt.gemm_fp8_bf16(e(M, 16), f(M, 1), e(0, 16), f(0, 1)).shape == (M, 0)


@pytest.mark.parametrize("M,N", [(3, 40), (70, 131)])
def test_nan_stays_in_its_row_and_column(env, M, N):
    """A NaN number, a NaN scale and an infinite scale reach their own row or column and nothing else."""
    torch, gt = env
    (A, sA), _, _ = _operand(torch, 1, M, 400, 1)
    (B, sB), _, _ = _operand(torch, 2, N, 400, 128)
    want = gt.gemm_fp8_bf16(A, sA, B, sB)
    A.view(torch.uint8)[1, 399] = 0x7F
    B.view(torch.uint8)[N - 1, 0] = 0xFF
    sA[2, 3] = float("nan")
    got = gt.gemm_fp8_bf16(A, sA, B, sB)
    clean = torch.ones(M, N, dtype=torch.bool, device="cuda")
    clean[1], clean[2], clean[:, N - 1] = False, False, False
    assert torch.isnan(got[~clean]).all() and torch.equal(got[clean], want[clean])


def test_quantise_then_multiply(env):
    """The operators as they are used: quantise a weight once and the activations each time, multiply, and take the
    two gradients, the last with both sides quantised by rows.  Against the exact product of what was quantised."""
    torch, gt = env
    g = torch.Generator().manual_seed(3)
    M, N, K = 160, 272, 400
    x, w, dy = ((torch.randn(*s, generator=g) * c).cuda().bfloat16() for s, c in (((M, K), 1), ((N, K), 0.05), ((M, N), 0.1)))

    def values(q, s, rows):
        s = s.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]
        return (torch.from_numpy(e4m3_values(q.view(torch.uint8).cpu().numpy())).cuda() * s)

    for a, b, b_rows in ((x, w, 128), (dy, w.t().contiguous(), 128), (dy.t().contiguous(), x.t().contiguous(), 1)):
        qa, sa = gt.quantize_fp8_rows_bf16(a)
        qb, sb = (gt.quantize_fp8_tiles_bf16 if b_rows == 128 else gt.quantize_fp8_rows_bf16)(b)
        D = gt.gemm_fp8_bf16(qa, sa, qb, sb).double()
        exact = values(qa, sa, 1) @ values(qb, sb, b_rows).t().contiguous()
        want, tol = block_product(*[np.asarray(v) for v in (
            e4m3_values(qa.view(torch.uint8).cpu().numpy()), sa.cpu().numpy(),
            e4m3_values(qb.view(torch.uint8).cpu().numpy()), sb.cpu().numpy())], b_rows, "bf16")
        np.testing.assert_allclose(exact.cpu().numpy(), want, rtol=1e-9, atol=1e-9)
        _check(D.cpu().numpy(), want, tol)
        # e4m3 keeps a number to 2^-4 of itself, or to half a subnormal step, 2^-10 of the scale: the product of the
        # 16-bit operands is this near.
        full = a.double() @ b.double().t().contiguous()
        ea = a.double().abs() * 2.0**-4 + sa.double().repeat_interleave(128, 1)[:, : a.shape[1]] * 2.0**-10
        eb = b.double().abs() * 2.0**-4 + sb.double().repeat_interleave(b_rows, 0)[: b.shape[0]].repeat_interleave(128, 1)[:, : b.shape[1]] * 2.0**-10
        far = (ea @ (b.double().abs() + eb).t().contiguous()) + (a.double().abs() @ eb.t().contiguous())
        assert ((D - full).abs().cpu().numpy() <= far.cpu().numpy() + tol).all()


def test_streams_and_graph(env):
    """On a stream of its own, and replayed from a graph with eager work between the replays."""
    torch, gt = env
    (A, sA), _, _ = _operand(torch, 1, 100, 528, 1)
    (B, sB), _, _ = _operand(torch, 2, 300, 528, 128)
    x = torch.randn(100, 528, device="cuda").half()
    want = gt.gemm_fp8_f16(A, sA, B, sB)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gt.gemm_fp8_f16(A, sA, B, sB, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    q, s, D = torch.empty_like(A), torch.empty_like(sA), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gt.quantize_fp8_rows_f16(x, q, s)
        gt.gemm_fp8_f16(q, s, B, sB, D)
    for seed in range(3):
        x.copy_(torch.randn(100, 528, generator=torch.Generator().manual_seed(seed)))
        eager = gt.gemm_fp8_f16(*gt.quantize_fp8_rows_f16(x), B, sB)
        D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, eager)
