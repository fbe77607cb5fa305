"""Block-scaled 8-bit products at the ends of the scales' range: products of two scales that are just normal FP32 numbers,
and very large ones (tolerances: blocks_reference.py).  bf16, which has FP32's range."""
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


# sa and sb: powers of two that the scales of A and B are 1 to 2 times.
ENDS = [(-80, -46), (-46, -80), (-126, 0), (100, 1), (3, 98), (118, -80), (-80, 118)]


@pytest.mark.parametrize("low_a,low_b", ENDS)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,N", [(3, 130), (31, 97), (200, 3000), (3300, 3400)])
def test_dense(env, M, N, rows, low_a, low_b):
    torch, gt = env
    K = 272
    g = np.random.default_rng(M)
    A, B = (torch.from_numpy(np.clip(g.standard_normal(s) * 60, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
            for s in ((M, K), (N, K)))
    sa = (g.uniform(1, 2, (M, 3)) * 2.0**low_a).astype(np.float32)
    sb = (g.uniform(1, 2, (-(-N // rows), 3)) * 2.0**low_b).astype(np.float32)
    D = gt.gemm_fp8_bf16(*[t.cuda() for t in (A, torch.from_numpy(sa), B, torch.from_numpy(sb))]).double().cpu().numpy()
    a, b = (e4m3_values(t.view(torch.uint8).numpy()) for t in (A, B))
    want, tol = block_product(a, sa, b, sb, rows, "bf16")
    assert np.abs(want).max() < 2.0**126
    bad = ~(np.abs(D - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, worst {np.abs(D - want)[bad].max()}"
