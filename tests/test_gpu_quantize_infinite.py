"""The quantisers on blocks with an infinity or a NaN, number by number: q is the e4m3 number nearest to x / scale, so over
an infinite scale a finite x is a zero of its sign and an infinite one NaN; over a NaN scale all are NaN."""
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


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["rows", "tiles"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_numbers_of_the_block(env, kind, fmt, bad):
    torch, gt = env
    g = np.random.default_rng(8)
    v = (g.standard_normal((256, 272)) * np.exp2(g.integers(-12, 12, (256, 272)))).astype(np.float32)
    v[3, ::5] = 0.0
    v[3, 131::10] = -0.0
    v[3, 140] = 60000.0
    v[3, 130], v[3, 201] = bad, bad
    x = torch.from_numpy(v).cuda().to(torch.float16 if fmt == "f16" else torch.bfloat16)
    q, s = getattr(gt, f"quantize_fp8_{kind}_{fmt}")(x)
    bits = q.view(torch.uint8).cpu().numpy()
    rows = slice(3, 4) if kind == "rows" else slice(0, 128)
    block, of = bits[rows, 128:256], x.double().cpu().numpy()[rows, 128:256]
    scale = float(s[(3, 1) if kind == "rows" else (0, 1)])
    if np.isnan(bad):
        assert np.isnan(scale) and ((block & 0x7F) == 0x7F).all()
        return
    assert scale == float("inf")
    finite = np.isfinite(of)
    assert (~finite).sum() == 2 and ((block[~finite] & 0x7F) == 0x7F).all()
    np.testing.assert_array_equal(block[finite], np.where(np.signbit(of[finite]), 0x80, 0))
