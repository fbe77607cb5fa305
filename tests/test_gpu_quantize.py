"""The e4m3 quantisers against a 64-bit reference, bit for bit: the scale is the correctly rounded quotient and every
number the nearest one of the real quotient, so there is one right answer."""
import numpy as np
import pytest

from blocks_reference import e4m3_values, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import gemv_tile_pipelined_amd as gt

    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    gt.load_library()
    return torch, gt


def _calls(gt, fmt):
    return {k: getattr(gt, f"quantize_fp8_{k}_{fmt}") for k in ("rows", "tiles")}


def _tensor(torch, x, fmt):
    return torch.from_numpy(np.asarray(x, np.float32)).to("cuda", torch.float16 if fmt == "f16" else torch.bfloat16)


def _check(env, x, fmt, kind):
    torch, gt = env
    t = _tensor(torch, x, fmt)
    q, scale = _calls(gt, fmt)[kind](t)
    bits, want = quantise(t.cpu().double().numpy(), 1 if kind == "rows" else 128)
    assert q.dtype == torch.float8_e4m3fn and q.shape == t.shape
    np.testing.assert_array_equal(scale.cpu().numpy(), want)
    np.testing.assert_array_equal(q.view(torch.uint8).cpu().numpy(), bits)


def _normal(seed, shape, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16), (1, 128), (3, 144), (7, 1040), (130, 272), (33, 4096)])
def test_rows(env, shape, fmt):
    _check(env, _normal(1, shape), fmt, "rows")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (129, 144), (300, 1040), (1, 16, 16), (3, 257, 400), (2, 127, 112)])
def test_tiles(env, shape, fmt):
    _check(env, _normal(2, shape, 0.02), fmt, "tiles")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["rows", "tiles"])
def test_ties_and_small_numbers(env, kind, fmt):
    """Quotients exactly between two numbers (in every binade and among the subnormals), next to such, and tiny ones;
    a scale of 1, 3 and 2^-5 (the last column of a block sets it)."""
    steps = [(8 + m + 0.5) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(7)] + [(m + 0.5) * 2.0**-9 for m in range(8)]
    rows = []
    for s in (1.0, 3.0, 2.0**-5):
        for shift in (1.0, 1.0 + 2.0**-7, 1.0 - 2.0**-8):
            v = np.array(steps + [2.0**-11, 0.0, -0.0]) * s * shift
            v = np.concatenate([np.where(np.arange(len(v)) % 2, -v, v), np.zeros(127 - len(v)), [448.0 * s]])
            rows.append(v)
    _check(env, np.stack(rows), fmt, kind)


@pytest.mark.parametrize("kind", ["rows", "tiles"])
def test_scale_range(env, kind):
    """Zeros and values below the scale's floor, the smallest and largest bf16 magnitudes."""
    x = np.zeros((6 * 128, 256))
    x[128:256, :128] = _normal(3, (128, 128), 1e-24)
    x[256:384] = _normal(4, (128, 256), 1e-38)
    x[384:512, ::3] = 3.0e38
    x[512:640, 5] = 2.0**-133
    x[640:, 200:] = _normal(5, (128, 56), 1e30)
    _check(env, x, "bf16", kind)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_every_f16_pattern(env, fmt):
    """All finite 16-bit patterns, 64 to a block beside a number that sets the block's scale."""
    torch, gt = env
    bits = np.arange(1 << 16, dtype=np.uint16)
    t = torch.from_numpy(bits.view(np.int16)).view(torch.float16 if fmt == "f16" else torch.bfloat16)
    v = t.double().numpy()
    v = v[np.isfinite(v)].reshape(-1, 64)
    _check(env, np.concatenate([v, v * 0.37], 1), fmt, "rows")


@pytest.mark.parametrize("kind", ["rows", "tiles"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_not_finite(env, kind, bad):
    """A block with an infinity or a NaN stands for NaN wherever it is multiplied; other blocks do not change."""
    torch, gt = env
    x = torch.from_numpy(_normal(6, (256, 384)).astype(np.float32)).cuda().half()
    want_q, want_s = _calls(gt, "f16")[kind](x)
    x[3, 130] = bad
    q, s = _calls(gt, "f16")[kind](x)
    at = (3, 1) if kind == "rows" else (0, 1)
    assert (torch.isnan(s) if np.isnan(bad) else torch.isinf(s))[at]
    rows = slice(3, 4) if kind == "rows" else slice(0, 128)
    value = torch.from_numpy(e4m3_values(q.view(torch.uint8).cpu().numpy())) * s[at].double().cpu()
    assert torch.isnan(value[rows, 128:256] * 0).all()
    other = torch.ones(256, 384, dtype=torch.bool)
    other[rows, 128:256] = False
    assert torch.equal(q.view(torch.uint8).cpu()[other], want_q.view(torch.uint8).cpu()[other])
    keep = torch.ones(s.shape, dtype=torch.bool)
    keep[at] = False
    assert torch.equal(s.cpu()[keep], want_s.cpu()[keep])


def test_outputs_given_and_nothing_else_written(env):
    torch, gt = env
    x = torch.randn(37, 272, device="cuda").half()
    q = torch.full((39, 272), 7.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((39, 3), 7.0, device="cuda")
    got = gt.quantize_fp8_rows_f16(x, q[1:38], s[1:38])
    assert got[0].data_ptr() == q[1:].data_ptr() and got[1].data_ptr() == s[1:].data_ptr()
    want = gt.quantize_fp8_rows_f16(x)
    assert torch.equal(q.view(torch.uint8)[1:38], want[0].view(torch.uint8)) and torch.equal(s[1:38], want[1])
    assert (q[[0, 38]].float() == 7).all() and (s[[0, 38]] == 7).all()
