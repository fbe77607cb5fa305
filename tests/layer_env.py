"""Device tensors and comparisons that the GPU tests of the operators around the products share."""
import numpy as np


class Env:
    def __init__(self):
        import torch

        import gemv_tile_pipelined_amd as gt

        assert torch.cuda.is_available(), "the gpu tests need a GPU"
        gt.load_library()
        self.torch, self.gt = torch, gt
        self.types = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}

    def call(self, name, fmt):
        return getattr(self.gt, f"{name}_{fmt}")

    def device(self, x, fmt="f32"):
        """x (numpy) on the GPU, rounded to the format."""
        return self.torch.from_numpy(np.ascontiguousarray(x)).to("cuda", self.types[fmt])

    def whole(self, x):
        """Whole numbers or bytes on the GPU as they are."""
        return self.torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    """A tensor's numbers in 64 bits (whole numbers as they are)."""
    return t.cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def near(got, want, tol):
    """got is within tol of want, and NaN where want is; infinities are equal."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want))
    bad = np.argwhere(~ok)
    assert not len(bad), (f"{len(bad)} of {got.size} outside the tolerance; first at {tuple(bad[0])}: "
                          f"{got[tuple(bad[0])]} for {want[tuple(bad[0])]}")
