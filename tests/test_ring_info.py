"""gemvtile_ring_trace without a place for its info, and with nothing written behind the ten numbers of it."""
import ctypes

import pytest

import gemv_tile_pipelined_amd as gt


@pytest.mark.parametrize("variant", [20, 10, 21, 23, 32])
def test_info(variant):
    lib = gt.load_library()
    info = (ctypes.c_int * 12)(*[-7] * 12)
    n = lib.gemvtile_ring_trace(variant, 5, None, 0, info)
    assert n > 0 and list(info[10:]) == [-7, -7] and all(v >= 0 for v in info[:10])
    assert lib.gemvtile_ring_trace(variant, 5, None, 0, None) == n


def test_spare_info_is_as_long():
    """The library's own array, used where the caller gives none, holds all that the trace writes."""
    import os
    import re

    csrc = os.path.join(os.path.dirname(gt.__file__), "csrc")
    api, gemm, shared = (open(os.path.join(csrc, f)).read() for f in ("api.hip", "gemm.hip", "kernels.hpp"))
    size = int(re.search(r"constexpr int kRingInfo = (\d+);", shared).group(1))
    assert re.search(r"int dummy\[gt::kRingInfo\];", api)
    assert max(int(i) for i in re.findall(r"info\[(\d+)\] = ", gemm)) == size - 1
