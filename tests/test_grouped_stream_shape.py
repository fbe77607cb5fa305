"""The launch shape of streamed grouped products, as the launch itself chooses it (host rules, no GPU)."""
import os

import pytest

import gemv_tile_pipelined_amd as gt


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gt.LIBRARY_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return gt.load_library()


@pytest.mark.parametrize("op", ["forward", "fp8"])
def test_two_blocks_once_they_fill_the_cus_twice(op):
    # More groups than rows: as many units as rows.  2 x 256 workgroups of 32 columns.
    for T, N, blocks in ((4, 4096, 2), (4, 4065, 2), (4, 4064, 1), (4, 2048, 1), (3, 5472, 2), (3, 5440, 1), (1, 16384, 2),
                         (1, 16352, 1), (32, 2048, 2), (8, 4096, 2), (300, 130, 2)):
        assert gt.grouped_plan(op, T, N, 2048, T + 700, 256)[0] == "stream"
        assert gt.grouped_stream_blocks(op, T, N, 2048, T + 700, 256) == blocks, (T, N)
    assert gt.grouped_stream_blocks(op, 32, 2048, 2048, 64, 256) == 2
    assert gt.grouped_stream_blocks(op, 4, 4096, 2048, 64, 304) == 1


def test_refusals():
    for bad in (("forward", 16384, 4096, 4096, 32, 256), ("wgrad", 8, 64, 64, 8, 256), ("fp8", 8, 16, 24, 8, 256),
                ("forward", 24, 2048, 2048, 8, 256)):
        with pytest.raises(gt.GemvTileError):
            gt.grouped_stream_blocks(*bad)
