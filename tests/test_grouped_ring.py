"""The K loop of the tiled grouped products, checked on the CPU: the library runs the kernels' loop on the host and records
its events (gemvtile_grouped_ring_trace), which a model of what they mean on the hardware replays.  Loads of a wave land
in the order of their issue, a wait with count n leaves only the n youngest in flight, and what has landed may be read
by other waves behind the next barrier; a stage may be filled again once every wave has read its K tile."""
import os

import pytest

import gemv_tile_pipelined_amd as gt

TILES = [(256, 256), (256, 128), (128, 128)]
LAST = (1 << 25) - 8  # K tiles of the longest sum, 2^31 - 512 rows


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gt.LIBRARY_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return gt.load_library()


def replay(events, info, first, ktu):
    per, stages = info["loads_per_tile"], info["stages"]
    pending = [(t, d) for t in range(first, first + info["ahead"]) for d in range(per)]
    issued = {load: 1 for load in pending}
    landed, visible = set(), set()
    reading, read, free = set(), set(), set()  # K tiles with reads in flight, read by this wave, read by every wave
    seen, inits = set(), 0
    for name, a, b, c, d in events:
        if name == "load":
            assert c == a % stages
            assert a - stages < first or a - stages in free, f"stage of K tile {a - stages} refilled while it may be read"
            assert (a, b) not in issued, f"load {b} of K tile {a} twice"
            issued[a, b] = 1
            pending.append((a, b))
        elif name == "wait":
            done = len(pending) - a
            if done > 0:
                landed.update(pending[:done])
                del pending[:done]
        elif name == "lds_wait":
            read |= reading
            reading = set()
        elif name == "barrier":
            visible |= landed
            free |= read
        elif name == "read":
            assert d == a % stages
            assert {(a, i) for i in range(per)} <= visible, f"K tile {a} read before all of it is known to have landed"
            assert a not in free, f"K tile {a} read after its stage was given up"
            reading.add(a)
            seen.add(a)
        elif name == "init":
            inits += 1
    assert inits == 1
    assert set(range(first, ktu)) <= seen
    assert all((t, i) in issued for t in range(first, ktu) for i in range(per))


@pytest.mark.parametrize("rows,cols", TILES)
@pytest.mark.parametrize("ktu", [1, 2, 3, 4, 5, 8, 33])
def test_from_the_start(rows, cols, ktu):
    replay(*gt.grouped_ring_trace(rows, cols, 0, ktu), 0, ktu)


@pytest.mark.parametrize("rows,cols", TILES)
@pytest.mark.parametrize("middle", [1 << 16, 1 << 20, 1 << 24, LAST - 16])
def test_far_along_a_long_sum(rows, cols, middle):
    """The waits do not weaken at any length of the sum: a group of a weight gradient has up to 2^31 - 512 rows."""
    first, ktu = middle - 16, middle + 16
    replay(*gt.grouped_ring_trace(rows, cols, first, ktu), first, ktu)


@pytest.mark.parametrize("rows,cols", TILES)
def test_every_wait_is_the_same(rows, cols):
    near = [e[1] for e in gt.grouped_ring_trace(rows, cols, 0, 64)[0] if e[0] == "wait"]
    assert len(set(near[1:])) == 1
    for first in ((1 << 24) - 32, LAST - 64):
        assert [e[1] for e in gt.grouped_ring_trace(rows, cols, first, first + 64)[0] if e[0] == "wait"] == near


def test_model_rejects_a_weaker_wait():
    for rows, cols in TILES:
        events, info = gt.grouped_ring_trace(rows, cols, 0, 8)
        at = [i for i, e in enumerate(events) if e[0] == "wait"][4]
        weak = (*events[at][:1], events[at][1] + info["loads_per_tile"], *events[at][2:])
        with pytest.raises(AssertionError):
            replay(events[:at] + [weak] + events[at + 1 :], info, 0, 8)


def test_refusals():
    for bad in ((256, 64, 0, 4), (256, 256, -1, 4), (256, 256, 4, 4), (256, 256, 0, LAST + 1), (128, 128, 0, 4097)):
        with pytest.raises(gt.GemvTileError):
            gt.grouped_ring_trace(*bad)
