"""The order of the dual-path linear's units (host side, no GPU).

Units wait for one another inside a launch. The same functions that the kernel and its
launcher use are compiled for the host and played through: CTAs start in the order of
their indices as far as there is room, and a CTA that waits keeps its place.
"""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("dual_units") / "libdual_units.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "lossless_decoding_b200", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "dual_units.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.dual_split_plan.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int] * 2 + \
        [ctypes.POINTER(ctypes.c_int)] * 2
    return L


def _plan(lib, t_units, main, resident, kb, few):
    tiles, k = ctypes.c_int(), ctypes.c_int()
    lib.dual_split_plan(t_units, main, resident, kb, few, ctypes.byref(tiles), ctypes.byref(k))
    return tiles.value, k.value


def _units(lib, t_units, main, split, k):
    """[(what it waits for)] per unit: T units first, whole tiles, pieces."""
    waits = [[] for _ in range(t_units)]
    waits += [list(range(t_units)) for _ in range(main - split)]
    first = len(waits)
    tile, piece = ctypes.c_int(), ctypes.c_int()
    at = {}
    for j in range(split * k):
        lib.dual_split_unit(j, k, ctypes.byref(tile), ctypes.byref(piece))
        assert (tile.value, piece.value) not in at
        at[tile.value, piece.value] = first + j
    assert sorted(at) == [(t, p) for t in range(split) for p in range(k)]
    for t in range(split * (k > 0)):
        for p in range(k):
            waits.append(None)
    for (t, p), u in at.items():
        # the finisher also adds the adapter's product, which reads T
        waits[u] = [] if p else [at[t, q] for q in range(1, k)] + list(range(t_units))
    return waits


def _completes(waits, grid, room):
    """Whether a launch of `grid` CTAs completes with `room` of them on the GPU at a time."""
    done, running, queue = set(), {}, list(range(grid))
    while True:
        while queue and len(running) < room:
            c = queue.pop(0)
            running[c] = c
        moved = False
        for c in list(running):
            while running[c] < len(waits) and all(w in done for w in waits[running[c]]):
                done.add(running[c])
                running[c] += grid
                moved = True
            if running[c] >= len(waits):
                del running[c]
                moved = True
        if not running and not queue:
            return len(done) == len(waits)
        if not moved:
            return False


RESIDENT = 148


@pytest.mark.parametrize("t_units", [0, 1, 2])
@pytest.mark.parametrize("main", [1, 2, 5, 8, 12, 24, 36, 37, 46, 47, 48, 49])
def test_few_tiles_complete_with_any_number_of_ctas_on_the_gpu(lib, t_units, main):
    split, k = _plan(lib, t_units, main, RESIDENT, 32, 1)
    if 3 * (t_units + main) <= RESIDENT:
        assert split == main and k in (3, 4)
    waits = _units(lib, t_units, main, split, k)
    assert len(waits) <= RESIDENT  # one round
    for room in (1, 2, 3, len(waits) // 2 + 1, len(waits)):
        assert _completes(waits, len(waits), room), room


@pytest.mark.parametrize("t_units,main", [(0, 180), (1, 160), (1, 190), (5, 240), (2, 330)])
@pytest.mark.parametrize("resident", [74, 148])
def test_units_wait_for_earlier_ones_only(lib, t_units, main, resident):
    split, k = _plan(lib, t_units, main, resident, 32, 0)
    waits = _units(lib, t_units, main, split, k)
    assert all(w < u for u, ws in enumerate(waits) for w in ws)
    assert _completes(waits, resident, resident)


def test_plans(lib):
    assert _plan(lib, 1, 1187, 148, 64, 0) == (4, 4)    # 1188 units: 8 rounds and 4 tiles
    assert _plan(lib, 0, 148, 148, 64, 0) == (0, 1)
    assert _plan(lib, 0, 200, 148, 64, 0) == (0, 1)     # 52 tiles over 148: two pieces do not pay
    assert _plan(lib, 0, 149, 148, 5, 0) == (0, 1)      # too few K-blocks for three pieces
    assert _plan(lib, 0, 149, 148, 6, 0) == (1, 3)
    assert _plan(lib, 150, 1, 148, 64, 0) == (0, 1)     # the last round would reach into the T tiles
    assert _plan(lib, 1, 8, 148, 32, 0) == (0, 1)
    assert _plan(lib, 1, 8, 148, 32, 1) == (8, 4)
