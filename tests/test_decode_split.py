"""The split of a paged decode call into ranges of key tiles, on the host: the borders that the joining
kernel is given, and what it takes from entries that no call wrote."""
import ctypes
import os

import numpy as np
import pytest

import dsa_sparse_mla_prefill_gb300 as dsa


@pytest.fixture(scope="module")
def lib():
    from dsa_sparse_mla_prefill_gb300 import build as b
    b.build()
    h = ctypes.CDLL(os.path.join(os.path.dirname(dsa.__file__), "libdsa_selftest.so"))
    h.dsa_selftest_range_begin.restype = ctypes.c_uint
    return h


def border(lib, total, ng, request, tiles, so_far, g, B, groups):
    cut = (ctypes.c_int * 4)()
    u, i = ctypes.c_uint, ctypes.c_int
    if lib.dsa_selftest_border(u(total), u(ng), i(request), i(tiles), i(so_far), u(g), i(B), i(groups), cut):
        return tuple(cut)
    return None


@pytest.mark.parametrize("tiles,groups", [([7], 152), ([1], 152), ([1024], 152), ([3, 0, 0, 9, 1, 1, 40], 38),
                                          ([5] * 300, 152), ([0, 0, 2], 76), ([2 ** 24 - 1], 152), ([2 ** 25, 3, 2 ** 30], 152)])
def test_borders_of_a_split(lib, tiles, groups):
    """Each range's last request, against the definition: tile t is of range g where floor(g W / G) <= t < floor((g+1) W / G)."""
    total = sum(tiles)
    ng = min(total, groups)
    begin = [g * total // ng for g in range(ng + 1)]
    assert [lib.dsa_selftest_range_begin(g, ctypes.c_uint(total), ng) for g in range(ng + 1)] == begin
    starts = np.concatenate([[0], np.cumsum(tiles)])
    for g in range(ng):
        b = int(np.searchsorted(starts, begin[g + 1], side="left")) - 1        # the request of tile begin[g+1] - 1
        so_far = begin[g + 1] - int(starts[b])
        got = border(lib, total, ng, b, tiles[b], so_far, g, len(tiles), groups)
        if so_far == tiles[b]:
            assert got is None
            continue
        first = max(x for x in range(ng) if begin[x] <= starts[b])
        last = max(x for x in range(ng) if begin[x] <= starts[b + 1] - 1)
        assert got == (b, first, last - first + 1, int(begin[first] == starts[b]))


def test_entries_that_no_call_wrote(lib):
    """Whatever a border's memory holds, what is taken from it lies within the call: a request of the batch, and
    ranges around this one."""
    rng = np.random.default_rng(3)
    edge = np.array([0, 1, -1, 2, 7, 8, 151, 152, 2 ** 24, 2 ** 31 - 1, -2 ** 31, 0x7f7f7f7f, 0x7fc00000, -8388608], dtype=np.int64)
    taken = 0
    for n in range(40000):
        groups = int(rng.choice([1, 2, 38, 76, 152]))
        total, ng = (int(x) & 0xffffffff for x in (rng.choice(edge), rng.choice(edge)))
        if n % 4:                                                               # a call's own head, and entries near it
            total = int(rng.integers(1, 5000))
            ng = min(total, groups)
        near = rng.integers(-2, 200, 3)
        entry = [int(x) for x in (near if n % 2 else rng.choice(edge, 3))]
        B, g = int(rng.integers(1, 100)), int(rng.integers(0, groups))
        got = border(lib, total, ng, *entry, g, B, groups)
        if got is None:
            continue
        taken += 1
        request, first, parts, _ = got
        assert 0 <= request < B and 0 <= first <= g and parts >= 2 and first + parts - 1 > g and first + parts <= ng <= groups
    assert taken > 100
    assert border(lib, 5000, 152, 0, 0, 0, 3, 9, 152) is None                   # what a range leaves whose waits ran out


@pytest.mark.parametrize("rows", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("d_qk", [512, 576])
@pytest.mark.parametrize("extra", [0, 8, 64, 72, 128, 576, 4096, 2 ** 28, 2 ** 31 - 1024])
def test_bytes_fetched_of_a_run(lib, rows, d_qk, extra):
    """Up to the end of what is read of the run's last row and no further, so that the columns behind it need not be
    memory; and not at all where more than an eighth would be fetched for nothing."""
    pitch, read = 2 * (d_qk + extra), 2 * d_qk
    size = lib.dsa_selftest_fetch(rows, ctypes.c_longlong(pitch), read)
    if 2 * extra * 8 <= read:
        assert size == (rows - 1) * pitch + read and size % 16 == 0
        assert size <= rows * read * 9 / 8
    else:
        assert size == 0
