"""The kernels' own arithmetic of the paged operators' work split
(csrc/work_split.h, compiled for the host): ranges, tickets, items, plans and
the sequence search."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from grouped_query_attention_gemv_gb300 import build as gbuild

HERE = os.path.dirname(os.path.abspath(__file__))
GRID = 152
WARPS = 8


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("split") / "work_split.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fwrapv", "-shared", "-fPIC", "-I", gbuild.CSRC,
                    os.path.join(HERE, "work_split.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def ints(x):
    return np.ascontiguousarray(x, dtype=np.int32)


def ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def ranges(split, total, parts):
    out = np.zeros(parts + 1, np.int32)
    split.ranges(total, parts, ptr(out))
    return out.astype(np.int64)


def holders(split, total, parts, units):
    units = ints(units)
    out = np.empty_like(units)
    split.holders(total, parts, ptr(units), len(units), ptr(out))
    return out


@pytest.mark.parametrize("total", [1, 7, 8, 151, 152, 153, 1216, 1217, 100003, (1 << 31) - 1])
def test_ranges_are_equal_and_know_their_units(split, total):
    for parts in {1, min(total, 2), min(total, 19), min(total, GRID)}:
        s = ranges(split, total, parts)
        assert s[0] == 0 and s[-1] == total
        size = np.diff(s)
        assert size.min() >= total // parts and size.max() <= -(-total // parts)
        for at in (s[:-1], s[1:] - 1, (s[:-1] + s[1:]) // 2):
            assert (holders(split, total, parts, at) == np.arange(parts)).all()


@pytest.mark.parametrize("c0,c1", [(0, 0), (5, 6), (5, 12), (9, 17), (1000, 8191), (0, 1 << 26), (2**31 - 100, 2**31 - 1)])
def test_warps_share_a_range(split, c0, c1):
    s = np.zeros(WARPS + 1, np.int32)
    split.shares(c0, c1, WARPS, ptr(s))
    assert s[0] == c0 and s[-1] == c1
    size = np.diff(s.astype(np.int64))
    assert size.min() >= (c1 - c0) // WARPS and size.max() <= -(-(c1 - c0) // WARPS)


@pytest.mark.parametrize("lens", [[1], [16], [17], [1000] * 16, [131072], [0, 5, 0, 300, 1], list(range(70)), [1] * 2000])
@pytest.mark.parametrize("n_kv", [1, 2, 8, 32])
def test_decode_segments_have_the_parts_their_ticket_counts(split, lens, n_kv):
    """A segment (sequence, KV head) that several CTAs hold has one part in each
    CTA from the holder of its first chunk to that of its last, which is what
    its ticket counts; a CTA begins no more than one such segment and goes on
    with no more than one."""
    chunks = np.repeat([-(-n // 16) for n in lens if n], n_kv)
    end = np.cumsum(chunks)
    first, total = end - chunks, int(end[-1])
    ctas = split.ctas(total, GRID, WARPS)
    assert 1 <= ctas <= GRID and total >= ctas and (ctas == GRID or total <= ctas * WARPS)
    s = ranges(split, total, ctas)
    a, z = holders(split, total, ctas, first), holders(split, total, ctas, end - 1)
    shared = np.flatnonzero(a != z)
    for i in shared:
        inside = [c for c in range(ctas) if s[c] < end[i] and s[c + 1] > first[i]]
        assert inside == list(range(a[i], z[i] + 1))
    assert len(set(a[shared])) == len(shared)          # a ticket, and the slot behind, for one segment
    assert len({c for i in shared for c in range(a[i] + 1, z[i] + 1)}) == sum(z[i] - a[i] for i in shared)


def items(tiles, unit):
    return np.concatenate([[0], np.cumsum([n + unit if n else 0 for n in tiles])]).astype(np.int32)


def pieces(split, units, parts, cum, n_kv):
    out = np.zeros((4 * parts + 2 * (len(cum) - 1) * n_kv + 8, 8), np.int32)
    n = split.pieces(units, parts, ptr(cum), len(cum) - 1, n_kv, ptr(out), len(out))
    assert 0 <= n <= len(out)
    return out[:n].tolist()


def check_pieces(split, tiles, n_kv, parts):
    cum = items(tiles, split.item_units())
    units = int(cum[-1]) * n_kv
    seen, began, went_on = {}, {}, {}
    for c, e, g, j0, j1, first, last, behind in pieces(split, units, parts, cum, n_kv):
        if c < 0:   # the item of the range's last unit: what goes on behind this range
            if first == -1 - c and last > first:
                went_on[-1 - c] = (e, g, last)
            continue
        if j1 <= j0:
            continue
        assert first <= c <= last and (j0 == 0) == (c == first) and (j1 == tiles[e]) == (c == last)
        if first != last and c == first:
            assert c not in began
            began[c] = (e, g, last)
        seen.setdefault((e, g), []).append((j0, j1, c, first, last))
    assert began == went_on
    for (e, g), got in seen.items():
        assert [x[0] for x in got] == [0] + [x[1] for x in got[:-1]] and got[-1][1] == tiles[e]
        assert [x[2] for x in got] == list(range(got[0][3], got[0][4] + 1))
        assert len({x[3:] for x in got}) == 1
    assert len(seen) == n_kv * sum(n > 0 for n in tiles)
    return max(len(x) for x in seen.values())


@pytest.mark.parametrize("tiles", [[64] * 4, [57, 58, 59, 60, 61, 62, 63, 64], [157, 1, 0, 3], [469], [1, 1, 20], [0, 0, 9, 0]])
@pytest.mark.parametrize("n_kv", [1, 2, 8])
def test_prefill_ranges_cover_every_key_tile_once(split, tiles, n_kv):
    units = int(items(tiles, split.item_units())[-1]) * n_kv
    for parts in {1, 2, min(GRID, units // 3), min(GRID, units)}:
        check_pieces(split, tiles, n_kv, parts)


@pytest.mark.parametrize("n_kv", [1, 2, 8, 32])
@pytest.mark.parametrize("few", [True, False])
def test_prefill_plans_bound_the_parts_of_an_item(split, n_kv, few):
    """Ranges of half the longest item: three parts at most, which is what an
    epilogue adds; shorter ones: what the second kernel has room for."""
    rng = random.Random(n_kv)
    for _ in range(60):
        top = rng.choice([4, 20, 300, 8192])
        tiles = [rng.randint(0, top) for _ in range(rng.choice([1, 1, 2, 3, rng.randint(4, 320)]))]
        units = int(items(tiles, split.item_units())[-1]) * n_kv
        if not units:
            continue
        longest = max(tiles) + split.item_units()
        size = split.range_units(units, GRID, longest, few)
        assert size >= -(-units // GRID)
        parts = split.parts_of(units, size, GRID)
        assert 1 <= parts <= GRID and units // parts >= size or parts == 1
        assert check_pieces(split, tiles, n_kv, parts) <= (3 if few else split.max_parts())


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 100, 1023, 1025, 2048])
def test_sequence_search(split, B):
    lens = [(b * 7 // 3) % 4 for b in range(B)]
    cu = ints(np.concatenate([[3], 3 + np.cumsum(lens)]))
    owner = [b for b, n in enumerate(lens) for _ in range(n)]
    for m, b in enumerate(owner):
        assert split.sequence(ptr(cu), B, 3 + m) == b
    assert split.sequence(ptr(cu), B, int(cu[-1])) == B


@pytest.mark.parametrize("total", [(1 << 31) - 1 - n for n in (0, 1, 6, 7, 8, 150, 151, 152, 400)])
def test_counts_up_to_their_limit(split, total):
    # a batch may have 2^31 - 1 chunks (units); rounding up must not pass that
    assert split.ctas(total, GRID, WARPS) == GRID
    assert split.range_units(total, GRID, 5, 1) == -(-total // GRID)
    assert split.parts_of(total, -(-total // GRID), GRID) in (GRID, GRID - 1)


@pytest.mark.parametrize("total", [1, 7, 8, 9, 1215, 1216, 1217])
def test_ctas_leave_each_warp_a_chunk(split, total):
    assert split.ctas(total, GRID, WARPS) == min(GRID, -(-total // WARPS))
