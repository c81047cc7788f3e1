"""How the own rows of a batch with shared rows are cut, and where the join
looks for their parts (csrc/work_split.h, compiled for the host)."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from grouped_query_attention_gemv_gb300 import build as gbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("split") / "work_split_shared.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fwrapv", "-shared", "-fPIC", "-I", gbuild.CSRC,
                    os.path.join(HERE, "work_split_shared.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def batches():
    rng = random.Random(3)
    yield [1], 1
    yield [1], 3
    yield [7], 1
    yield [0, 0, 5, 0], 1
    yield [1] * 2048, 1
    yield [8192], 8
    yield [0, 1, 0, 300, 2], 8
    for _ in range(25):
        n_kv = rng.choice([1, 2, 3, 8, 32])
        yield [rng.choice([0, 1, 2, rng.randint(1, 40), rng.randint(1, 600)]) for _ in range(rng.randint(1, 90))], n_kv


@pytest.mark.parametrize("grid", [1, 2, 37, 87, 151, 152])
def test_the_join_finds_every_part_once(split, grid):
    for chunks, n_kv in batches():
        total = sum(chunks) * n_kv
        if not total:
            continue
        ctas = split.ctas(total, grid)
        assert 1 <= ctas <= grid and (total < 8 or total // ctas >= 8)
        starts = np.zeros(8 * ctas + 1, np.int32)
        split.warps(total, ctas, starts.ctypes.data_as(ctypes.c_void_p))
        assert starts[0] == 0 and (np.diff(starts) >= 0).all()
        places, first = set(), 0
        for b, n in enumerate(chunks):
            for h in range(n_kv):
                if not n:
                    continue
                end = first + n
                holds = np.flatnonzero(np.maximum(starts[:-1], first) < np.minimum(starts[1:], end)).tolist()
                out = (ctypes.c_int * 2)()
                split.span(first, end, total, ctas, out)
                assert holds == list(range(out[0], out[1] + 1)), (chunks, n_kv, b, h)
                # the places of the parts: (sequence, KV head) + warp
                for w in holds:
                    place = b * n_kv + h + w
                    assert place not in places
                    places.add(place)
                first = end
        assert first == total
        assert max(places) < len(chunks) * n_kv + 8 * grid


@pytest.mark.parametrize("total", [8, 1215, 1216, 100003, (1 << 31) - 1])
def test_large_counts(split, total):
    ctas = split.ctas(total, 152)
    out = (ctypes.c_int * 2)()
    split.span(0, total, total, ctas, out)
    assert (out[0], out[1]) == (0, 8 * ctas - 1)
    for u in (0, total // 3, total - 1):
        split.span(u, u + 1, total, ctas, out)
        assert 0 <= out[0] == out[1] < 8 * ctas
