"""How chunk attention shares out the frames of a clip's few queries among workgroups (cache_index.h, compiled for the
CPU): for every query the splits together hold each frame it sees once, also where some of them go over their part for
one query alone, as they do after a result that is not finite, and others do not."""

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MANY = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("shared") / "shared.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "residual_vector_quantization_amd", "csrc"),
                    os.path.join(ROOT, "tests", "rows_shared_host.cpp"), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def check(lib, past, new, window, sinks, splits, mixes):
    first, last = past, past + new - 1
    for position in range(first, last + 1):
        want = [int(j <= position and (position - j < window or j < sinks)) for j in range(max(last, 0) + 1)]
        counts = []
        for alone in (0, 1):
            counts.append([])
            for split in range(splits):
                c = (ctypes.c_int32 * len(want))()
                lib.shared_count(first, last, window, sinks, splits, split, position, alone, c)
                counts[-1].append(list(c))
        # a split's part is the same in both, so that any mix is a partition
        assert counts[0] == counts[1]
        for mix in mixes:
            got = [sum(x) for x in zip(*(counts[mix(split)][split] for split in range(splits)))]
            assert got == want, (past, new, window, sinks, splits, position)


ALL = (lambda s: 0, lambda s: 1, lambda s: s & 1, lambda s: int(s == 0))


@pytest.mark.parametrize("past,new,window,sinks,splits", [
    (1533, 4, MANY, 0, 4), (5000, 4, 2000, 4, 5), (0, 1, MANY, 0, 1), (0, 8, 3, 1, 2), (700, 16, 0, 5, 3), (700, 16, 0, 0, 3),
    (100, 5, 1, 0, 2), (31, 4, 32, 33, 7), (-3, 6, MANY, 0, 2), (-9, 4, MANY, 2, 2), (64, 3, 60, MANY, 4)])
def test_every_frame_once(lib, past, new, window, sinks, splits):
    check(lib, past, new, window, sinks, splits, ALL)


def test_every_frame_once_in_random_turns(lib):
    rng = random.Random(5)
    for _ in range(60):
        past, new = rng.choice([rng.randrange(-4, 40), rng.randrange(900)]), rng.randrange(1, 6)
        check(lib, past, new, rng.choice([0, 1, rng.randrange(100), rng.randrange(900), MANY]),
              rng.choice([0, rng.randrange(8), rng.randrange(200)]), rng.randrange(1, 9), ALL)


def test_only_what_is_seen_is_gone_over(lib):
    assert lib.shared_frames(5000, 5003, 2000, 4) == 2003 + 4
    assert lib.shared_frames(10, 12, MANY, 0) == 13 and lib.shared_frames(10, 12, 0, 0) == 2
    assert lib.shared_frames(-5, -1, 10, 3) == 0 and lib.shared_frames(MANY - 3, MANY - 1, 10, 3) == 15
