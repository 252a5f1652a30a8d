"""The cache kernels' page arithmetic (cache_index.h), compiled for the CPU: division by the page size, which frames
are seen, and that table entries outside the pool and positions beyond the table are never followed."""

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NO_PAGE = 0xffffffff


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("index") / "index.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "residual_vector_quantization_amd", "csrc"),
                    os.path.join(ROOT, "tests", "cache_index_host.cpp"), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.index_divide.restype = lib.index_row.restype = ctypes.c_uint32
    return lib


def test_division(lib):
    rng = random.Random(1)
    for d in list(range(1, 70)) + [100, 127, 128, 129, 1000, 4095, 65536, 65537, 2 ** 20 - 1, 2 ** 30 + 1, 2 ** 31 - 1]:
        numbers = [0, 1, d - 1, d, d + 1, 2 ** 31 - 1, 2 ** 31 - 2] + [rng.randrange(2 ** 31) for _ in range(200)]
        numbers += [k * d + e for k in (1, 2, 3, (2 ** 31 - 1) // d) for e in (-1, 0, 1)]
        for n in numbers:
            if 0 <= n < 2 ** 31:
                assert lib.index_divide(n, d) == n // d, (n, d)


def test_seen_frames(lib):
    for length in (-3, 0, 1, 2, 5, 9):
        for window in (0, 1, 2, 4, 9, 100, 2 ** 31 - 1):
            for sinks in (0, 1, 3, 50, 2 ** 31 - 1):
                want = [j for j in range(max(length, 0)) if length - 1 - j < window or j < sinks]
                assert lib.index_seen(length, window, sinks, -1) == len(want)
                assert [lib.index_seen(length, window, sinks, i) for i in range(len(want))] == want
    big = 2 ** 31 - 1
    assert lib.index_seen(big, 10, 3, -1) == 13 and lib.index_seen(big, 10, 3, 12) == big - 1


def test_rows_and_bad_pages(lib):
    entries = [4, -1, 0, 7, 8, -2 ** 31, 2 ** 31 - 1]
    row = (ctypes.c_int32 * len(entries))(*entries)
    for page_size in (1, 3, 16):
        for position in list(range(len(entries) * page_size + 3)) + [2 ** 31 - 1, 2 ** 30]:
            e, heads = position // page_size, 5
            for head in (0, 4):
                got = lib.index_row(row, position, page_size, len(entries), 8, heads, head)
                if e < len(entries) and 0 <= entries[e] < 8:
                    assert got == (entries[e] * heads + head) * page_size + position % page_size
                else:
                    assert got == NO_PAGE
    assert lib.index_row(row, 0, 16, 0, 8, 1, 0) == NO_PAGE      # a table without columns
    assert lib.index_row(row, 0, 16, 7, 0, 1, 0) == NO_PAGE      # a pool without pages
