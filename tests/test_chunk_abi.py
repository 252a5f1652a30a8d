"""Chunks over the paged cache: refusals before anything is enqueued, workspace sizes (no GPU)."""

import ctypes
import math
import os

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import residual_vector_quantization_amd as rvq
    from residual_vector_quantization_amd import attention, build
    if not os.path.exists(rvq.LIBRARY):
        build.build()
    return attention._lib()


def _call(lib, **change):
    from residual_vector_quantization_amd import attention as a
    h, p = ctypes.byref(a._Heads(4096, 256, 64)), 4096
    shape = dict(dtype=2, n_clips=2, kv_heads=2, dim=64, page_size=16, n_pages=8, table_ld=4)
    args = dict(q_heads=4, tokens=10, cu=p, q=h, k_pool=p, v_pool=p, table=p, lens=p, window=-1, sinks=0, scale=0.125,
                out=h, lse=None, work=p, given=1 << 40)
    for n, x in change.items():
        (shape if n in shape else args)[n] = x
    return lib.rvq_cache_chunk_attention(ctypes.byref(a._CacheShape(*shape.values())), *args.values(), None)


def heads(*x):
    from residual_vector_quantization_amd import attention as a
    return ctypes.byref(a._Heads(*x))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), -1), (dict(n_clips=-1), -1), (dict(kv_heads=0), -1), (dict(dim=48), -2), (dict(page_size=0), -1),
    (dict(n_pages=-1), -1), (dict(table_ld=-1), -1), (dict(table_ld=2 ** 20, page_size=2 ** 12), -2),
    (dict(n_clips=2 ** 20 + 1), -2), (dict(q_heads=3), -1), (dict(q_heads=0), -1), (dict(q_heads=65536 * 2), -2),
    (dict(tokens=-1), -1), (dict(tokens=2 ** 31 - 1), -2), (dict(tokens=3, cu=None), -1), (dict(cu=4097), -1),
    (dict(q=None), -1), (dict(k_pool=None), -1), (dict(v_pool=4104), -1), (dict(table=None), -1), (dict(lens=None), -1),
    (dict(lens=4098), -1), (dict(sinks=-1), -1), (dict(scale=math.nan), -1), (dict(scale=-1.0), -1), (dict(out=None), -1),
    (dict(lse=4098), -1), (dict(tokens=0), 0), (dict(n_clips=0), 0)])
def test_arguments(lib, change, status):
    assert _call(lib, **change) == status


def test_rows(lib):
    assert _call(lib, q=heads(4100, 256, 64)) == -1 and _call(lib, q=heads(4096, 255, 64)) == -1
    assert _call(lib, out=heads(4096, 64, 64)) == -1       # heads on top of each other


def test_workspace(lib):
    from residual_vector_quantization_amd import attention as a
    size = lib.rvq_cache_chunk_attention_bytes
    long = ctypes.byref(a._CacheShape(2, 1, 8, 128, 64, 1000, 704))
    wanted = size(long, 32, 4)
    assert wanted > 0
    h = heads(4096, 4096, 128)
    for work, given in ((None, wanted), (4096, wanted - 1), (4104, wanted)):
        assert lib.rvq_cache_chunk_attention(long, 32, 4, 4096, h, 4096, 4096, 4096, 4096, -1, 0, 0.1, h, None, work, given, None) == -1
    assert size(long, 33, 4) == -1 and size(long, 32, -1) == -1 and size(None, 32, 4) == -1
    # it stays small beside the queries and the cache: 2048 workgroups of 32 rows, or 1024 of 128
    for clips in (1, 2, 7, 100, 5000):
        for tokens in (1, 10, 1000, 100000):
            for q_heads in (8, 32, 256):
                shape = ctypes.byref(a._CacheShape(2, clips, 8, 128, 64, 1000, 704))
                n = size(shape, q_heads, tokens)
                assert 0 <= n <= (4096 * 32 + 1024 * 128) * 130 * 4 + 64


def test_binding_refuses():
    import residual_vector_quantization_amd as rvq
    q, pool = torch.zeros(4, 2, 64), torch.zeros(2, 2, 4, 64)
    table, lens = torch.zeros((4, 1), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rvq.rvq_cache_chunk_attention(q, pool, pool, table, lens)
