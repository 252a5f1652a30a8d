"""Shapes of rotary positions, chunk and cross attention that no launch can hold are refused as such, before anything is
enqueued, and shapes are not refused for a second launch that they do not need (no GPU)."""

import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def a():
    import residual_vector_quantization_amd as rvq
    from residual_vector_quantization_amd import attention, build
    if not os.path.exists(rvq.LIBRARY):
        build.build()
    attention._lib()
    return attention


P, BIG = 4096, 1 << 60


def heads(a, n):
    return ctypes.byref(a._Heads(P, n * 64, 64))


@pytest.mark.parametrize("clips,hq,hk,tokens", [(2 ** 20, 64, 64, 2 ** 20), (2 ** 20, 1024, 1, 0x7ffffb00), (2 ** 18, 65535, 65535, 100)])
def test_cross_attention(a, clips, hq, hk, tokens):
    s = a._AttentionShape(2, clips, hq, hk, 64, 0, -1, tokens, tokens, P, P, 0.125)
    q, k = heads(a, hq), heads(a, hk)
    assert a._lib().rvq_cross_attention(ctypes.byref(s), q, k, k, q, None, P, BIG, None) == -2
    assert a._lib().rvq_cross_attention_backward(ctypes.byref(s), q, q, k, k, q, P, q, k, k, P, BIG, None) == -2


@pytest.mark.parametrize("clips,hq,hk,tokens", [(2 ** 20, 64, 64, 2 ** 20), (2 ** 20, 1024, 1, 0x7ffffb00), (2 ** 20, 65280, 255, 100)])
def test_chunk_attention(a, clips, hq, hk, tokens):
    s, q = a._CacheShape(2, clips, hk, 64, 1, 8, 1), heads(a, hq)
    assert a._lib().rvq_cache_chunk_attention(ctypes.byref(s), hq, tokens, P, q, P, P, P, P, -1, 0, 0.125, q, None, P, BIG, None) == -2


def test_rotary(a):
    r = ctypes.byref(a._Rotation(P, 64, 0, 0, 1.0))
    s, q, k = a._CacheShape(2, 4, 1, 64, 16, 8, 4), heads(a, 65535), heads(a, 1)
    assert a._lib().rvq_rotary(r, 0, 0x7ffffb00, 1, 0, 128, 1, P, None, None, ctypes.byref(a._Heads(P, 128, 128)), None,
                               ctypes.byref(a._Heads(2 * P, 128, 128)), None, None) == -2
    assert a._lib().rvq_rotary_append(ctypes.byref(s), r, 0, None, k, k, 0x7ffffb00, P, P, P, None, P, P, None) == -2


def test_outputs_that_begin_where_inputs_do(a):
    r = ctypes.byref(a._Rotation(P, 64, 0, 0, 1.0))
    x, wider = ctypes.byref(a._Heads(P, 256, 64)), ctypes.byref(a._Heads(P, 512, 64))
    call = a._lib().rvq_rotary
    assert call(r, 2, 10, 4, 0, 64, 1, P, None, None, x, None, wider, None, None) == -1
    assert call(r, 2, 10, 0, 4, 64, 1, P, None, None, None, wider, None, x, None) == -1
    s = ctypes.byref(a._CacheShape(2, 4, 4, 64, 16, 8, 4))
    assert a._lib().rvq_rotary_append(s, r, 4, x, x, x, 10, P, P, P, wider, P, P, None) == -1
