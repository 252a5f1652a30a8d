"""Shapes of the streaming-attention operators that no launch can hold are refused as such, before anything is
enqueued (no GPU)."""

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


@pytest.mark.parametrize("clips,hq,hk,tokens", [(2 ** 20, 64, 64, 2 ** 20), (1, 1024, 1, 2 ** 21), (2 ** 20, 16, 1, 0x7ffffbff),
                                                (2 ** 20, 65535, 65535, 100)])
def test_windowed_attention(a, clips, hq, hk, tokens):
    s = a._AttentionShape(2, clips, hq, hk, 64, 0, -1, tokens, tokens, P, P, 0.125)
    q, k = heads(a, hq), heads(a, hk)
    assert a._lib().rvq_window_attention(ctypes.byref(s), q, k, k, q, None, None) == -2
    assert a._lib().rvq_window_attention_backward(ctypes.byref(s), q, q, k, k, q, P, q, k, k, P, BIG, None) == -2


def test_gradient_of_many_keys(a):
    s = a._AttentionShape(2, 2 ** 20, 64, 64, 64, 0, -1, 0, 2 ** 20, P, P, 0.125)
    k = heads(a, 64)
    assert a._lib().rvq_window_attention_backward(ctypes.byref(s), None, None, k, k, None, None, None, k, k, P, BIG, None) == -2


@pytest.mark.parametrize("clips,hq,hk", [(2 ** 20, 16, 16), (2 ** 20, 272, 1), (2 ** 18, 65535, 65535)])
def test_cache_attention(a, clips, hq, hk):
    s, q = a._CacheShape(2, clips, hk, 64, 1, 8, 1), heads(a, hq)
    assert a._lib().rvq_cache_attention(ctypes.byref(s), hq, q, P, P, P, P, -1, 0, 0.125, q, P, BIG, None) == -2


def test_append(a):
    s, k = a._CacheShape(2, 4, 1, 64, 16, 8, 4), heads(a, 1)
    assert a._lib().rvq_cache_append(ctypes.byref(s), k, k, 2 ** 27, P, P, P, P, P, None) == -2
