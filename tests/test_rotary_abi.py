"""Rotary positions: frequencies on the host, refusals before anything is enqueued (no GPU)."""

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


def test_packed_structure_is_the_structure():
    from residual_vector_quantization_amd import attention as a
    assert bytes(a._Rotation(2 ** 47, 64, 1, 0, 0.5)) == a._pack_rotation(2 ** 47, 64, 1, 0, 0.5)
    assert bytes(a._Rotation(2 ** 47, 64, 1, 1, 0.5)) == a._pack_rotation(2 ** 47, 64, True, True, 0.5)


def test_frequencies(lib):
    import residual_vector_quantization_amd as rvq
    rot, base = 64, 10000.0
    plain = rvq.rvq_rotary_frequencies(rot, base)
    want = torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    # pow and ** are each good to a step or two of float64
    torch.testing.assert_close(plain, want, rtol=4e-16, atol=0)
    torch.testing.assert_close(rvq.rvq_rotary_frequencies(rot, base, "linear", 8.0), want / 8, rtol=1e-15, atol=0)
    by_base = rvq.rvq_rotary_frequencies(rot, base, "base", 8.0)
    # the exponent's rounding grows with the logarithm of the base, about 12
    torch.testing.assert_close(by_base[-1], want[-1] / 8, rtol=1e-14, atol=0)
    assert by_base[0] == 1 and (by_base[1:] < want[1:]).all() and (by_base[1:] > want[1:] / 8 * (1 - 1e-12)).all()
    ramp = rvq.rvq_rotary_frequencies(rot, base, "ramp", 8.0, context=4096, slow=1, fast=32)
    turns = 4096 * want / (2 * math.pi)
    assert torch.equal(ramp[turns > 32.001], plain[turns > 32.001])
    torch.testing.assert_close(ramp[turns < 0.999], want[turns < 0.999] / 8, rtol=1e-15, atol=0)
    between = (turns > 1.001) & (turns < 31.999)
    keep = (turns[between] - 1) / 31
    assert between.any()
    torch.testing.assert_close(ramp[between], want[between] * (keep + (1 - keep) / 8), rtol=1e-14, atol=0)
    assert rvq.rvq_rotary_frequencies(2, scaling="base", factor=4.0).tolist() == [1.0]


@pytest.mark.parametrize("change", [dict(rot=0), dict(rot=7), dict(rot=-2), dict(base=0.0), dict(base=math.inf),
                                    dict(base=math.nan), dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.0),
                                    dict(scaling=2, factor=math.nan), dict(scaling=3, context=0.0),
                                    dict(scaling=3, slow=32.0), dict(scaling=3, fast=math.inf), dict(out=None)])
def test_frequency_arguments(lib, change):
    space = (ctypes.c_double * 64)()
    args = dict(rot=64, base=1e4, scaling=0, factor=2.0, context=100.0, slow=1.0, fast=32.0, out=space)
    args.update(change)
    assert lib.rvq_rotary_frequencies(*args.values()) == -1
    assert not any(space)


def test_binding_refusals():
    import residual_vector_quantization_amd as rvq
    with pytest.raises(ValueError):
        rvq.rvq_rotary_frequencies(63)
    with pytest.raises(ValueError):
        rvq.rvq_rotary_frequencies(64, scaling="other")
    with pytest.raises(rvq.RVQError):
        rvq.rvq_rotary_frequencies(64, scaling="ramp", factor=2.0)
    q, f = torch.zeros(4, 2, 64), rvq.rvq_rotary_frequencies(64)
    with pytest.raises(ValueError):
        rvq.rvq_rotary(None, None, f)
    with pytest.raises(ValueError):
        rvq.rvq_rotary(q, q, f, cu=torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(TypeError):
        rvq.rvq_rotary(q.double(), q.double(), f)


def _rotary(lib, out=(4096, 256, 64), heads=(4096, 256, 64), **change):
    from residual_vector_quantization_amd import attention as a
    rotation = dict(frequencies=4096, rot_dim=64, interleaved=0, inverse=0, amplitude=1.0)
    args = dict(dtype=2, tokens=10, q_heads=4, kv_heads=2, dim=64, clips=1, cu=4096, first=None, positions=None)
    for n, x in change.items():
        (rotation if n in rotation else args)[n] = x
    r = ctypes.byref(a._Rotation(*rotation.values()))
    h, o = ctypes.byref(a._Heads(*heads)), ctypes.byref(a._Heads(*out))
    return lib.rvq_rotary(r, *args.values(), h, h, o, o, None)


@pytest.mark.parametrize("change,status", [
    (dict(frequencies=0), -1), (dict(frequencies=4100), -1), (dict(rot_dim=0), -1), (dict(rot_dim=5), -1),
    (dict(rot_dim=66), -1), (dict(amplitude=math.nan), -1), (dict(amplitude=math.inf), -1), (dict(dtype=3), -1),
    (dict(tokens=-1), -1), (dict(q_heads=-1), -1), (dict(kv_heads=-1), -1), (dict(dim=0), -1), (dict(dim=96), -2),
    (dict(clips=-1), -1), (dict(tokens=2 ** 31), -2), (dict(q_heads=65536), -2), (dict(kv_heads=65536), -2),
    (dict(clips=2 ** 20 + 1), -2), (dict(cu=None), -1), (dict(cu=4098), -1), (dict(first=4098), -1),
    (dict(positions=4098), -1), (dict(heads=(0, 256, 64)), -1), (dict(heads=(4104, 256, 64)), -1),
    (dict(heads=(4096, 257, 64)), -1), (dict(out=(0, 256, 64)), -1), (dict(out=(4096, 64, 64)), -1),
    (dict(tokens=0), 0), (dict(clips=0), 0), (dict(q_heads=0, kv_heads=0), 0)])
def test_rotary_arguments(lib, change, status):
    assert _rotary(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(rotation=None), -1), (dict(inverse=1), -1), (dict(rot_dim=80), -1), (dict(dim=96), -2), (dict(q_heads=-1), -1),
    (dict(tokens=-1), -1), (dict(tokens=3, cu=None), -1), (dict(lens=None), -1), (dict(lens=4098), -1),
    (dict(table=None), -1), (dict(k_pool=None), -1), (dict(v_pool=4104), -1), (dict(q=None), -1), (dict(q_out=None), -1),
    (dict(k=None), -1), (dict(cu=4097), -1), (dict(q_heads=65536), -2), (dict(tokens=0), 0), (dict(n_clips=0), 0)])
def test_append_arguments(lib, change, status):
    from residual_vector_quantization_amd import attention as a
    h, p = ctypes.byref(a._Heads(4096, 256, 64)), 4096
    shape = dict(dtype=2, n_clips=2, kv_heads=2, dim=64, page_size=16, n_pages=8, table_ld=4)
    rotation = dict(frequencies=p, rot_dim=64, interleaved=0, inverse=0, amplitude=1.0)
    args = dict(q_heads=4, q=h, k=h, v=h, tokens=10, cu=p, table=p, lens=p, q_out=h, k_pool=p, v_pool=p)
    given = True
    for n, x in change.items():
        if n == "rotation":
            given = False
        else:
            next(d for d in (shape, rotation, args) if n in d)[n] = x
    r = ctypes.byref(a._Rotation(*rotation.values())) if given else None
    assert lib.rvq_rotary_append(ctypes.byref(a._CacheShape(*shape.values())), r, *args.values(), None) == status
