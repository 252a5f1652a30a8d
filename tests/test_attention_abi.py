"""include/rvq_attention.h: exports, refusals before anything is enqueued, sizes (no GPU), and the float64 oracle
of the operators against torch's own softmax."""

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import attention_oracle as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rvq_attention.h")


@pytest.fixture(scope="module")
def lib():
    import residual_vector_quantization_amd as rvq
    from residual_vector_quantization_amd import attention, build
    if not os.path.exists(rvq.LIBRARY):
        build.build()
    return attention._lib()


def declared():
    return sorted(set(re.findall(r"RVQ_API[^;(]*?\b(rvq_\w+)\s*\(", open(HEADER).read())))


def test_header_binding_and_library_agree(lib):
    import residual_vector_quantization_amd as rvq
    assert declared() == sorted(rvq.EXPORTED_ATTENTION)
    for name in declared():
        assert hasattr(lib, name) and callable(getattr(rvq, name))


def test_packed_structures_are_the_structures():
    from residual_vector_quantization_amd import attention as a
    assert bytes(a._Heads(1, 2, 3)) == a._pack_heads(1, 2, 3)
    assert bytes(a._CacheShape(1, 2, 3, 4, 5, 6, 7)) == a._pack_cache(1, 2, 3, 4, 5, 6, 7)
    fields = (1, 2, 3, 4, 5, 6, -7, 2 ** 40, 9, 2 ** 47, 11, 0.5)
    assert bytes(a._AttentionShape(*fields)) == a._pack_attention(*fields)


def test_header_is_c99(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "rvq_attention.h"\nint main(void) { rvq_heads h = {0, 0, 0}; rvq_cache_shape s = '
                   '{RVQ_BF16, 1, 1, 64, 16, 1, 1}; return h.data != 0 || s.dim != 64; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    "-fsyntax-only", str(src)], check=True)


def _attention(lib, heads=None, out=None, **change):
    from residual_vector_quantization_amd import attention as a
    fields = dict(dtype=2, n_clips=1, q_heads=4, kv_heads=2, dim=64, sinks=0, window=-1, q_tokens=10, k_tokens=10,
                  cu_q=4096, cu_k=4096, scale=0.125)
    fields.update(change)
    s = a._AttentionShape(**fields)
    h = ctypes.byref(a._Heads(*(heads or (4096, 256, 64))))
    o = ctypes.byref(a._Heads(*(out or (4096, 256, 64))))
    return lib.rvq_window_attention(ctypes.byref(s), h, h, h, o, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(n_clips=-1), -1), (dict(q_heads=0), -1), (dict(q_heads=3), -1),
    (dict(kv_heads=0), -1), (dict(dim=0), -1), (dict(dim=96), -2), (dict(dim=32), -2), (dict(sinks=-1), -1),
    (dict(q_tokens=-1), -1), (dict(k_tokens=-1), -1), (dict(q_tokens=2 ** 31), -2), (dict(k_tokens=2 ** 40), -2),
    (dict(scale=-0.5), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(cu_q=None), -1),
    (dict(cu_k=4097), -1), (dict(heads=(0, 256, 64)), -1), (dict(heads=(4100, 256, 64)), -1),
    (dict(heads=(4096, 257, 64)), -1), (dict(heads=(4096, -256, 64)), -1), (dict(heads=(4096, 256, 4)), -1),
    (dict(out=(4096, 64, 64)), -1), (dict(out=(4096, 0, 64)), -1), (dict(out=(4096, 256, 0)), -1),
    (dict(out=(4096, 2 ** 62, 2 ** 62)), -1),
    (dict(n_clips=0), 0), (dict(q_tokens=0), 0)])
def test_attention_arguments(lib, change, status):
    assert _attention(lib, **change) == status


def test_backward_arguments(lib):
    from residual_vector_quantization_amd import attention as a
    s = a._AttentionShape(2, 1, 4, 2, 64, 0, -1, 10, 10, 4096, 4096, 0.125)
    size = lib.rvq_window_attention_backward_bytes(ctypes.byref(s))
    assert size >= 4 * 10 * 4
    h, kv = ctypes.byref(a._Heads(4096, 256, 64)), ctypes.byref(a._Heads(4096, 128, 64))

    def call(lse=4096, dq=h, dk=kv, work=4096, given=size):
        return lib.rvq_window_attention_backward(ctypes.byref(s), h, h, kv, kv, h, lse, dq, dk, kv, work, given, None)

    assert call(lse=None) == -1
    assert call(work=None) == -1
    assert call(given=size - 1) == -1
    assert call(work=4104) == -1
    assert call(dq=None) == -1
    assert call(dk=ctypes.byref(a._Heads(4096, 64, 64))) == -1
    s.dim = 80
    assert lib.rvq_window_attention_backward_bytes(ctypes.byref(s)) == -2
    assert lib.rvq_window_attention_backward_bytes(None) == -1


def _cache(a, **change):
    fields = dict(dtype=2, n_clips=2, kv_heads=2, dim=64, page_size=16, n_pages=8, table_ld=4)
    fields.update(change)
    return ctypes.byref(a._CacheShape(**fields))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), -1), (dict(n_clips=-1), -1), (dict(kv_heads=0), -1), (dict(dim=-64), -1), (dict(dim=48), -2),
    (dict(page_size=0), -1), (dict(n_pages=-1), -1), (dict(table_ld=-1), -1),
    (dict(table_ld=2 ** 20, page_size=2 ** 12), -2)])
def test_cache_shapes(lib, change, status):
    from residual_vector_quantization_amd import attention as a
    h = ctypes.byref(a._Heads(4096, 256, 64))
    p = 4096
    assert lib.rvq_cache_attention_bytes(_cache(a, **change), 4) == status
    assert lib.rvq_cache_attention(_cache(a, **change), 4, h, p, p, p, p, -1, 0, 0.125, h, p, 1 << 40, None) == status
    assert lib.rvq_cache_append(_cache(a, **change), h, h, 2, None, p, p, p, p, None) == status
    assert lib.rvq_cache_copy(_cache(a, **change), 1, p, p, 1, p, p, None) == status
    assert lib.rvq_cache_compact(_cache(a, **change), 1, p, p, p, p, p, p, p, p, 1 << 40, None) == status


def test_cache_arguments(lib):
    from residual_vector_quantization_amd import attention as a
    h = ctypes.byref(a._Heads(4096, 256, 64))
    p, big = 4096, 1 << 40

    def attend(heads=4, q=h, pool=p, table=p, lens=p, sinks=0, scale=0.125, work=p, given=big):
        return lib.rvq_cache_attention(_cache(a), heads, q, pool, pool, table, lens, -1, sinks, scale, h, work, given, None)

    assert attend(heads=3) == -1 and attend(heads=0) == -1 and attend(heads=65536 * 2) == -2
    assert attend(q=None) == -1 and attend(pool=None) == -1 and attend(pool=4104) == -1
    assert attend(table=None) == -1 and attend(lens=4098) == -1 and attend(sinks=-1) == -1
    assert attend(scale=math.inf) == -1
    wanted = lib.rvq_cache_attention_bytes(_cache(a, table_ld=10000), 4)
    assert wanted >= 0
    if wanted:
        assert lib.rvq_cache_attention(_cache(a, table_ld=10000), 4, h, p, p, p, p, -1, 0, 0.125, h, p, wanted - 1, None) == -1
    assert lib.rvq_cache_append(_cache(a), h, h, 3, None, p, p, p, p, None) == -1      # one frame a clip
    assert lib.rvq_cache_append(_cache(a), h, h, -1, p, p, p, p, p, None) == -1
    assert lib.rvq_cache_append(_cache(a), h, h, 0, p, p, p, p, p, None) == 0
    assert lib.rvq_cache_append(_cache(a), h, h, 2, None, p, p, 4100, p, None) == -1
    assert lib.rvq_cache_copy(_cache(a), 0, p, p, 1, p, p, None) == -1
    assert lib.rvq_cache_copy(_cache(a), 1, p, p, 0, p, p, None) == 0
    assert lib.rvq_cache_copy(_cache(a), 1, p, None, 1, p, p, None) == -1
    size = lib.rvq_cache_scratch_bytes(2, 8)
    assert size > 0 and lib.rvq_cache_scratch_bytes(-1, 8) == -1 and lib.rvq_cache_scratch_bytes(2 ** 21, 8) == -2
    assert lib.rvq_cache_reserve(p, p, p, p, 2, 4, 16, 8, p, p, p, p, size - 1, None) == -1
    assert lib.rvq_cache_reserve(p, p, p, p, 2, 4, 0, 8, p, p, p, p, size, None) == -1
    assert lib.rvq_cache_reserve(p, p, p, p, 2, 4, 16, 8, p, p, None, p, size, None) == -1
    assert lib.rvq_cache_fork(_cache(a), 1, p, p, p, p, p, 3, p, p, p, p, p, p, p, size, None) == -1
    assert lib.rvq_cache_fork(_cache(a), 1, p, p, p, None, p, 2, p, p, p, p, p, p, p, size, None) == -1
    assert lib.rvq_cache_free(p, p, p, None, 2, 4, 16, 8, 5, -1, p, p, p, None) == -1
    assert lib.rvq_cache_free(p, None, p, None, 2, 4, 16, 8, 5, 0, p, p, p, None) == -1
    assert lib.rvq_cache_compact(_cache(a), 1, p, p, p, p, p, p, None, p, size, None) == -1


def test_binding_refuses_cpu_tensors():
    import residual_vector_quantization_amd as rvq
    q, cu = torch.zeros(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        rvq.rvq_window_attention(q, q, q, cu)
    pool, table, lens = torch.zeros(2, 2, 4, 64), torch.zeros((4, 1), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rvq.rvq_cache_attention(q, pool, pool, table, lens)
    with pytest.raises(ValueError):
        rvq.rvq_cache_reserve(table, lens, lens, lens, 4)


# ---------------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("window,sinks", [(None, 0), (5, 0), (7, 3), (0, 2), (1, 0)])
def test_oracle_gradients_against_autograd(window, sinks):
    g = torch.Generator().manual_seed(1)
    cu_q, cu_k = [0, 9, 9, 30], [0, 20, 22, 37]
    q, k, v, dout = (torch.randn(n, h, 64, generator=g, dtype=torch.float64).requires_grad_()
                     for n, h in ((30, 4), (37, 2), (37, 2), (30, 4)))
    outs = []
    for b in range(3):
        rows = []
        for h in range(4):
            mask = oracle.sees(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], window, sinks)
            x = (q[cu_q[b]:cu_q[b + 1], h] @ k[cu_k[b]:cu_k[b + 1], h // 2].t()) / 8
            x = x.masked_fill(~mask, -1e300)
            w = torch.softmax(x, -1) * mask.any(1, keepdim=True)
            rows.append(w @ v[cu_k[b]:cu_k[b + 1], h // 2])
        outs.append(torch.stack(rows, 1))
    out = torch.cat(outs)
    (out * dout.detach()).sum().backward()
    got = oracle.attention(q.detach(), k.detach(), v.detach(), cu_q, cu_k, window, sinks, 1 / 8, dout.detach())
    torch.testing.assert_close(got["out"][0], out.detach(), rtol=0, atol=1e-12)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        torch.testing.assert_close(got[name][0], x.grad, rtol=0, atol=1e-11)


def test_oracle_pages_by_hand():
    # page size 4; clip 0 holds 6 frames, clip 1 shares its first page and holds 4
    table, lens, refs = [[2, 0, -1], [2, -1, -1]], [6, 4], [1, 0, 2, 0]
    assert oracle.reserve(table, lens, [8, 9], refs, 4) == ([[2, 0, -1], [2, 1, 3]], [1, 1, 2, 1], 0)
    assert oracle.reserve(table, lens, [17, 9], refs, 4) == ([[2, 0, 1], [2, 3, -1]], [1, 1, 2, 1], 3)
    copies = []
    assert oracle.fork(table, lens, refs, [0], [1], 4, copies) == ([[2, 0, -1], [2, 1, -1]], [6, 6], [1, 1, 2, 0], 0)
    assert copies == [(0, 1)]
    assert oracle.free(table, lens, refs, 4, [0, 1], None, 0) == ([[2, 0, -1], [-1, -1, -1]], [6, 0], [1, 0, 1, 0])
    assert oracle.free(table, lens, refs, 4, None, 3, 0) == ([[-1, 0, -1], [2, -1, -1]], [6, 4], [1, 0, 1, 0])
    copies = []
    assert oracle.compact(table, refs, copies) == ([[1, 0, -1], [1, -1, -1]], [1, 2, 0, 0], 2)
    assert copies == [(2, 1)]
