"""Cross attention: refusals before anything is enqueued, workspace sizes, and the float64 oracle's gradients (no GPU)."""

import ctypes
import math
import os

import pytest
import torch

import cross_oracle as oracle


@pytest.fixture(scope="module")
def lib():
    import residual_vector_quantization_amd as rvq
    from residual_vector_quantization_amd import attention, build
    if not os.path.exists(rvq.LIBRARY):
        build.build()
    return attention._lib()


def _shape(**change):
    from residual_vector_quantization_amd import attention as a
    fields = dict(dtype=2, n_clips=1, q_heads=4, kv_heads=2, dim=64, sinks=0, window=-1, q_tokens=10, k_tokens=12,
                  cu_q=4096, cu_k=4096, scale=0.125)
    fields.update(change)
    return ctypes.byref(a._AttentionShape(**fields))


def _heads(*x):
    from residual_vector_quantization_amd import attention as a
    return ctypes.byref(a._Heads(*x))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), -1), (dict(n_clips=-1), -1), (dict(q_heads=0), -1), (dict(q_heads=3), -1), (dict(kv_heads=0), -1),
    (dict(dim=0), -1), (dict(dim=96), -2), (dict(q_tokens=-1), -1), (dict(k_tokens=-1), -1),
    (dict(q_tokens=2 ** 31), -2), (dict(k_tokens=2 ** 40), -2), (dict(n_clips=2 ** 20 + 1), -2), (dict(scale=-0.5), -1),
    (dict(scale=math.nan), -1), (dict(cu_q=None), -1), (dict(cu_q=4097), -1), (dict(cu_k=None), -1),
    (dict(cu_k=4098), -1), (dict(n_clips=0), 0)])
def test_arguments(lib, change, status):
    h, kv, p, big = _heads(4096, 256, 64), _heads(4096, 128, 64), 4096, 1 << 40
    assert lib.rvq_cross_attention(_shape(**change), h, kv, kv, h, None, p, big, None) == status
    assert lib.rvq_cross_attention_backward(_shape(**change), h, h, kv, kv, h, p, h, kv, kv, p, big, None) == status
    # window and sinks are not read
    assert lib.rvq_cross_attention_bytes(_shape(sinks=-1, window=5)) == lib.rvq_cross_attention_bytes(_shape())


def test_rows_and_workspace(lib):
    h, kv, p = _heads(4096, 256, 64), _heads(4096, 128, 64), 4096
    for bad in (_heads(0, 256, 64), _heads(4100, 256, 64), _heads(4096, 257, 64)):
        assert lib.rvq_cross_attention(_shape(), bad, kv, kv, h, None, p, 1 << 40, None) == -1
        assert lib.rvq_cross_attention(_shape(), h, bad, kv, h, None, p, 1 << 40, None) == -1
        assert lib.rvq_cross_attention(_shape(), h, kv, bad, h, None, p, 1 << 40, None) == -1
        assert lib.rvq_cross_attention(_shape(), h, kv, kv, bad, None, p, 1 << 40, None) == -1
    assert lib.rvq_cross_attention(_shape(), h, kv, kv, _heads(4096, 64, 64), None, p, 1 << 40, None) == -1
    assert lib.rvq_cross_attention(_shape(), h, kv, kv, h, 4098, p, 1 << 40, None) == -1
    assert lib.rvq_cross_attention(_shape(q_tokens=0), None, None, None, None, None, None, 0, None) == 0
    # one query a clip
    assert lib.rvq_cross_attention_bytes(_shape(cu_q=None, n_clips=10)) >= 0
    long = _shape(k_tokens=100000)
    wanted = lib.rvq_cross_attention_bytes(long)
    assert wanted > 0 and lib.rvq_cross_attention_bytes(None) == -1
    for work, given in ((None, wanted), (p, wanted - 1), (4104, wanted)):
        assert lib.rvq_cross_attention(long, h, kv, kv, h, None, work, given, None) == -1
    wanted = lib.rvq_cross_attention_backward_bytes(_shape())
    assert wanted > 0 and lib.rvq_cross_attention_backward_bytes(None) == -1
    for work, given in ((None, wanted), (p, wanted - 1), (4104, wanted)):
        assert lib.rvq_cross_attention_backward(_shape(), h, h, kv, kv, h, p, h, kv, kv, work, given, None) == -1


def test_binding_refuses():
    import residual_vector_quantization_amd as rvq
    q, cu = torch.zeros(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        rvq.rvq_cross_attention(q, q, q, cu, cu)
    with pytest.raises(ValueError):
        rvq.rvq_cross_attention_backward(q, q, q, q, q, q, None, cu)


def test_oracle_gradients_against_autograd():
    g = torch.Generator().manual_seed(1)
    cu_q, cu_k = [0, 9, 9, 30, 33], [0, 20, 22, 37, 37]
    q, k, v, dout = (torch.randn(n, h, 64, generator=g, dtype=torch.float64).requires_grad_()
                     for n, h in ((33, 4), (37, 2), (37, 2), (33, 4)))
    outs = []
    for b in range(4):
        a, e, c, d = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if c == d:
            outs.append(torch.zeros(e - a, 4, 64, dtype=torch.float64))
            continue
        outs.append(torch.stack([torch.softmax(q[a:e, h] @ k[c:d, h // 2].t() / 8, -1) @ v[c:d, h // 2] for h in range(4)], 1))
    out = torch.cat(outs)
    (out * dout.detach()).sum().backward()
    got = oracle.attention(q.detach(), k.detach(), v.detach(), cu_q, cu_k, 1 / 8, dout.detach())
    torch.testing.assert_close(got["out"][0], out.detach(), rtol=0, atol=1e-12)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        torch.testing.assert_close(got[name][0], x.grad, rtol=0, atol=1e-11)
