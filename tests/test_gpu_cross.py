"""Cross attention and its gradient on the GPU against float64 (cross_oracle)."""

import math

import pytest
import torch

import cross_oracle as oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, make, offsets

pytestmark = [pytest.mark.gpu, needs_gpu]


def check(typ, dim, hq, hk, q_lens, k_lens, scale=None, train=True, seed=0, fused=False):
    m = rvq()
    announce("cross", typ=typ, dim=dim, heads=(hq, hk), q=q_lens, k=k_lens)
    q, k, v, dout = make(TYPES[typ], dim, hq, hk, q_lens, k_lens, seed)
    if fused:
        kv = torch.cat([k, v], 1)
        k, v = kv[:, :hk], kv[:, hk:]
    cu_q, cu_k = offsets(q_lens), offsets(k_lens)
    out, lse = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k), scale=scale)
    torch.cuda.synchronize()
    want = oracle.attention(q, k, v, cu_q, cu_k, 1 / math.sqrt(dim) if scale is None else scale, dout if train else None)
    close("out", out, want["out"])
    close("lse", lse, want["lse"])
    if train:
        grads = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, ints(cu_q), ints(cu_k), scale=scale)
        torch.cuda.synchronize()
        for name, got in zip(("dq", "dk", "dv"), grads):
            close(name, got, want[name])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("typ", list(TYPES))
def test_short_and_empty_clips(typ, dim):
    check(typ, dim, 2, 1, [1], [1])
    check(typ, dim, 3, 3, [1, 0, 2, 17, 0, 25, 4], [5, 3, 0, 33, 0, 1, 90])
    check(typ, dim, 2, 2, [3, 40], [0, 0])


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("length", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_lengths_around_tiles(typ, dim, length):
    check(typ, dim, 2, 1, [length, 5], [70, length])
    check(typ, dim, 2, 1, [40, length], [length, 131])


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (5, 5), (8, 2), (7, 1), (12, 4), (40, 1), (33, 1)])
@pytest.mark.parametrize("typ", ["bf16", "fp32"])
def test_head_groups(typ, hq, hk):
    check(typ, 64, hq, hk, [150, 33, 1], [90, 40, 7])
    check(typ, 64, hq, hk, [1, 2], [90, 40])


@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("fp16", 64), ("fp32", 128)])
def test_many_keys_and_many_queries(typ, dim):
    check(typ, dim, 2, 1, [4, 1, 9], [5000, 12, 2049], train=False)
    check(typ, dim, 2, 1, [100, 3], [4000, 1500])
    check(typ, dim, 4, 1, [1500], [200], fused=True)


@pytest.mark.parametrize("typ", list(TYPES))
def test_many_queries_of_few_keys(typ):
    """The queries of a key are shared out among workgroups, within a head too."""
    check(typ, 64, 1, 1, [3000], [20])
    check(typ, 64, 3, 1, [1100, 1, 0, 700], [5, 1, 9, 0])
    check(typ, 128, 2, 2, [900, 1300], [130, 3])


@pytest.mark.parametrize("typ", list(TYPES))
def test_one_query_each(typ):
    """With and without offsets; the gradient through offsets."""
    m, lens = rvq(), [300, 1, 0, 65, 64, 2500]
    check(typ, 64, 4, 2, [1] * len(lens), lens)
    q, k, v, _ = make(TYPES[typ], 64, 4, 2, [1] * len(lens), lens)
    cu = ints(offsets(lens))
    out, lse = m.rvq_cross_attention(q, k, v, None, cu)
    want = oracle.attention(q, k, v, list(range(len(lens) + 1)), offsets(lens), 0.125)
    close("out", out, want["out"])
    close("lse", lse, want["lse"])


def test_many_clips():
    k_lens = [(37 * b) % 90 for b in range(200)]
    check("bf16", 64, 2, 1, [1 if b % 3 else 0 for b in range(200)], k_lens)
    check("bf16", 64, 2, 1, [1 if b % 50 else 140 for b in range(200)], k_lens)
    check("fp32", 64, 2, 2, [1] * 130, k_lens[:130])


def test_other_scales():
    check("bf16", 64, 4, 2, [30], [300], scale=1.0)
    check("fp32", 64, 4, 2, [5], [300], scale=0.0)


def test_no_keys_at_all_and_no_queries():
    m = rvq()
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, [30, 1], [0, 0])
    cu_q, cu_k = ints([0, 30, 31]), ints([0, 0, 0])
    out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k)
    assert (dq == 0).all() and dk.shape == (0, 2, 64) and dv.shape == (0, 2, 64)
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, [0, 0], [30, 1])
    out, lse = m.rvq_cross_attention(q, k, v, cu_k, cu_q)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    dq, dk, dv = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_k, cu_q)
    assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("typ", list(TYPES))
def test_rows_outside_clips(typ):
    m = rvq()
    q, k, v, dout = make(TYPES[typ], 64, 4, 2, [200], [300])
    cu_q, cu_k = [7, 150, 153], [20, 120, 290]
    to = [torch.full_like(x, 5.0) for x in (q, q, k, v)]
    k[:20], k[290:], v[:20], v[290:], dout[153:], q[153:] = (math.nan,) * 6
    out, lse = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k), out=to[0])
    grads = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, ints(cu_q), ints(cu_k), grads=to[1:])
    want = oracle.attention(q[7:153], k[20:290], v[20:290], [0, 143, 146], [0, 100, 270], 0.125, dout[7:153])
    close("out", out[7:153], want["out"])
    for name, got, a, e in zip(("dq", "dk", "dv"), grads, (7, 20, 20), (153, 290, 290)):
        close(name, got[a:e], want[name])
        assert (got[:a] == 5).all() and (got[e:] == 5).all()
    assert (out[:7] == 5).all() and (out[153:] == 5).all()


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("nq", [3, 90])
def test_values_that_are_not_finite_stay_in_their_clip(typ, dim, nq):
    m = rvq()
    q, k, v, dout = make(TYPES[typ], dim, 2, 1, [nq, nq], [70, 70])
    cu_q, cu_k = ints([0, nq, 2 * nq]), ints([0, 70, 140])
    out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
    grads = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k)
    for value in (math.inf, -math.inf, math.nan):
        v2 = v.clone()
        v2[69, 0, 3] = value
        got, _ = m.rvq_cross_attention(q, k, v2, cu_q, cu_k)
        assert torch.equal(got[nq:], out[nq:]) and not torch.isfinite(got[:nq, :, 3]).any()
        keep = [d for d in range(dim) if d != 3]
        assert torch.isfinite(got[:nq][..., keep]).all()
        again = m.rvq_cross_attention_backward(dout, q, k, v2, got, lse, cu_q, cu_k)
        for x, y, n in zip(again, grads, (nq, 70, 70)):
            assert torch.equal(x[n:], y[n:]) if typ != "fp16" else torch.isfinite(x[n:]).all()


def test_gradient_against_differences():
    """The directional derivative of sum(out dout) by float64 differences of the definition, against the GPU's gradients;
    they may be off by their bounds. The differences are good to step^2 of the third derivative: the softmax of scores of
    order 1 keeps it below some hundred times the first, 1e-6 with a step of 1e-4."""
    m = rvq()
    q, k, v, dout = make(torch.float32, 64, 4, 2, [40, 3], [30, 70])
    cu_q, cu_k = [0, 40, 43], [0, 30, 100]
    out, lse = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k))
    grads = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, ints(cu_q), ints(cu_k))
    want = oracle.attention(q, k, v, cu_q, cu_k, 0.125, dout)
    g, x = torch.Generator().manual_seed(5), [t.double().cpu() for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        way = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        ends = []
        for step in (1e-4, -1e-4):
            moved = [t + step * way if n == i else t for n, t in enumerate(x)]
            ends.append((oracle.attention(*moved, cu_q, cu_k, 0.125)["out"][0] * dout.double().cpu()).sum().item())
        slope, got = (ends[0] - ends[1]) / 2e-4, (grads[i].double().cpu() * way).sum().item()
        size = (want[name][0].abs() * way.abs()).sum().item()
        assert abs(got - slope) <= (want[name][1] * way.abs()).sum().item() + 1e-6 * size


def test_training_step_captured_beside_an_eager_one():
    m = rvq()
    q, k, v, dout = make(torch.float16, 64, 4, 2, [70, 1, 200], [90, 400, 3])
    cu_q, cu_k = ints([0, 70, 71, 271]), ints([0, 90, 490, 493])

    def step():
        out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
        return (out, lse, *m.rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = step()
    for i in range(4):
        for t in (q, k, v, dout):
            t.normal_()
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for x, y in zip(result, eager):
            assert torch.equal(x, y)


def test_given_workspace_and_other_stream():
    m = rvq()
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, [3, 60], [3000, 200])
    cu_q, cu_k = ints([0, 3, 63]), ints([0, 3000, 3200])
    want = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
    size = m.rvq_cross_attention_bytes(q, k, v, cu_q, cu_k)
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = m.rvq_cross_attention(q, k, v, cu_q, cu_k, out=torch.empty_like(q), workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    size = m.rvq_cross_attention_backward_bytes(q, k, v, cu_q, cu_k)
    with pytest.raises(m.RVQError):
        m.rvq_cross_attention_backward(dout, q, k, v, *want, cu_q, cu_k,
                                       workspace=torch.empty(size - 16, dtype=torch.uint8, device=DEV))
