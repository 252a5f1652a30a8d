"""Windowed attention with sinks and its gradient on the GPU against float64 (attention_oracle)."""

import math

import pytest
import torch

import attention_oracle as oracle
from gpu_util import DEV, announce, needs_gpu, rvq

pytestmark = [pytest.mark.gpu, needs_gpu]

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def offsets(lens):
    return [0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(typ, dim, hq, hk, q_lens, k_lens, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(typ).to(DEV)

    tq, tk = sum(q_lens), sum(k_lens)
    if fused:
        x = normal(tq, hq + 2 * hk, dim)
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], normal(tq, hq, dim)
    return normal(tq, hq, dim), normal(tk, hk, dim), normal(tk, hk, dim), normal(tq, hq, dim)


def close(name, got, want):
    value, bound = want
    got = got.double().cpu()
    assert got.shape == value.shape
    finite = torch.isfinite(value)
    assert torch.equal(got[~finite], value[~finite]), f"{name}: infinities differ"
    off = (got - value).abs()[finite] / bound[finite].clamp(min=1e-300)
    worst = off.max().item() if off.numel() else 0.0
    print(f"{name}: {worst:.3f} of the bound", flush=True)
    assert not torch.isnan(got[finite]).any(), f"{name}: NaN"
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound"


def check(typ, dim, hq, hk, q_lens, k_lens=None, window=None, sinks=0, scale=None, fused=False, train=True, seed=0):
    m = rvq()
    k_lens = q_lens if k_lens is None else k_lens
    announce("attention", typ=typ, dim=dim, heads=(hq, hk), q=q_lens, k=k_lens, window=window, sinks=sinks)
    q, k, v, dout = make(TYPES[typ], dim, hq, hk, q_lens, k_lens, seed, fused)
    cu_q, cu_k = offsets(q_lens), offsets(k_lens)
    args = dict(window=window, sinks=sinks, scale=scale)
    out, lse = m.rvq_window_attention(q, k, v, ints(cu_q), ints(cu_k), **args)
    torch.cuda.synchronize()
    want = oracle.attention(q, k, v, cu_q, cu_k, window, sinks, 1 / math.sqrt(dim) if scale is None else scale,
                            dout if train else None)
    close("out", out, want["out"])
    close("lse", lse, want["lse"])
    if train:
        grads = m.rvq_window_attention_backward(dout, q, k, v, out, lse, ints(cu_q), ints(cu_k), **args)
        torch.cuda.synchronize()
        for name, got in zip(("dq", "dk", "dv"), grads):
            close(name, got, want[name])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("typ", list(TYPES))
def test_one_frame_and_short_clips(typ, dim):
    check(typ, dim, 2, 1, [1])
    check(typ, dim, 3, 3, [1, 0, 2, 17, 0, 25])


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("length", [31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 300])
def test_lengths_around_tiles(typ, dim, length):
    check(typ, dim, 2, 1, [length, 5], window=None if length % 2 else 70, sinks=3)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (1, 1), (2, 40), (32, 0), (33, 1), (64, 4), (65, 70),
                                          (127, 33), (128, 64), (200, 5), (1000, 2), (None, 9)])
@pytest.mark.parametrize("typ", list(TYPES))
def test_windows_and_sinks(typ, window, sinks):
    check(typ, 64, 4, 2, [300, 40, 129], window=window, sinks=sinks, seed=window or 0)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (5, 5), (8, 2), (7, 1), (12, 4)])
def test_head_groups(hq, hk):
    check("bf16", 64, hq, hk, [150, 33], window=90, sinks=2)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("window,sinks", [(None, 0), (50, 3)])
def test_queries_continue_known_frames(typ, window, sinks):
    check(typ, 64, 4, 2, [1, 70, 130, 5], [140, 200, 130, 64], window=window, sinks=sinks)


@pytest.mark.parametrize("typ", list(TYPES))
def test_more_queries_than_keys_leave_empty_rows(typ):
    check(typ, 64, 2, 1, [80, 5, 3], [10, 0, 1])
    check(typ, 128, 2, 2, [200], [70], window=20, sinks=2)


@pytest.mark.parametrize("typ", list(TYPES))
def test_many_sink_rows_far_from_their_queries(typ):
    check(typ, 64, 2, 1, [1500], window=40, sinks=70)
    check(typ, 64, 4, 1, [1100, 700], window=100, sinks=4)


@pytest.mark.parametrize("typ,dim,q_lens,k_lens,window,sinks", [
    ("bf16", 64, [4500], None, 100, 4), ("fp32", 64, [4700, 90, 1500], None, 300, 64), ("fp16", 128, [4200], [4400], 129, 33),
    ("fp32", 128, [4300], [4300], 0, 5)])
def test_sinks_of_long_clips(typ, dim, q_lens, k_lens, window, sinks):
    """Clips long enough for the sinks' gradients to be added up from pieces."""
    check(typ, dim, 2, 1, q_lens, k_lens, window=window, sinks=sinks)


@pytest.mark.parametrize("typ,dim,hq,hk,q_lens,k_lens,window", [
    ("bf16", 64, 8, 1, [700], None, None), ("fp16", 128, 7, 1, [500, 0, 333], None, None), ("fp32", 64, 5, 1, [300], [380], 90),
    ("bf16", 128, 12, 2, [450, 130], None, 300)])
def test_query_heads_shared_out(typ, dim, hq, hk, q_lens, k_lens, window):
    """Few key heads and clips: several workgroups share the query heads of a key head."""
    check(typ, dim, hq, hk, q_lens, k_lens, window=window, sinks=2)


def test_large_scores_and_other_scales():
    check("bf16", 64, 2, 1, [140], scale=3.0, train=False)
    check("fp32", 64, 2, 1, [140], scale=0.0)
    check("fp16", 128, 2, 1, [140], scale=0.7, train=False)


@pytest.mark.parametrize("typ", ["bf16", "fp32"])
def test_slices_of_a_fused_projection(typ):
    check(typ, 64, 6, 2, [130, 41], window=60, sinks=2, fused=True)


def test_gradients_into_slices_and_another_order_of_dims():
    m = rvq()
    lens = [100, 37]
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, lens, lens)
    cu = ints(offsets(lens))
    out, lse = m.rvq_window_attention(q, k, v, cu, window=30, sinks=1)
    plain = m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, window=30, sinks=1)
    # head-major storage, and gradients into one buffer whose other parts stay
    hq, hk, hv, hd = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, dout))
    buffer = torch.full((sum(lens), 10, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out2, lse2 = m.rvq_window_attention(hq, hk, hv, cu, window=30, sinks=1)
    m.rvq_window_attention_backward(hd, hq, hk, hv, out2, lse2, cu, window=30, sinks=1,
                                    grads=(buffer[:, :4], buffer[:, 4:6], buffer[:, 7:9]))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for a, b in zip(plain, (buffer[:, :4], buffer[:, 4:6], buffer[:, 7:9])):
        assert torch.equal(a, b)
    assert (buffer[:, 6] == 7).all() and (buffer[:, 9] == 7).all()


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_seen_do_not_matter(typ, bad):
    """Frame j is not finite: frames that do not see it keep their output bit for bit."""
    m = rvq()
    n, window = 200, 50
    q, k, v, _ = make(TYPES[typ], 64, 2, 1, [n], [n])
    cu = ints([0, n])
    for j in (0, 37, 64, 150, 199):
        sinks = 2
        clean, lse = m.rvq_window_attention(q, k, v, cu, window=window, sinks=sinks)
        k2, v2 = k.clone(), v.clone()
        k2[j, 0, 5] = bad
        v2[j] = bad
        blind = ~oracle.sees(n, n, window, sinks)[:, j]
        got, got_lse = m.rvq_window_attention(q, k2, v2, cu, window=window, sinks=sinks)
        assert torch.equal(got[blind.to(DEV)], clean[blind.to(DEV)]), f"frame {j}"
        assert torch.equal(got_lse[:, blind.to(DEV)], lse[:, blind.to(DEV)])
        got, _ = m.rvq_window_attention(q, k, v2, cu, window=window, sinks=sinks)
        assert torch.equal(got[blind.to(DEV)], clean[blind.to(DEV)]), f"frame {j}"
        assert not torch.isfinite(got[(~blind).to(DEV)]).any()


def test_scores_of_minus_infinity():
    m = rvq()
    q, k, v, _ = make(torch.float32, 64, 1, 1, [40], [40])
    q[...] = q.abs()
    k[10:] = -math.inf
    out, lse = m.rvq_window_attention(q, k, v, ints([0, 40]), window=5)
    assert torch.isfinite(out[:14]).all()
    assert (out[14:] == 0).all() and (lse[:, 14:] == -math.inf).all()


def test_rows_outside_the_clips_are_left():
    m = rvq()
    q, k, v, dout = make(torch.bfloat16, 64, 2, 1, [60], [60])
    cu = ints([10, 30, 50])
    out = torch.full_like(q, 5.0)
    _, lse = m.rvq_window_attention(q, k, v, cu, out=out)
    grads = tuple(torch.full_like(x, 5.0) for x in (q, k, v))
    m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, grads=grads)
    for x in (out, *grads):
        assert (x[:10] == 5).all() and (x[50:] == 5).all() and not (x[10:50] == 5).all()


def test_the_same_bits_every_time_and_alone():
    """A clip's results do not depend on the call or on the clips beside it."""
    m = rvq()
    lens = [333, 70, 128]
    q, k, v, dout = make(torch.bfloat16, 128, 4, 2, lens, lens)
    cu = ints(offsets(lens))

    def both(q, k, v, dout, cu):
        out, lse = m.rvq_window_attention(q, k, v, cu, window=100, sinks=3)
        return (out, *m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, window=100, sinks=3))

    first = both(q, k, v, dout, cu)
    for a, b in zip(first, both(q, k, v, dout, cu)):
        assert torch.equal(a, b)
    s = slice(333, 403)
    for a, b in zip(first, both(q[s], k[s], v[s], dout[s], ints([0, 70]))):
        assert torch.equal(a[s], b)


@pytest.mark.parametrize("typ", list(TYPES))
def test_gradient_is_the_slope(typ):
    """<dq, step> etc. against central differences of the float64 forward: the gradient kernels against the
    function itself, at the types' rounding (the float64 values of the same inputs are differentiated)."""
    m = rvq()
    lens, window, sinks = [90], 33, 2
    q, k, v, dout = make(TYPES[typ], 64, 2, 1, lens, lens, seed=4)
    cu = [0, 90]
    out, lse = m.rvq_window_attention(q, k, v, ints(cu), window=window, sinks=sinks)
    grads = m.rvq_window_attention_backward(dout, q, k, v, out, lse, ints(cu), window=window, sinks=sinks)
    want = oracle.attention(q, k, v, cu, cu, window, sinks, 1 / 8, dout)
    g = torch.Generator().manual_seed(9)
    base = [x.double().cpu() for x in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        step = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        h, value = 1e-4, []
        for sign in (1, -1):
            moved = list(base)
            moved[i] = base[i] + sign * h * step
            o = oracle.attention(*moved, cu, cu, window, sinks, 1 / 8)["out"][0]
            value.append((o * dout.double().cpu()).sum())
        slope = (value[0] - value[1]) / (2 * h)
        got = (grads[i].double().cpu() * step).sum()
        bound = (want[name][1] * step.abs()).sum() + 1e-5 * slope.abs() + 1e-6
        assert abs(got - slope) <= bound, (name, got, slope, bound)


def test_another_stream_and_a_graph():
    m = rvq()
    lens = [200, 60]
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, lens, lens)
    cu = ints(offsets(lens))

    def both():
        out, lse = m.rvq_window_attention(q, k, v, cu, window=64, sinks=2)
        return (out, *m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, window=64, sinks=2))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for turn in range(4):
        with torch.no_grad():
            q.normal_()
            dout.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, both()):
            assert torch.equal(a, b), f"replay {turn}"
        torch.cuda.synchronize()


def test_refusals():
    m = rvq()
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, [20], [20])
    cu = ints([0, 20])
    call = m.rvq_window_attention
    with pytest.raises(TypeError):
        call(q, k.float(), v, cu)
    with pytest.raises(TypeError):
        call(q.double(), k.double(), v.double(), cu)
    with pytest.raises(ValueError):
        call(q[:, :3], k, v, cu)                 # 3 query heads over 2
    with pytest.raises(ValueError):
        call(q, k, v[:, :1], cu)
    with pytest.raises(ValueError):
        call(q, k[:10], v[:10], cu)              # cu_k missing
    with pytest.raises(ValueError):
        call(q, k, v, cu, ints([0, 10, 20]))
    with pytest.raises(ValueError):
        call(q, k, v, cu, window=-1)
    with pytest.raises(ValueError):
        call(q, k, v, cu, sinks=-1)
    with pytest.raises(ValueError):
        call(q.cpu(), k.cpu(), v.cpu(), cu.cpu())
    with pytest.raises(TypeError):
        call(q, k, v, cu.long())
    for scale in (-1.0, math.nan, math.inf):
        with pytest.raises(m.RVQError) as e:
            call(q, k, v, cu, scale=scale)
        assert e.value.status == m.RVQ_ERR_INVALID_ARG
    with pytest.raises(m.RVQError) as e:
        call(q[..., :32], k[..., :32], v[..., :32], cu)
    assert e.value.status == m.RVQ_ERR_UNSUPPORTED
    odd = torch.zeros(20 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(20, 4, 64)
    with pytest.raises(m.RVQError) as e:
        call(odd, k, v, cu)                      # not 16-byte aligned
    assert e.value.status == m.RVQ_ERR_INVALID_ARG
    with pytest.raises(m.RVQError) as e:
        call(q, k, v, cu, out=q[:1].expand(20, 4, 64))      # output rows on top of each other
    assert e.value.status == m.RVQ_ERR_INVALID_ARG
    out, lse = call(q, k, v, cu)
    with pytest.raises(ValueError):
        m.rvq_window_attention_backward(dout, q, k, v, out, lse[:, :5].contiguous(), cu)
    with pytest.raises(ValueError):
        m.rvq_window_attention_backward(dout[:5], q, k, v, out, lse, cu)


def test_nothing_to_do():
    m = rvq()
    q, k, v, dout = make(torch.bfloat16, 64, 4, 2, [0], [0])
    out, lse = m.rvq_window_attention(q, k, v, ints([0]))
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    m.rvq_window_attention_backward(dout, q, k, v, out, lse, ints([0, 0]))
    # keys that no query sees
    _, k, v, _ = make(torch.bfloat16, 64, 4, 2, [0], [70])
    dq, dk, dv = m.rvq_window_attention_backward(dout, q, k, v, out, lse, ints([0, 0]), ints([0, 70]))
    assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("typ", list(TYPES))
def test_gradients_of_frames_apart_from_one_that_is_not_finite(typ):
    """Frame j is not finite: queries that do not see it, and keys that no query with it sees, keep their gradients."""
    m = rvq()
    n, window, sinks = 300, 40, 2
    q, k, v, dout = make(TYPES[typ], 64, 2, 1, [n], [n])
    cu = ints([0, n])
    out, lse = m.rvq_window_attention(q, k, v, cu, window=window, sinks=sinks)
    clean = m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, window=window, sinks=sinks)
    sees = oracle.sees(n, n, window, sinks).to(DEV)
    for j in (37, 100, 160, 299):
        for bad in (math.nan, math.inf):
            for which in ("k", "v", "q", "dout"):
                args = dict(q=q, k=k, v=v, dout=dout)
                args[which] = args[which].clone()
                args[which][j, 0, 7] = bad
                x = [args[name] for name in ("dout", "q", "k", "v")]
                o, s = m.rvq_window_attention(*x[1:], cu, window=window, sinks=sinks)
                dq, dk, dv = m.rvq_window_attention_backward(*x, o, s, cu, window=window, sinks=sinks)
                hurt = sees[:, j] if which in "kv" else torch.arange(n, device=DEV) == j     # queries
                blind = ~(sees & hurt[:, None]).any(0)                                       # keys none of them sees
                assert torch.equal(dq[~hurt], clean[0][~hurt]), (j, bad, which)
                assert torch.equal(dk[blind], clean[1][blind]) and torch.equal(dv[blind], clean[2][blind]), (j, bad, which)
                assert not torch.isfinite(dq[hurt][:, 0]).all(-1).any()


def test_float16_gradients_of_small_and_large_size():
    """dout of 2^-12 and of 2^9: the same relative error as at 1, to float16's own range."""
    m = rvq()
    lens = [500]
    q, k, v, dout = make(torch.float16, 64, 2, 1, lens, lens)
    cu = ints(offsets(lens))
    out, lse = m.rvq_window_attention(q, k, v, cu)
    for power in (-12, 9):
        g = dout * 2.0 ** power
        want = oracle.attention(q, k, v, offsets(lens), offsets(lens), None, 0, 1 / 8, g)
        for name, x in zip(("dq", "dk", "dv"), m.rvq_window_attention_backward(g, q, k, v, out, lse, cu)):
            close(name, x, want[name])
