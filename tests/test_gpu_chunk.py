"""Attention of chunks of new frames over the paged cache on the GPU against float64 (attention_oracle), whose bounds
hold here as they are: the products, the weights' rounding and the sums are the windowed attention's."""

import math

import pytest
import torch

import attention_oracle as oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, offsets
from test_gpu_cache import cache

pytestmark = [pytest.mark.gpu, needs_gpu]


def gathered(pool, table, lens):
    """The clips' rows packed; zeros where the table has no page."""
    page, pool, rows = pool.shape[2], pool.cpu(), []
    for b, n in enumerate(lens):
        for j in range(n):
            p = table[b][j // page]
            rows.append(pool[p, :, j % page] if p >= 0 else torch.zeros(pool.shape[1], pool.shape[3], dtype=pool.dtype))
    return torch.stack(rows) if rows else torch.zeros(0, pool.shape[1], pool.shape[3], dtype=pool.dtype)


def want(q, k_pool, v_pool, table, lens, new, window, sinks, scale):
    return oracle.attention(q, gathered(k_pool, table, lens), gathered(v_pool, table, lens), offsets(new), offsets(lens),
                            window, sinks, scale)


def check(typ, dim, hq, hk, page, past, new, window=None, sinks=0, scale=None, seed=0):
    m = rvq()
    announce("chunk", typ=typ, dim=dim, heads=(hq, hk), page=page, past=past, new=new, window=window, sinks=sinks)
    lens = [a + b for a, b in zip(past, new)]
    reach = None if window is None else window + max(new)      # what the first of the new frames sees stays
    k, v, table, _ = cache(typ, dim, hk, page, lens, seed=seed, window=reach, sinks=sinks)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(sum(new), hq, dim, generator=g).to(TYPES[typ]).to(DEV)
    out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(lens), ints(offsets(new)), window=window,
                                           sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    ref = want(q, k, v, table, lens, new, window, sinks, 1 / math.sqrt(dim) if scale is None else scale)
    close("out", out, ref["out"])
    close("lse", lse, ref["lse"])
    return m, q, k, v, table, lens, out, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [1, 7, 16, 100])
def test_lengths_and_pages(typ, dim, page):
    check(typ, dim, 4, 2, page, [0, 5, 0, 31, 200, 64, 63, 1, 0], [1, 1, 0, 2, 3, 9, 1, 5, 8])
    check(typ, dim, 2, 1, page, [0, 70, 130], [150, 40, 0])


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("new", [8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_chunks_around_tiles(typ, dim, new):
    """One clip alone, and one beside others with a frame each."""
    check(typ, dim, 2, 1, 16, [100], [new], window=None if new % 2 else 70, sinks=3)
    check(typ, dim, 2, 1, 16, [100] + [40, 0, 9] * 7, [new] + [1] * 21, window=None if new % 2 else 70, sinks=3)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (5, 5), (16, 1), (17, 1), (24, 1), (40, 1), (33, 1), (96, 1), (12, 4), (32, 8)])
@pytest.mark.parametrize("typ", ["bf16", "fp32"])
def test_head_groups(typ, hq, hk):
    check(typ, 64, hq, hk, 16, [200, 3, 77], [4, 1, 2])
    check(typ, 64, hq, hk, 16, [200, 3, 77], [1, 60, 35], window=50, sinks=1)
    check(typ, 64, hq, hk, 16, [90], [70])


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 2), (1, 0), (1, 4), (16, 3), (33, 40), (64, 64), (100, 1), (4000, 3), (None, 5)])
@pytest.mark.parametrize("typ", list(TYPES))
def test_windows_and_sinks(typ, window, sinks):
    check(typ, 64, 4, 2, 16, [300, 16, 0, 65, 10, 128], [3, 1, 5, 4, 0, 2], window=window, sinks=sinks)
    check(typ, 64, 4, 2, 16, [300, 16, 0, 65], [130, 1, 40, 2], window=window, sinks=sinks)
    check(typ, 128, 2, 1, 16, [200], [180], window=window, sinks=sinks)


@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("fp16", 64), ("fp32", 128)])
def test_long_caches_are_split_and_joined(typ, dim):
    check(typ, dim, 4, 2, 32, [5000, 12, 4097, 2049], [4, 1, 8, 3])
    check(typ, dim, 2, 1, 24, [9001], [100])
    check(typ, dim, 2, 1, 32, [3000, 700, 4, 5, 60], [130, 1, 2, 90, 1])
    check(typ, dim, 2, 1, 32, [3000, 700], [130, 1], window=2000, sinks=70)


@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("fp16", 64), ("fp32", 128), ("fp32", 64)])
def test_two_sets_of_rows(typ, dim):
    """17 to 32 rows a clip: alone, with a clip of more beside them, and a clip of many in turns."""
    check(typ, dim, 8, 1, 16, [100, 700, 3], [4, 3, 4], window=300, sinks=2)
    check(typ, dim, 16, 2, 16, [100] * 20, [4] * 17 + [40, 1, 3])
    check(typ, dim, 8, 1, 16, [3000, 3], [29, 3])


def test_many_clips():
    """Offsets searched in more than one step, and blocks of queries found by marks."""
    past = [(37 * b) % 90 for b in range(200)]
    check("bf16", 64, 2, 1, 16, past, [1 if b % 3 else 0 for b in range(200)])
    check("bf16", 64, 2, 1, 16, past, [1 if b % 50 else 40 for b in range(200)])
    check("bf16", 64, 1, 1, 16, past, [1 if b % 50 else 140 for b in range(200)], window=30)
    check("fp16", 64, 8, 1, 16, past[:70], [5 if b % 5 else 0 for b in range(70)])


@pytest.mark.parametrize("typ", list(TYPES))
def test_one_longer_clip_among_few_rows(typ):
    """So few rows in all that one kind of workgroup takes them, a longer clip in turns; with its last values not finite,
    and over keys that are split."""
    check(typ, 64, 4, 2, 16, [40, 3, 90], [14, 1, 2], window=30, sinks=2)
    check(typ, 128, 2, 1, 16, [5000, 10, 10], [14, 1, 1])
    m, lens, new = rvq(), [54, 4, 92], [14, 1, 2]
    k, v, table, _ = cache(typ, 64, 2, 16, lens)
    q = torch.randn(17, 4, 64, generator=torch.Generator().manual_seed(3)).to(TYPES[typ]).to(DEV)
    ref = want(q, k, v, table, lens, new, None, 0, 0.125)
    v = v.clone()
    v[table[0][53 // 16], :, 53 % 16, 7] = math.inf
    v[table[0][51 // 16], 1, 51 % 16, 9] = math.nan
    out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(lens), ints(offsets(new)))
    fine = [i for i in range(17) if i not in (11, 12, 13)]
    close("out", out[fine], tuple(x[fine] for x in ref["out"]))
    close("lse", lse, ref["lse"])
    odd = ~torch.isfinite(out[11:14]).cpu()
    assert odd[2, :, 7].all() and odd[:, 2:, 9].all() and not odd[:, :2, 9].any() and not odd[:2, :, 7].any()
    assert odd.sum() == 4 + 6


def test_two_calls_at_once():
    """On two streams, without anything in common."""
    m = rvq()
    sets = []
    for seed, (past, new) in enumerate((([9000, 40], [2, 1]), ([700, 3000, 40], [100, 1, 60]))):
        lens = [a + b for a, b in zip(past, new)]
        k, v, table, _ = cache("bf16", 64, 2, 16, lens, seed=seed)
        q = torch.randn(sum(new), 4, 64, device=DEV).to(torch.bfloat16)
        args = (q, k, v, ints(table), ints(lens), ints(offsets(new)))
        sets.append((args, m.rvq_cache_chunk_attention(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(5):
        got = []
        for args, _, stream in sets:
            with torch.cuda.stream(stream):
                got.append(m.rvq_cache_chunk_attention(*args))
        torch.cuda.synchronize()
        for x, (_, y, _) in zip(got, sets):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_other_scales():
    check("bf16", 64, 4, 2, 16, [300], [20], scale=2.5)
    check("fp32", 64, 4, 2, 16, [300], [5], scale=0.0)


@pytest.mark.parametrize("typ", list(TYPES))
def test_more_queries_than_frames_leave_empty_rows(typ):
    m = rvq()
    lens, new = [10, 0, 2], [80, 5, 3]
    k, v, table, _ = cache(typ, 64, 1, 16, lens)
    q = torch.randn(sum(new), 2, 64, generator=torch.Generator().manual_seed(3)).to(TYPES[typ]).to(DEV)
    out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(lens), ints(offsets(new)))
    ref = want(q, k, v, table, lens, new, None, 0, 0.125)
    close("out", out, ref["out"])
    close("lse", lse, ref["lse"])
    assert (out[:70] == 0).all() and (lse[:, :70] == -math.inf).all()


def test_one_frame_each_without_offsets():
    m = rvq()
    lens = [300, 1, 0, 65, 64, 5000]
    for typ, hq, hk in (("bf16", 4, 2), ("fp32", 2, 2), ("fp16", 40, 1)):
        k, v, table, _ = cache(typ, 64, hk, 16, lens)
        q = torch.randn(len(lens), hq, 64, generator=torch.Generator().manual_seed(3)).to(TYPES[typ]).to(DEV)
        args = (k, v, ints(table), ints(lens))
        out, lse = m.rvq_cache_chunk_attention(q, *args, window=200, sinks=2)
        close("out", out, oracle.cache_attention(q, k, v, ints(table), ints(lens), 200, 2, 0.125))
        again = m.rvq_cache_chunk_attention(q, *args, ints(range(len(lens) + 1)), window=200, sinks=2)
        torch.testing.assert_close(again[1], lse, rtol=0, atol=1e-5)
        assert lse[0, 2] == -math.inf


def test_rows_outside_clips_and_strides():
    m = rvq()
    lens, k_heads = [100, 40], 2
    k, v, table, _ = cache("bf16", 64, k_heads, 16, lens)
    wide = torch.randn(60, 9, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    q, cu = wide[:, 2:6], ints([7, 9, 50])
    to = torch.full((60, 8, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(lens), cu, out=to[:, 3:7])
    ref = want(q[7:50], k, v, table, lens, [2, 41], None, 0, 0.125)
    close("out", out[7:50], ref["out"])
    close("lse", lse[:, 7:50].contiguous(), ref["lse"])
    assert (to[:, :3] == 5).all() and (to[:, 7:] == 5).all() and (to[:7] == 5).all() and (to[50:] == 5).all()


def test_no_queries_no_clips():
    m = rvq()
    k, v, table, _ = cache("bf16", 64, 2, 16, [20])
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints([20]), ints([0, 0]))
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    out, _ = m.rvq_cache_chunk_attention(q, k, v, torch.empty(0, 3, dtype=torch.int32, device=DEV), ints([]), ints([0]))
    assert out.shape == (0, 4, 64)


# ---------------------------------------------------------------- values that are not finite, pages that are not there

@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("new", [5, 90])
def test_unseen_values_that_are_not_finite(typ, dim, new):
    """The last new frames' keys and values are infinite or NaN: only the queries that see them notice."""
    m, q, k, v, table, lens, out, lse = check(typ, dim, 2, 1, 16, [150, 40], [new, new], window=60, sinks=2)
    page, ref = k.shape[2], want(q, k, v, table, lens, [new, new], 60, 2, 1 / math.sqrt(dim))
    for value in (math.inf, -math.inf, math.nan):
        for pool in (k, v):
            bad = pool.clone()
            for b, n in enumerate(lens):
                for j in (n - 1, n - 3):
                    bad[table[b][j // page], 0, j % page, 5] = value
            # in places that no query sees: before the window
            bad[table[0][80 // page], 0, 80 % page] = value
            pools = (bad, v) if pool is k else (k, bad)
            got, got_lse = m.rvq_cache_chunk_attention(q, *pools, ints(table), ints(lens), ints(offsets([new, new])),
                                                       window=60, sinks=2)
            for b in range(2):
                fine = slice(b * new, b * new + new - 3)
                close("out", got[fine], tuple(x[fine] for x in ref["out"]))
                if pool is v:
                    assert not torch.isfinite(got[b * new + new - 1, :, 5]).any()
                    keep = [d for d in range(dim) if d != 5]
                    assert torch.isfinite(got[b * new + new - 1][:, keep]).all()


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("past,new", [([150, 40], [4, 6]), ([150, 40], [90, 3]), ([3000, 5000], [4, 120])])
def test_missing_pages_and_counts_beyond_the_table(typ, past, new):
    m, q, k, v, table, lens, out, lse = check(typ, 64, 2, 1, 16, past, new, window=50, sinks=2)
    cu, broken = offsets(new), [list(r) for r in table]
    # the page of a frame in the middle of clip 0's window, by a missing, a negative and a far page number
    j = lens[0] - 20
    for page in (-1, -7, k.shape[0], 2 ** 31 - 1):
        broken[0][j // 16] = page
        got, got_lse = m.rvq_cache_chunk_attention(q, k, v, ints(broken), ints(lens), ints(cu), window=50, sinks=2)
        for i in range(new[0]):
            p = lens[0] - new[0] + i
            seen = any(t <= p and p - t < 50 for t in range(j // 16 * 16, j // 16 * 16 + 16))
            row, stat = got[i], got_lse[:, i]
            assert torch.isnan(row).all() and torch.isnan(stat).all() if seen else torch.equal(row, out[i])
        assert torch.equal(got[cu[1]:], out[cu[1]:])
    far = [lens[0], len(table[1]) * 16 + 1]
    got, _ = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(far), ints(cu), window=50, sinks=2)
    assert torch.equal(got[:cu[1]], out[:cu[1]]) and torch.isnan(got[cu[1]:]).all()
    got, _ = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints([lens[0], 2 ** 31 - 1]), ints(cu))
    assert torch.isnan(got[cu[1]:]).all()
    nothing = k[:0]
    got, _ = m.rvq_cache_chunk_attention(q, nothing, nothing, ints(table), ints(lens), ints(cu), window=50, sinks=2)
    assert torch.isnan(got).all()


def test_scores_of_any_size():
    """One key far above the others, scores far below 0, all scores -inf."""
    m = rvq()
    for typ in TYPES:
        for new in (3, 70):
            lens = [200]
            k, v, table, _ = cache(typ, 64, 1, 16, lens)
            q = torch.randn(new, 1, 64, generator=torch.Generator().manual_seed(9)).to(TYPES[typ]).to(DEV)
            for scale in (1.0, 30.0):
                out, lse = m.rvq_cache_chunk_attention(q, k, v, ints(table), ints(lens), ints([0, new]), scale=scale)
                ref = want(q, k, v, table, lens, [new], None, 0, scale)
                close("out", out, ref["out"])
                close("lse", lse, ref["lse"])


# ---------------------------------------------------------------- graphs, workspaces

def test_captured_steps_share_nothing():
    """Two graphs of different shapes, replayed in turn with eager work between them."""
    m = rvq()
    graphs = []
    for seed, (past, new) in enumerate((([3000, 70], [3, 100]), ([500, 9000, 40], [1, 2, 1]))):
        lens = [a + b for a, b in zip(past, new)]
        k, v, table, _ = cache("bf16", 64, 2, 16, lens, seed=seed)
        q = torch.randn(sum(new), 4, 64, device=DEV).to(torch.bfloat16)
        args = (q, k, v, ints(table), ints(lens), ints(offsets(new)))
        m.rvq_cache_chunk_attention(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = m.rvq_cache_chunk_attention(*args)
        graphs.append((graph, args, result))
    for i in range(4):
        for graph, args, result in graphs:
            args[0].normal_()
            graph.replay()
            eager = m.rvq_cache_chunk_attention(*args)
            torch.cuda.synchronize()
            assert torch.equal(result[0], eager[0]) and torch.equal(result[1], eager[1])


def test_given_workspace_and_other_stream():
    m = rvq()
    lens, new = [5000, 300], [2, 60]
    k, v, table, _ = cache("fp16", 64, 2, 16, lens)
    q = torch.randn(62, 4, 64, device=DEV).to(torch.float16)
    args = (q, k, v, ints(table), ints(lens), ints(offsets(new)))
    want_out, want_lse = m.rvq_cache_chunk_attention(*args)
    size = m.rvq_cache_chunk_attention_bytes(k, args[3], 4, 62)
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, lse = m.rvq_cache_chunk_attention(*args, out=out, workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    assert got is out and torch.equal(got, want_out) and torch.equal(lse, want_lse)
    if size:
        with pytest.raises(m.RVQError):
            m.rvq_cache_chunk_attention(*args, workspace=work[:size - 16])
