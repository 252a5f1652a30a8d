"""Rotary positions, the paged cache, chunk and cross attention as a streaming decoder layer uses them together, and in
training; tables and pools of more than 4 GiB.

Several rounded steps follow one another here, so each is held to the bound of its own oracle on the inputs that it
really had, and what has to be equal is compared bit for bit.
"""

import math
import random

import pytest
import torch

import attention_oracle
import cross_oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, offsets
from test_gpu_chunk import want as chunk_want
from test_gpu_rotary import turned

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("typ,dim,hq,hk,window,sinks", [("bf16", 64, 4, 2, None, 0), ("fp16", 128, 8, 2, 40, 3), ("fp32", 64, 2, 2, 25, 0)])
def test_streams_in_pieces(typ, dim, hq, hk, window, sinks):
    """Clips come in pieces of uneven length, single frames among them; pages behind the window are given back."""
    m, rng, g = rvq(), random.Random(4), torch.Generator().manual_seed(4)
    announce("decoder layer", typ=typ, dim=dim, heads=(hq, hk), window=window, sinks=sinks)
    lens, states, page = [70, 5, 133, 0, 40], [30, 0, 200, 7, 1], 8
    clips, total = len(lens), sum(lens)
    normal = lambda *s: torch.randn(*s, generator=g).to(TYPES[typ]).to(DEV)     # noqa: E731
    qkv, query = normal(total, hq + 2 * hk, dim), normal(total, hq, dim)
    kv = normal(sum(states), 2 * hk, dim)
    f = m.rvq_rotary_frequencies(dim // 2).to(DEV)
    first = [sum(lens[:b]) for b in range(clips)]

    # whole clips at once
    cu, cu_k = ints(offsets(lens)), ints(offsets(states))
    q_all, k_all = m.rvq_rotary(qkv[:, :hq], qkv[:, hq:hq + hk], f, cu=cu)
    whole, whole_lse = m.rvq_window_attention(q_all, k_all, qkv[:, hq + hk:], cu, window=window, sinks=sinks)
    close("whole", whole, attention_oracle.attention(q_all, k_all, qkv[:, hq + hk:], offsets(lens), offsets(lens), window, sinks,
                                                     1 / math.sqrt(dim))["out"])
    cross_all, _ = m.rvq_cross_attention(query, kv[:, :hk], kv[:, hk:], cu, cu_k)

    # in pieces
    cols = -(-max(lens) // page)
    pages = clips * cols + 2
    pools = [torch.full((pages, hk, page, dim), math.nan, dtype=TYPES[typ], device=DEV) for _ in range(2)]
    table = torch.full((clips, cols), -1, dtype=torch.int32, device=DEV)
    counts, refs = ints([0] * clips), ints([0] * pages)
    done = [0] * clips
    out, lse = torch.zeros_like(whole), torch.full_like(whole_lse, 7.0)
    crossed = torch.zeros_like(cross_all)
    while any(d < n for d, n in zip(done, lens)):
        new = [min(n - d, rng.choice([0, 1, 1, 4, 33, 90])) for d, n in zip(done, lens)]
        rows = [first[b] + done[b] + i for b in range(clips) for i in range(new[b])]
        if not rows:
            continue
        more = counts + ints(new)
        table, refs, missing = m.rvq_cache_reserve(table, counts, more, refs, page)
        assert missing.item() == 0
        x, cu_new = qkv[rows], ints(offsets(new))
        q = m.rvq_rotary_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], f, *pools, table, counts, cu_new)
        assert torch.equal(q, q_all[rows])
        counts = more
        part, part_lse = m.rvq_cache_chunk_attention(q, *pools, table, counts, cu_new, window=window, sinks=sinks)
        out[rows], lse[:, rows] = part, part_lse
        crossed[rows] = m.rvq_cross_attention(query[rows], kv[:, :hk], kv[:, hk:], cu_new, cu_k)[0]
        table, counts, refs = m.rvq_cache_free(table, counts, refs, page, window=window, sinks=sinks)
        done = [d + n for d, n in zip(done, new)]
    torch.cuda.synchronize()
    want = attention_oracle.attention(q_all, k_all, qkv[:, hq + hk:], offsets(lens), offsets(lens), window, sinks, 1 / math.sqrt(dim))
    close("pieces", out, want["out"])
    close("lse", lse, want["lse"])
    want = cross_oracle.attention(query, kv[:, :hk], kv[:, hk:], offsets(lens), offsets(states), 1 / math.sqrt(dim))
    close("cross", crossed, want["out"])
    close("cross whole", cross_all, want["out"])


@pytest.mark.parametrize("typ", list(TYPES))
def test_training_step(typ):
    """Rotation, windowed attention, cross attention with its output as queries, and all gradients back to the
    projection; each gradient against its own formula, then the rotation's."""
    m, g = rvq(), torch.Generator().manual_seed(6)
    announce("training step", typ=typ)
    lens, states, h, dim = [50, 0, 130, 1], [20, 9, 70, 0], 4, 64
    normal = lambda *s: torch.randn(*s, generator=g).to(TYPES[typ]).to(DEV)     # noqa: E731
    qkv, kv, dout = normal(sum(lens), 3 * h, dim), normal(sum(states), 2 * h, dim), normal(sum(lens), h, dim)
    f, cu, cu_k = m.rvq_rotary_frequencies(dim).to(DEV), ints(offsets(lens)), ints(offsets(states))
    position = torch.tensor([i for n in lens for i in range(n)])

    q, k = m.rvq_rotary(qkv[:, :h], qkv[:, h:2 * h], f, cu=cu)
    v = qkv[:, 2 * h:]
    mid, lse = m.rvq_window_attention(q, k, v, cu, window=30)
    out, cross_lse = m.rvq_cross_attention(mid, kv[:, :h], kv[:, h:], cu, cu_k)
    dkv = torch.empty_like(kv)
    dmid, dk2, dv2 = m.rvq_cross_attention_backward(dout, mid, kv[:, :h], kv[:, h:], out, cross_lse, cu, cu_k,
                                                    grads=(torch.empty_like(mid), dkv[:, :h], dkv[:, h:]))
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = m.rvq_window_attention_backward(dmid, q, k, v, mid, lse, cu, window=30,
                                                 grads=(dqkv[:, :h], dqkv[:, h:2 * h], dqkv[:, 2 * h:]))
    before = dqkv.clone()
    m.rvq_rotary(dq, dk, f, cu=cu, inverse=True, out=(dq, dk))      # in place, in the fused gradient
    torch.cuda.synchronize()

    want = cross_oracle.attention(mid, kv[:, :h], kv[:, h:], offsets(lens), offsets(states), 0.125, dout)
    for name, got in (("out", out), ("dq", dmid), ("dk", dk2), ("dv", dv2)):
        close(name, got, want[name])
    want = attention_oracle.attention(q, k, v, offsets(lens), offsets(lens), 30, 0, 0.125, dmid)
    for name, got in (("dq", before[:, :h]), ("dk", before[:, h:2 * h]), ("dv", before[:, 2 * h:])):
        close(name, got, want[name])
    assert torch.equal(dqkv[:, 2 * h:], before[:, 2 * h:])
    for at in (slice(0, h), slice(h, 2 * h)):
        value, bound = turned(before[:, at], position, f.cpu(), False, 1.0, -1)
        assert ((dqkv[:, at].double().cpu() - value).abs() <= bound).all()


@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("fp32", 64)])
def test_pools_of_more_than_4_gib(typ, dim):
    """Pages at the far end of pools whose byte offsets, and in the bfloat16 case whose value offsets too, pass 32 bits."""
    m, g, hk, page = rvq(), torch.Generator().manual_seed(8), 2, 64
    size = 2 if typ == "bf16" else 4
    pages = (9 << 30 if typ == "bf16" else 5 << 30) // (hk * page * dim * size)
    pools = [torch.empty(pages, hk, page, dim, dtype=TYPES[typ], device=DEV) for _ in range(2)]
    past, new = [100, 60], [3, 90]
    lens = [a + b for a, b in zip(past, new)]
    table, last = [], pages - 1
    for n in lens:
        table.append([last - i for i in range(3)])
        last -= 3
    used = sorted(p for row in table for p in row)
    small = [torch.randn(len(used), hk, page, dim, generator=g).to(TYPES[typ]) for _ in range(2)]
    for pool, x in zip(pools, small):
        pool[used[0]:used[-1] + 1] = x.to(DEV)
    near = [[used.index(p) for p in row] for row in table]
    f = m.rvq_rotary_frequencies(dim).to(DEV)
    qkv = torch.randn(sum(new), 8, dim, generator=g).to(TYPES[typ]).to(DEV)
    close_pools = [x.to(DEV) for x in small]
    for where, t in ((pools, table), (close_pools, near)):
        q = m.rvq_rotary_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], f, *where, ints(t), ints(past), ints(offsets(new)))
        got = m.rvq_cache_chunk_attention(q, *where, ints(t), ints(lens), ints(offsets(new)))
        if where is pools:
            far = got
    torch.cuda.synchronize()
    assert torch.equal(far[0], got[0]) and torch.equal(far[1], got[1])
    for pool, x in zip(pools, close_pools):
        assert torch.equal(pool[used[0]:used[-1] + 1], x)
    ref = chunk_want(q, *close_pools, near, lens, new, None, 0, 1 / math.sqrt(dim))
    close("out", got[0], ref["out"])


def test_the_same_pages_in_several_clips():
    """Forked clips share pages: drafts that go on from one past, each with frames of its own."""
    m, g = rvq(), torch.Generator().manual_seed(9)
    past, drafts, new, page = 37, 3, 4, 8
    pools = [torch.zeros(40, 2, page, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.full((drafts + 1, 8), -1, dtype=torch.int32, device=DEV)
    counts, refs = ints([0] * (drafts + 1)), ints([0] * 40)
    x = torch.randn(past, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    f = m.rvq_rotary_frequencies(64).to(DEV)
    more = ints([past] + [0] * drafts)
    table, refs, _ = m.rvq_cache_reserve(table, counts, more, refs, page)
    m.rvq_rotary_append(None, x[:, 4:6], x[:, 6:], f, *pools, table, counts, ints([0, past] + [past] * drafts))
    counts = more
    parents, children = ints([0] * drafts), ints(range(1, drafts + 1))
    table, counts, refs, missing = m.rvq_cache_fork(table, counts, refs, parents, children, *pools)
    assert missing.item() == 0
    y = torch.randn(drafts * new, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    cu = [0, 0] + [new * (i + 1) for i in range(drafts)]
    more = counts + ints([0] + [new] * drafts)
    table, refs, missing = m.rvq_cache_reserve(table, counts, more, refs, page)
    assert missing.item() == 0
    q = m.rvq_rotary_append(y[:, :4], y[:, 4:6], y[:, 6:], f, *pools, table, counts, ints(cu))
    out, lse = m.rvq_cache_chunk_attention(q, *pools, table, more, ints(cu))
    torch.cuda.synchronize()
    _, k = m.rvq_rotary(None, x[:, 4:6], f, cu=ints([0, past]))
    for b in range(drafts):
        rows = slice(b * new, (b + 1) * new)
        _, own = m.rvq_rotary(None, y[rows, 4:6], f, cu=ints([0, new]), first=ints([past]))
        want = attention_oracle.attention(q[rows], torch.cat([k, own]), torch.cat([x[:, 6:], y[rows, 6:]]), [0, new],
                                          [0, past + new], None, 0, 0.125)
        close("out", out[rows], want["out"])
        close("lse", lse[:, rows].contiguous(), want["lse"])
