"""Chunk and cross attention on the GPU where values, keys or scores are not finite, with keys that are split among
workgroups and without, few rows a clip and many, against float64 (attention_oracle, cross_oracle).

A value that a query does not see has no influence on it. Of those seen (a score of -inf counts as not seen) an infinite
one makes the result infinite there, with its sign, however small its weight; NaN or both signs make it NaN. All other
results keep to the oracle's bounds.
"""

import math

import pytest
import torch

import attention_oracle
import cross_oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, make, offsets
from test_gpu_cache import cache
from test_gpu_chunk import gathered, want

pytestmark = [pytest.mark.gpu, needs_gpu]

VALUES = (math.inf, -math.inf, math.nan)


def signs(v, cu_q, cu_k, sees, heads):
    """Bool [Tq, heads, dim] each: whether some seen value is +inf or NaN, and -inf or NaN."""
    v = v.double().cpu()
    group = heads // v.shape[1]
    res = [torch.zeros(cu_q[-1], heads, v.shape[2], dtype=torch.bool) for _ in range(2)]
    for b in range(len(cu_q) - 1):
        rows = v[cu_k[b]:cu_k[b + 1]]
        mask = sees(cu_q[b + 1] - cu_q[b], len(rows)).double()
        for h in range(heads):
            x = rows[:, h // group]
            for to, bad in zip(res, (torch.isposinf(x) | torch.isnan(x), torch.isneginf(x) | torch.isnan(x))):
                to[cu_q[b]:cu_q[b + 1], h] = mask @ bad.double() > 0
    return res


def check_out(out, ref, plus, minus):
    """``ref``: (value, bound) with finite values in the place of the others."""
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), plus & minus)
    assert torch.equal(torch.isposinf(got), plus & ~minus)
    assert torch.equal(torch.isneginf(got), minus & ~plus)
    rest = ~(plus | minus)
    close("out", got[rest], tuple(x[rest] for x in ref))


# ---------------------------------------------------------------- signs of infinities that are seen

@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 64), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("new,past", [([1], [0]), ([1, 3], [0, 200]), ([20], [100]), ([90, 2], [40, 7]), ([1, 1], [3000, 9]),
                                      ([200], [3000]), ([30, 2], [3000, 9])])
@pytest.mark.parametrize("hq,hk", [(4, 2), (16, 2), (40, 2)])
def test_chunk_infinities_keep_their_sign(typ, dim, new, past, hq, hk):
    m, lens = rvq(), [a + b for a, b in zip(past, new)]
    announce("chunk, signs", typ=typ, dim=dim, past=past, new=new, heads=(hq, hk))
    k, v, table, _ = cache(typ, dim, hk, 16, lens)
    q = torch.randn(sum(new), hq, dim, generator=torch.Generator().manual_seed(2)).to(TYPES[typ]).to(DEV)
    ref = want(q, k, v, table, lens, new, None, 0, 1 / math.sqrt(dim))
    bad = v.clone()
    for b, n in enumerate(lens):
        for j, d, value in ((0, 3, math.inf), (n // 2, 4, -math.inf), (n - 1, 9, math.inf), (n // 3, 11, math.nan),
                            (0, 17, math.inf), (n // 2, 17, -math.inf), (n - 1, dim - 1, -math.inf)):
            bad[table[b][j // 16], 1, j % 16, d] = value
    marks = signs(gathered(bad, table, lens), offsets(new), offsets(lens),
                  lambda nq, nk: attention_oracle.sees(nq, nk, None, 0), hq)
    for cu in (ints(offsets(new)), *((None,) if set(new) == {1} else ())):
        out, lse = m.rvq_cache_chunk_attention(q, k, bad, ints(table), ints(lens), cu)
        torch.cuda.synchronize()
        close("lse", lse, ref["lse"])
        check_out(out, ref["out"], *marks)


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 64), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 70), (3, 2500), (7, 40), (90, 70), (200, 4000)])
def test_cross_infinities_keep_their_sign(typ, dim, nq, nk):
    m = rvq()
    announce("cross, signs", typ=typ, dim=dim, nq=nq, nk=nk)
    q, k, v, _ = make(TYPES[typ], dim, 4, 2, [nq, nq], [nk, 5])
    cu_q, cu_k = offsets([nq, nq]), offsets([nk, 5])
    ref = cross_oracle.attention(q, k, v, cu_q, cu_k, 1 / math.sqrt(dim))
    for j, d, value in ((0, 3, math.inf), (nk // 2, 4, -math.inf), (nk - 1, 9, math.inf), (nk // 3, 11, math.nan),
                        (0, 17, math.inf), (nk - 1, 17, -math.inf), (nk + 4, dim - 1, -math.inf)):
        v[j, 1, d] = value
    got = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k))
    torch.cuda.synchronize()
    marks = signs(v, cu_q, cu_k, lambda a, b: torch.ones(a, b), 4)
    close("lse", got[1], ref["lse"])
    check_out(got[0], ref["out"], *marks)
    if nq == 1:
        out, lse = m.rvq_cross_attention(q, k, v, None, ints(cu_k))
        check_out(out, ref["out"], *marks)


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("nq,nk", [(2, 40), (2, 3000), (90, 300), (150, 4000)])
@pytest.mark.parametrize("strong", [0, -1])
def test_infinities_of_weights_that_are_no_float32(typ, dim, nq, nk, strong):
    """One key scores so far above all others that their weights are below float32's smallest number; an infinite value
    of theirs stays infinite, in the strong key's wavefront and split and in others. All queries are one vector of
    numbers of 1 and -1, so that the scores of the strong key are 3 dim exactly and others are below 0."""
    m = rvq()
    announce("cross, far weights", typ=typ, dim=dim, nq=nq, nk=nk, strong=strong)
    _, k, v, _ = make(TYPES[typ], dim, 2, 1, [nq], [nk])
    way = torch.where(torch.rand(dim, generator=torch.Generator().manual_seed(4)) < 0.5, 1.0, -1.0).to(k.dtype).to(DEV)
    q = way.expand(nq, 2, dim).contiguous()
    k[:, 0] = -way
    k[strong, 0] = 3 * way
    scale = 1.0
    clean = v.clone()
    for j, d, value in ((1, 3, math.inf), (nk // 2, 4, -math.inf), (nk - 2, 9, math.inf), (nk // 3, 11, math.nan)):
        v[j, 0, d] = value
    out, lse = m.rvq_cross_attention(q, k, v, ints([0, nq]), ints([0, nk]), scale=scale)
    torch.cuda.synchronize()
    ref = cross_oracle.attention(q, k, clean, [0, nq], [0, nk], scale)
    close("lse", lse, ref["lse"])
    check_out(out, ref["out"], *signs(v, [0, nq], [0, nk], lambda a, b: torch.ones(a, b), 2))
    # the same keys in pages: the last query of a chunk sees all of them
    pages = -(-nk // 16)
    pools = [torch.full((pages, 1, 16, dim), math.nan, dtype=k.dtype, device=DEV) for _ in range(2)]
    for pool, x in zip(pools, (k, v)):
        pool.view(pages * 16, dim)[:nk] = x[:, 0]
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    new = min(nq, nk)
    got, got_lse = m.rvq_cache_chunk_attention(q[:new], *pools, table, ints([nk]), ints([0, new]), scale=scale)
    torch.cuda.synchronize()
    ref = attention_oracle.attention(q[:new], k, clean, [0, new], [0, nk], None, 0, scale)
    close("lse", got_lse, ref["lse"])
    check_out(got, ref["out"], *signs(v, [0, new], [0, nk], lambda a, b: attention_oracle.sees(a, b, None, 0), 2))


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 128), ("fp32", 64)])
@pytest.mark.parametrize("nq,nk,hq", [(1, 40, 2), (3, 700, 2), (2, 5000, 16), (90, 700, 2)])
def test_all_values_of_a_clip(typ, dim, nq, nk, hq):
    """All dims of every result of one clip are NaN, or of NaN and infinities; its lse and the other clip stay."""
    m = rvq()
    announce("cross, all values", typ=typ, dim=dim, nq=nq, nk=nk, heads=hq)
    q, k, v, _ = make(TYPES[typ], dim, hq, 1, [nq, nq], [nk, nk])
    cu_q, cu_k = offsets([nq, nq]), offsets([nk, nk])
    ref = cross_oracle.attention(q, k, v, cu_q, cu_k, 1 / math.sqrt(dim))
    out, lse = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k))
    close("lse", lse, ref["lse"])
    for value, first in ((math.nan, 0), (math.nan, nk - 1), (math.inf, 0)):
        x = v.clone()
        x[first:nk, :, 1:] = value
        if value == math.inf:
            x[nk // 2, :, 2:] = -math.inf
        got, got_lse = m.rvq_cross_attention(q, k, x, ints(cu_q), ints(cu_k))
        torch.cuda.synchronize()
        assert torch.equal(got_lse, lse) and torch.equal(got[nq:], out[nq:])
        check_out(got, ref["out"], *signs(x, cu_q, cu_k, lambda a, b: torch.ones(a, b), hq))
    k[5:nk] = math.nan
    got, got_lse = m.rvq_cross_attention(q, k, v, ints(cu_q), ints(cu_k))
    torch.cuda.synchronize()
    assert torch.isnan(got[:nq]).all() and torch.isnan(got_lse[:, :nq]).all()
    assert torch.equal(got[nq:], out[nq:]) and torch.equal(got_lse[:, nq:], lse[:, nq:])


# ---------------------------------------------------------------- scores at the ends of their range

@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 64), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("nq,nk", [(3, 200), (3, 3000), (100, 200), (100, 3000)])
def test_scores_of_minus_infinity(typ, dim, nq, nk):
    """Of all keys: output 0, lse -inf, also where the values are infinite. Of some: as if they were not there."""
    m = rvq()
    announce("scores of -inf", typ=typ, dim=dim, nq=nq, nk=nk)
    q, k, v, _ = make(TYPES[typ], dim, 2, 1, [nq], [nk])
    q[..., 2] = q[..., 2].abs() + 0.5
    k[..., 2] = -math.inf
    cu_q, cu_k = ints([0, nq]), ints([0, nk])
    for j in (None, 7):
        if j is not None:
            v[j] = math.inf
        out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
        torch.cuda.synchronize()
        assert (out == 0).all() and (lse == -math.inf).all()
    gone = nk // 2 + 3
    k[gone:, :, 2] = 1.0
    out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
    torch.cuda.synchronize()
    ref = cross_oracle.attention(q, k[gone:], v[gone:], [0, nq], [0, nk - gone], 1 / math.sqrt(dim))
    close("lse", lse, ref["lse"])
    close("out", out, ref["out"])


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("new,past", [(3, 200), (3, 3000), (100, 200), (100, 3000)])
def test_scores_far_below_zero_and_one_key_above_the_others(typ, dim, new, past):
    m, lens = rvq(), [past + new]
    announce("scores at the ends", typ=typ, dim=dim, new=new, past=past)
    k, v, table, _ = cache(typ, dim, 1, 16, lens)
    g = torch.Generator().manual_seed(9)
    way = torch.where(torch.rand(dim, generator=g) < 0.5, 1.0, -1.0)
    q = (way + 0.25 * torch.randn(new, 2, dim, generator=g)).to(TYPES[typ]).to(DEV)

    def check(keys):
        out, lse = m.rvq_cache_chunk_attention(q, keys, v, ints(table), ints(lens), ints([0, new]), scale=1.0)
        torch.cuda.synchronize()
        ref = want(q, keys, v, table, lens, [new], None, 0, 1.0)
        close("out", out, ref["out"])
        close("lse", lse, ref["lse"])

    check((k.cpu().float() * 0.1 - 3 * way).to(k.dtype).to(DEV))      # about -3 dim each
    for j in (0, 33, past // 2, past - 1):
        keys = (k.float() * 0.1).to(k.dtype)
        keys[table[0][j // 16], :, j % 16] = (2 * way).to(k.dtype).to(DEV)
        check(keys)


# ---------------------------------------------------------------- gradients

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [3, 90, 200])
def test_float16_gradients_of_other_clips_keep_their_bits(dim, nq):
    """Their powers of two come from the clip's own rows."""
    m = rvq()
    q, k, v, dout = make(torch.float16, dim, 2, 1, [nq, nq], [70, 70])
    cu_q, cu_k = ints([0, nq, 2 * nq]), ints([0, 70, 140])
    out, lse = m.rvq_cross_attention(q, k, v, cu_q, cu_k)
    grads = m.rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k)
    for value in (*VALUES, 60000.0):
        x = v.clone()
        x[69, 0, 3] = value
        got, _ = m.rvq_cross_attention(q, k, x, cu_q, cu_k)
        assert torch.equal(got[nq:], out[nq:])
        for a, b, n in zip(m.rvq_cross_attention_backward(dout, q, k, x, got, lse, cu_q, cu_k), grads, (nq, 70, 70)):
            assert torch.equal(a[n:], b[n:])
