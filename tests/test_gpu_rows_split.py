"""Chunk attention on the GPU where keys are split among workgroups and something is not finite that some queries of a
clip see and others do not, against float64 (attention_oracle): the workgroups that meet it go over their part again,
query by query, others do not, and every key counts once all the same."""

import math

import pytest
import torch

import attention_oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, offsets
from test_gpu_cache import cache
from test_gpu_chunk import gathered, want

pytestmark = [pytest.mark.gpu, needs_gpu]

VALUES = (math.inf, -math.inf, math.nan)


def odd(v, new, lens, window, sinks, heads):
    """Bool [T, heads, dim]: whether some value that is seen is not finite."""
    bad, cu_q, cu_k = ~torch.isfinite(v.cpu()), offsets(new), offsets(lens)
    res = torch.zeros(sum(new), heads, v.shape[2], dtype=torch.bool)
    for b, n in enumerate(new):
        mask = attention_oracle.sees(n, lens[b], window, sinks).double()
        for h in range(heads):
            rows = bad[cu_k[b]:cu_k[b + 1], h * v.shape[1] // heads]
            res[cu_q[b]:cu_q[b + 1], h] = mask @ rows.double() > 0
    return res


SPLIT = [  # past, new, heads, window, sinks
    ([1533] * 3, [4] * 3, (4, 2), None, 0),
    ([5000, 40], [4, 4], (4, 2), 2000, 4),
    ([5000, 4100], [4, 3], (8, 1), 2000, 4),
    ([1533, 1400, 300], [4, 5, 100], (4, 2), None, 0),
    ([1533, 5000], [13, 2], (2, 2), 1700, 0),
    ([2500], [150], (2, 1), None, 0),
]


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("fp16", 128), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("past,new,heads,window,sinks", SPLIT)
def test_splits_go_over_every_key_once(typ, dim, past, new, heads, window, sinks):
    """Values of the newest frames and of one that leaves the window within the turn. With scale 0 every key weighs the
    same and lse is the log of their number: one key more or less of 2000 moves it by 2^-11, and its bound is 2^-13."""
    m, lens = rvq(), [a + b for a, b in zip(past, new)]
    announce("chunk, split", typ=typ, dim=dim, past=past, new=new, heads=heads, window=window)
    hq, hk = heads
    k, v, table, _ = cache(typ, dim, hk, 16, lens)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(sum(new), hq, dim, generator=g).to(TYPES[typ]).to(DEV)
    cu = offsets(new)
    at = [(b, j) for b, n in enumerate(lens) for j in (n - 1, n - 3, *(() if window is None or n <= window else (n - 1 - window,)))]
    for scale in (0.0, None):
        ref = want(q, k, v, table, lens, new, window, sinks, 1 / math.sqrt(dim) if scale is None else scale)
        for value in VALUES:
            for head in {0, hk - 1}:
                bad = v.clone()
                for b, j in at:
                    bad[table[b][j // 16], head, j % 16, 5] = value
                out, lse = m.rvq_cache_chunk_attention(q, k, bad, ints(table), ints(lens), ints(cu), window=window,
                                                       sinks=sinks, scale=scale)
                torch.cuda.synchronize()
                close("lse", lse, ref["lse"])
                gone = odd(gathered(bad, table, lens), new, lens, window, sinks, hq)
                assert torch.equal(~torch.isfinite(out).cpu(), gone)
                close("out", out.cpu()[~gone], tuple(x[~gone] for x in ref["out"]))
    # keys: every query that does not see them is as it was
    rows = [i for b in range(len(new)) for i in range(cu[b], cu[b + 1])
            if not any(c == b and attention_oracle.sees(new[b], lens[b], window, sinks)[i - cu[b], j] for c, j in at)]
    for value in VALUES:
        bad = k.clone()
        for b, j in at:
            bad[table[b][j // 16], :, j % 16, 5] = value
        out, lse = m.rvq_cache_chunk_attention(q, bad, v, ints(table), ints(lens), ints(cu), window=window, sinks=sinks)
        torch.cuda.synchronize()
        close("lse", lse[:, rows], tuple(x[:, rows] for x in ref["lse"]))
        close("out", out[rows], tuple(x[rows] for x in ref["out"]))
