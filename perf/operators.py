"""Workloads of the streaming-attention operators: windowed attention with its gradient, the attention of
one new frame over a paged key-value cache, and the upkeep of the cache's pages.

Sequences of code frames are packed: the frames of all clips stand one after another, ``cu[b]..cu[b+1]`` are
clip b's. A frame at position p sees the frames j <= p with p - j < window, and the first ``sinks`` frames.
Pools of cache pages are [layers, pages, kv heads, page size, head dim].

``run`` computes each operator in elementary torch operations in 32 bits, or through the package's entry
points where ``own`` is true.
"""

import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a few short utterances arriving together (1 s at 25 Hz and less), a small 64-wide codec transformer
        dict(name="prefill_turns", kind="prefill", type="bf16", clips=3, longest=25, ragged=True, past=0,
             q_heads=8, kv_heads=8, dim=64, window=None, sinks=0),
        # a chunk of a long recording whose earlier frames are already known, grouped heads, bounded window
        dict(name="prefill_long", kind="prefill", type="bf16", clips=1, longest=16384, ragged=False, past=1500,
             q_heads=16, kv_heads=4, dim=128, window=4096, sinks=4),
        # training in the codec's own precision on ragged clips of up to 30 s at 25 Hz
        dict(name="train_fp32", kind="train", type="fp32", clips=6, longest=750, ragged=True, past=0,
             q_heads=8, kv_heads=8, dim=64, window=200, sinks=0),
        # training on whole clips of 2000 frames, every earlier frame visible
        dict(name="train_clips", kind="train", type="fp16", clips=8, longest=2000, ragged=False, past=0,
             q_heads=16, kv_heads=8, dim=64, window=None, sinks=0),
        # training on one long recording with a short window and sinks
        dict(name="train_window", kind="train", type="bf16", clips=2, longest=8192, ragged=True, past=0,
             q_heads=16, kv_heads=4, dim=128, window=750, sinks=4),
        # one listener: the next frame after 60 s at 25 Hz; latency counts
        dict(name="decode_one", kind="decode", type="bf16", clips=1, longest=1500, ragged=False,
             q_heads=16, kv_heads=8, dim=128, window=None, sinks=0, page=16),
        # many streams of uneven age, bounded window with sinks; what left the window has been given back
        dict(name="decode_window", kind="decode", type="fp16", clips=96, longest=9000, ragged=True,
             q_heads=16, kv_heads=16, dim=64, window=1500, sinks=4, page=32),
        # hour-long recordings (45000 frames at 12.5 Hz), whole history
        dict(name="decode_hour", kind="decode", type="bf16", clips=12, longest=45000, ragged=True,
             q_heads=32, kv_heads=8, dim=128, window=None, sinks=0, page=64),
        # clips join or continue: pages for their new frames, and the frames' keys and values written there
        dict(name="admit_clips", kind="admit", type="bf16", clips=64, longest=1500, ragged=True, add=750,
             layers=1, kv_heads=8, dim=128, page=16),
        # a beam step: every hypothesis goes on from a chosen one; full pages are shared, partial ones copied
        dict(name="fork_beams", kind="fork", type="bf16", clips=8, longest=250, ragged=True,
             layers=4, kv_heads=8, dim=64, page=16),
        # the same for many streams, a deep stack and large pages
        dict(name="fork_streams", kind="fork", type="fp16", clips=256, longest=2000, ragged=True,
             layers=8, kv_heads=8, dim=64, page=64),
        # streams end and others leave frames behind their window; the pool is compacted
        dict(name="retire_streams", kind="retire", type="bf16", clips=128, longest=9000, ragged=True,
             layers=2, kv_heads=8, dim=64, page=32, window=1500, sinks=4),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["prefill", "train", "decode", "admit", "fork", "retire"])
    kv_heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    case = dict(kind=kind, type=rng.choice(["bf16", "fp16", "fp32"]), kv_heads=kv_heads, dim=rng.choice([64, 128]),
                ragged=rng.random() < 0.7)
    window = rng.choice([None, _log(rng, 1, 4096)])
    sinks = 0 if window is None else rng.choice([0, 1, 4, _log(rng, 5, 100)])
    if kind in ("prefill", "train"):
        clips = _log(rng, 1, 24)
        # the plain form holds every pair of frames of a head
        most = int(math.sqrt((3e8 if kind == "train" else 1e9) / (clips * kv_heads * group)))
        case.update(clips=clips, longest=_log(rng, 3, min(4096, most)), past=rng.choice([0, _log(rng, 1, 300)]) if kind == "prefill" else 0,
                    q_heads=kv_heads * group, window=window, sinks=sinks)
    elif kind == "decode":
        longest = _log(rng, 1, 30000)
        most = max(1, int(2e8 / (longest * kv_heads * case["dim"])))
        case.update(clips=_log(rng, 1, min(128, most)), longest=longest, q_heads=kv_heads * group,
                    window=window, sinks=sinks, page=rng.choice([1, 8, 16, 24, 32, 64, 100]))
    else:
        longest = _log(rng, 5, 4000)
        page = rng.choice([8, 16, 24, 32, 64])
        case["layers"] = 1 if kind == "admit" else rng.choice([1, 2, 3, 5])
        most = max(2, int(1.5e8 / (longest * kv_heads * case["dim"] * case["layers"])))
        case.update(clips=_log(rng, 2, min(200, most)), longest=longest, page=page)
        if kind == "admit":
            case["add"] = rng.choice([1, _log(rng, 2, 600)])
        if kind == "retire":
            case.update(window=_log(rng, 1, 2000), sinks=rng.choice([0, 1, 4, 40]))
    return case


# ---------------------------------------------------------------- shapes that a case stands for

def _shape_rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, rng):
    """A length for each clip, the longest among them."""
    n, top = case["clips"], case["longest"]
    if not case["ragged"]:
        return [top] * n
    got = [rng.randint(max(1, top // 8), top) for _ in range(n)]
    got[rng.randrange(n)] = top
    return got


def _pairs(q_len, k_len, window, sinks):
    """How many (query, key) pairs see each other."""
    p = np.arange(k_len - q_len, k_len, dtype=np.int64)
    w = p + 1 if window is None else np.minimum(p + 1, window)
    s = np.minimum(sinks, p + 1 - w)
    return int((w + s).sum())


def _table(case, lengths, rng, spare, window=None, sinks=0):
    """Page table, reference counts and the pool's size for clips of these lengths, pages in random places."""
    page = case["page"]
    wide = max(1, -(-(max(lengths) + case.get("add", 0)) // page) + 1)
    table = np.full((len(lengths), wide), -1, dtype=np.int32)
    for b, n in enumerate(lengths):
        for e in range(-(-n // page)):
            # a page behind the window of every later frame has been given back
            if window is None or e * page < sinks or (e + 1) * page > n - window:
                table[b, e] = 1
    held = int((table > 0).sum())
    pages = held + spare + 1
    order = list(range(pages))
    rng.shuffle(order)
    table[table > 0] = order[:held]
    refs = np.zeros(pages, dtype=np.int32)
    refs[order[:held]] = 1
    return table, refs, pages


def _added(case, lengths, rng):
    if case["add"] == 1:
        return [1] * len(lengths)
    return [rng.randint(1, case["add"]) for _ in lengths]


def _meta(case):
    """Host-side description of a page case: table, refs, pages, lengths and what is asked for."""
    rng = _shape_rng(case)
    lengths = _lengths(case, rng)
    page = case["page"]
    m = dict(lengths=lengths)
    if case["kind"] == "decode":
        m["table"], m["refs"], m["pages"] = _table(case, lengths, rng, 3, case["window"], case["sinks"])
    elif case["kind"] == "admit":
        m["add"] = _added(case, lengths, rng)
        need = sum(-(-(n + a) // page) - -(-n // page) for n, a in zip(lengths, m["add"]))
        m["table"], m["refs"], m["pages"] = _table(case, lengths, rng, need + 5)
    elif case["kind"] == "fork":
        m["table"], m["refs"], m["pages"] = _table(case, lengths, rng, case["clips"] + 7)
        m["parents"] = [rng.randrange(case["clips"]) for _ in lengths]
        m["children"] = list(range(case["clips"]))
    else:
        m["table"], m["refs"], m["pages"] = _table(case, lengths, rng, 9)
        m["drop"] = [int(rng.random() < 0.3) for _ in lengths]
    return m


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kind, typ, dim = case["kind"], TYPES[case["type"]], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(typ)

    def noise(*shape):
        # large pools: uniform values are quicker to make
        return torch.empty(*shape, device=dev, dtype=typ).uniform_(-2, 2, generator=gen)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    state = dict(case, scale=1 / math.sqrt(dim))
    if kind in ("prefill", "train"):
        q_lens = _lengths(case, _shape_rng(case))
        k_lens = [n + case["past"] for n in q_lens]
        state.update(q_lens=q_lens, k_lens=k_lens, cu_q=ints([0] + list(np.cumsum(q_lens))),
                     cu_k=ints([0] + list(np.cumsum(k_lens))))
        hq, hk = case["q_heads"], case["kv_heads"]
        if case["past"]:
            state["q"] = normal(sum(q_lens), hq, dim)
            kv = normal(sum(k_lens), 2 * hk, dim)
            state["k"], state["v"] = kv[:, :hk], kv[:, hk:]
        else:
            # one projection makes all three
            qkv = normal(sum(q_lens), hq + 2 * hk, dim)
            state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        if kind == "train":
            state["dout"] = normal(sum(q_lens), hq, dim)
        return state
    m = _meta(case)
    state.update(table=ints(m["table"]), refs=ints(m["refs"]), lens=ints(m["lengths"]), longest=max(m["lengths"]))
    layers = case.get("layers", 1)
    shape = (layers, m["pages"], case["kv_heads"], case["page"], dim)
    state["k_pool"], state["v_pool"] = noise(*shape), noise(*shape)
    if kind == "decode":
        state["q"] = normal(case["clips"], case["q_heads"], dim)
        state["k_pool"], state["v_pool"] = state["k_pool"][0], state["v_pool"][0]
    elif kind == "admit":
        state["new_lens"] = ints([n + a for n, a in zip(m["lengths"], m["add"])])
        state["cu_new"] = ints([0] + list(np.cumsum(m["add"])))
        kv = normal(sum(m["add"]), 2 * case["kv_heads"], dim)
        state["k"], state["v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]
    elif kind == "fork":
        state["parents"], state["children"] = ints(m["parents"]), ints(m["children"])
    else:
        state["drop"] = ints(m["drop"])
    return state


def work(case):
    size, dim = BYTES[case["type"]], case["dim"]
    kind = case["kind"]
    if kind in ("prefill", "train"):
        q_lens = _lengths(case, _shape_rng(case))
        pairs = sum(_pairs(n, n + case["past"], case["window"], case["sinks"]) for n in q_lens) * case["q_heads"]
        nq = sum(q_lens) * case["q_heads"] * dim
        nk = sum(n + case["past"] for n in q_lens) * case["kv_heads"] * dim
        if kind == "prefill":
            return {"bytes": size * (2 * nq + 2 * nk) + 4 * nq // dim, "flops": 4 * pairs * dim}
        # forward (scores, values) and backward (scores again, and the four gradient products)
        return {"bytes": size * (4 * nq + 4 * nk), "flops": 14 * pairs * dim}
    m = _meta(case)
    meta = 4 * (m["table"].size + len(m["lengths"]))
    row = 2 * case["kv_heads"] * dim * size * case.get("layers", 1)
    if kind == "decode":
        seen = sum(n if case["window"] is None else min(n, case["window"] + min(case["sinks"], max(0, n - case["window"])))
                   for n in m["lengths"])
        return {"bytes": seen * row + 2 * case["clips"] * case["q_heads"] * dim * size + meta,
                "flops": 4 * seen * case["q_heads"] * dim}
    meta = 2 * meta + 8 * m["pages"]
    if kind == "admit":
        return {"bytes": 2 * sum(m["add"]) * row + meta, "flops": 0}
    if kind == "fork":
        part = sum(m["lengths"][p] % case["page"] for p in m["parents"])
        return {"bytes": 2 * part * row + meta, "flops": 0}
    _, _, refs = _free_host(m, case)
    live = int((refs > 0).sum())
    moved = int((refs[live:] > 0).sum())
    return {"bytes": 2 * moved * case["page"] * row + meta, "flops": 0}


def _free_host(m, case):
    """Table, lengths and reference counts after the ended streams and the frames behind the window left."""
    table, refs, lens = m["table"].copy(), m["refs"].copy(), np.array(m["lengths"])
    page, e = case["page"], np.arange(m["table"].shape[1])
    gone = (e * page >= case["sinks"])[None] & ((e + 1) * page <= lens[:, None] - case["window"] + 1)
    gone |= np.array(m["drop"], dtype=bool)[:, None]
    gone &= table >= 0
    np.subtract.at(refs, table[gone], 1)
    table[gone] = -1
    lens[np.array(m["drop"], dtype=bool)] = 0
    return table, lens, refs


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _plain_prefill, "train": _plain_train, "decode": _plain_decode, "admit": _plain_admit,
            "fork": _plain_fork, "retire": _plain_retire}[s["kind"]](s)


def _run_own(s):
    import residual_vector_quantization_amd as rvq
    kind = s["kind"]
    if kind in ("prefill", "train"):
        out, lse = rvq.rvq_window_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], window=s["window"],
                                            sinks=s["sinks"], scale=s["scale"])
        if kind == "prefill":
            return out, lse
        grads = rvq.rvq_window_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"],
                                                  window=s["window"], sinks=s["sinks"], scale=s["scale"])
        return (out, *grads)
    if kind == "decode":
        return rvq.rvq_cache_attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], window=s["window"],
                                       sinks=s["sinks"], scale=s["scale"])
    if kind == "admit":
        table, refs, missing = rvq.rvq_cache_reserve(s["table"], s["lens"], s["new_lens"], s["refs"], s["page"])
        rvq.rvq_cache_append(s["k"], s["v"], s["k_pool"][0], s["v_pool"][0], table, s["lens"], s["cu_new"])
        return table, refs, missing, s["k_pool"], s["v_pool"]
    if kind == "fork":
        table, lens, refs, missing = rvq.rvq_cache_fork(s["table"], s["lens"], s["refs"], s["parents"], s["children"],
                                                        s["k_pool"], s["v_pool"])
        return table, lens, refs, missing, s["k_pool"], s["v_pool"]
    table, lens, refs = rvq.rvq_cache_free(s["table"], s["lens"], s["refs"], s["page"], drop=s["drop"],
                                           window=s["window"], sinks=s["sinks"])
    table, refs, live = rvq.rvq_cache_compact(table, refs, s["k_pool"], s["v_pool"])
    return table, lens, refs, live, s["k_pool"], s["v_pool"]


# ---------------------------------------------------------------- plain forms

def _padded(x, cu, longest):
    """[T, H, D] packed -> [B, H, longest, D] in 32 bits, zeros behind each clip's end."""
    at = torch.arange(longest, device=x.device)
    n = (cu[1:] - cu[:-1]).long()
    index = (cu[:-1].long()[:, None] + at).clamp(max=x.shape[0] - 1)
    y = x[index].float() * (at < n[:, None])[..., None, None]
    return y.transpose(1, 2).contiguous()


def _packed(y, cu, total):
    """[B, H, L, D] -> [T, H, D]: each clip's own rows."""
    t = torch.arange(total, device=y.device)
    clip = torch.searchsorted(cu[1:].contiguous(), t.int(), right=True)
    return y[clip, :, t - cu[clip].long()]


def _plain_scores(s):
    lq, lk, group = max(s["q_lens"]), max(s["k_lens"]), s["q_heads"] // s["kv_heads"]
    q, k, v = _padded(s["q"], s["cu_q"], lq), _padded(s["k"], s["cu_k"], lk), _padded(s["v"], s["cu_k"], lk)
    b, d = q.shape[0], q.shape[3]
    q = q.view(b, s["kv_heads"], group * lq, d)
    nq, nk = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), (s["cu_k"][1:] - s["cu_k"][:-1]).long()
    i, j = torch.arange(lq, device=q.device), torch.arange(lk, device=q.device)
    p = i + (nk - nq)[:, None]                                          # a query's position among its clip's keys
    sees = (j <= p[..., None]) & (j < nk[:, None, None])
    if s["window"] is not None:
        sees &= (p[..., None] - j < s["window"]) | (j < s["sinks"])
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).view(b, s["kv_heads"], group, lq, lk) * s["scale"]
    x = x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    x = x / torch.where(total == 0, torch.ones_like(total), total)
    return q, k, v, x.view(b, s["kv_heads"], group * lq, lk), lse.view(b, s["q_heads"], lq)


def _plain_prefill(s):
    q, k, v, p, lse = _plain_scores(s)
    out = torch.matmul(p, v).view(q.shape[0], s["q_heads"], -1, q.shape[3])
    out = _packed(out, s["cu_q"], s["q"].shape[0]).to(s["q"].dtype)
    return out, _packed(lse[..., None], s["cu_q"], s["q"].shape[0])[..., 0].t().contiguous()


def _plain_train(s):
    q, k, v, p, _ = _plain_scores(s)
    b, heads, rows, d = q.shape
    typ, nq, nk = s["q"].dtype, s["q"].shape[0], s["k"].shape[0]
    out = torch.matmul(p, v)
    do = _padded(s["dout"], s["cu_q"], max(s["q_lens"])).view(b, heads, rows, d)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = ds.sub_((do * out).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q) * s["scale"]
    out, dq = out.view(b, s["q_heads"], -1, d), dq.view(b, s["q_heads"], -1, d)
    return (_packed(out, s["cu_q"], nq).to(typ), _packed(dq, s["cu_q"], nq).to(typ), _packed(dk, s["cu_k"], nk).to(typ),
            _packed(dv, s["cu_k"], nk).to(typ))


def _plain_decode(s):
    q, table, lens, page = s["q"], s["table"], s["lens"].long(), s["page"]
    b, hq, d = q.shape
    hk = s["kv_heads"]
    if s["window"] is None or s["window"] + s["sinks"] >= s["longest"]:
        at = torch.arange(s["longest"], device=q.device).expand(b, -1)
        sees = at < lens[:, None]
        if s["window"] is not None:
            sees = sees & ((at >= lens[:, None] - s["window"]) | (at < s["sinks"]))
    else:
        # the first frames, then the window's
        first = torch.arange(s["sinks"], device=q.device).expand(b, -1)
        last = lens[:, None] - s["window"] + torch.arange(s["window"], device=q.device)
        at = torch.cat([first, last], 1)
        sees = torch.cat([first < lens[:, None], last >= s["sinks"]], 1)
    at = at.clamp(0, table.shape[1] * page - 1)
    where, slot = table.long().gather(1, at // page).clamp(min=0), at % page
    k = s["k_pool"][where, :, slot].float().permute(0, 2, 3, 1).contiguous()     # [B, Hk, D, N]
    v = s["v_pool"][where, :, slot].float().transpose(1, 2).contiguous()         # [B, Hk, N, D]
    x = torch.matmul(q.float().view(b, hk, hq // hk, d), k) * s["scale"]
    x = x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / torch.where(total == 0, torch.ones_like(total), total)
    return out.view(b, hq, d).to(q.dtype)


def _free_pages(refs):
    """Page numbers, the free ones first and in order, and how many are free."""
    return torch.argsort((refs != 0).int(), stable=True), (refs == 0).sum()


def _plain_admit(s):
    table, refs, page = s["table"], s["refs"], s["page"]
    lens, new = s["lens"].long(), s["new_lens"].long()
    e = torch.arange(table.shape[1], device=table.device)
    need = (e >= ((lens + page - 1) // page)[:, None]) & (e < ((new + page - 1) // page)[:, None])
    rank = torch.cumsum(need.flatten().long(), 0) - 1
    order, free = _free_pages(refs)
    given = need & (rank < free).view_as(need)
    page_of = order[rank.clamp(0, refs.shape[0] - 1)].view_as(need)
    table = torch.where(given, page_of.int(), table)
    refs = refs.clone().index_add_(0, page_of.flatten(), given.flatten().int())
    missing = (need.sum() - free).clamp(min=0).int().view(1)
    t = torch.arange(s["k"].shape[0], device=table.device)
    clip = torch.searchsorted(s["cu_new"][1:].contiguous(), t.int(), right=True)
    at = lens[clip] + t - s["cu_new"][clip].long()
    where, slot = table[clip, at // page].long(), at % page
    s["k_pool"][0][where, :, slot] = s["k"]
    s["v_pool"][0][where, :, slot] = s["v"]
    return table, refs, missing, s["k_pool"], s["v_pool"]


def _plain_fork(s):
    old, lens, page = s["table"], s["lens"], s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    rows, n = old[parents], lens[parents].long()
    e = torch.arange(old.shape[1], device=old.device)
    part = (e == (n // page)[:, None]) & ((n % page) > 0)[:, None]          # the page that goes on being written
    order, free = _free_pages(s["refs"])
    rank = torch.cumsum(part.any(1).long(), 0) - 1
    got = part.any(1) & (rank < free)
    fresh = order[rank.clamp(0, order.shape[0] - 1)]
    refs = s["refs"].clone()
    left = old[children]
    refs.index_add_(0, left.clamp(min=0).long().flatten(), -(left >= 0).int().flatten())
    shared = (rows >= 0) & ~part
    refs.index_add_(0, rows.clamp(min=0).long().flatten(), shared.int().flatten())
    refs.index_add_(0, fresh, got.int())
    source = rows.gather(1, (n // page).clamp(max=old.shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
    target = torch.where(got, fresh, source)                                # a clip without a part copies onto itself
    s["k_pool"][:, target] = s["k_pool"][:, source]
    s["v_pool"][:, target] = s["v_pool"][:, source]
    rows = torch.where(part, torch.where(got, fresh, torch.full_like(fresh, -1)).int()[:, None], rows)
    table, new_lens = old.clone(), lens.clone()
    table[children], new_lens[children] = rows, lens[parents]
    missing = (part.any(1).sum() - free).clamp(min=0).int().view(1)
    return table, new_lens, refs, missing, s["k_pool"], s["v_pool"]


def _plain_retire(s):
    table, refs, page, lens = s["table"], s["refs"].clone(), s["page"], s["lens"]
    e = torch.arange(table.shape[1], device=table.device)
    ended = s["drop"] != 0
    gone = (e * page >= s["sinks"]) & ((e + 1) * page <= lens[:, None] - s["window"] + 1)
    gone = (gone | ended[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -gone.int().flatten())
    table, lens = torch.where(gone, -1, table), torch.where(ended, 0, lens)
    alive, at = refs > 0, torch.arange(refs.shape[0], device=refs.device)
    live = alive.sum()
    moves, holes = alive & (at >= live), ~alive & (at < live)
    order = torch.argsort((~holes).int(), stable=True)
    new = torch.where(moves, order[(torch.cumsum(moves.long(), 0) - 1).clamp(min=0)], at)
    source = moves.nonzero()[:, 0]
    s["k_pool"][:, new[source]] = s["k_pool"][:, source]
    s["v_pool"][:, new[source]] = s["v_pool"][:, source]
    table = torch.where(table >= 0, new[table.clamp(min=0).long()].int(), table)
    refs = torch.zeros_like(refs).index_add_(0, new, refs)
    return table, lens, refs, live.int().view(1), s["k_pool"], s["v_pool"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _softmax64(x):
    top = x.max(-1, keepdim=True).values
    x = (x - top).exp()
    return x / x.sum(-1, keepdim=True), top[..., 0] + x.sum(-1).log()


def exact(case, seed):
    kind = case["kind"]
    if kind in ("prefill", "train"):
        return _exact_attention(prepare(case, seed), kind == "train")
    if kind == "decode":
        return _exact_decode(prepare(case, seed))
    return None         # pages are copied, not computed


def _exact_attention(s, train):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    dev, group = q.device, s["q_heads"] // s["kv_heads"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[1::-1], -math.inf, dtype=torch.float64, device=dev)
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    q0 = k0 = 0
    step = 2048
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        for h in range(s["q_heads"]):
            kh, vh = k[k0:k0 + nk, h // group], v[k0:k0 + nk, h // group]
            for i0 in range(0, nq, step):
                i1 = min(nq, i0 + step)
                p = torch.arange(i0 + nk - nq, i1 + nk - nq, device=dev)
                last, first = nk - nq + i1, 0
                if s["window"] is not None and nk - nq + i0 - s["window"] + 1 > s["sinks"]:
                    first = nk - nq + i0 - s["window"] + 1
                j = torch.cat([torch.arange(min(s["sinks"], first), device=dev), torch.arange(first, last, device=dev)])
                hidden = j > p[:, None]
                if s["window"] is not None:
                    hidden |= (j <= p[:, None] - s["window"]) & (j >= s["sinks"])
                rows = slice(q0 + i0, q0 + i1)
                qi, kj, vj = q[rows, h], kh[j], vh[j]
                x = (qi @ kj.t() * s["scale"]).masked_fill(hidden, -math.inf)
                w, l = _softmax64(x)
                o = w @ vj
                out[rows, h], lse[h, rows] = o, l
                if train:
                    g = s["dout"][rows, h].double()
                    dw = g @ vj.t()
                    dx = w * (dw - (w * dw).sum(-1, keepdim=True)) * s["scale"]
                    dq[rows, h] = dx @ kj
                    dk[:, h // group].index_add_(0, j + k0, dx.t() @ qi)
                    dv[:, h // group].index_add_(0, j + k0, w.t() @ g)
        q0, k0 = q0 + nq, k0 + nk
    return (out, dq, dk, dv) if train else (out, lse)


def _exact_decode(s):
    q, group = s["q"].double(), s["q_heads"] // s["kv_heads"]
    out = torch.zeros_like(q)
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device=q.device)
        if s["window"] is not None:
            j = j[(j > n - 1 - s["window"]) | (j < s["sinks"])]
        pages = s["table"][b].long()[j // s["page"]]
        k, v = (s[p][pages, :, j % s["page"]].double() for p in ("k_pool", "v_pool"))
        for h in range(s["q_heads"]):
            w, _ = _softmax64(k[:, h // group] @ q[b, h] * s["scale"])
            out[b, h] = w @ v[:, h // group]
    return out
