"""Workloads of the operators around streaming attention: rotary positions with their gradient, alone and on the way
into the paged cache; attention of a chunk of new frames over the cache; cross attention to an encoder's states.

Sequences of code frames are packed: the frames of all clips stand one after another, ``cu[b]..cu[b+1]`` are
clip b's. Pools of cache pages are [pages, kv heads, page size, head dim].

* Rotary: of a head's first ``rot`` values pair i turns by position * frequencies[i]; pairs are (i, i + rot / 2), or
  neighbours where ``interleaved``; turned values are scaled by ``amplitude``.
* Chunk: clip b's cache holds ``lens[b]`` frames, the last ``cu[b+1] - cu[b]`` of them are the queries. A frame at
  position p sees the frames j <= p with p - j < window, and the first ``sinks`` frames.
* Cross: every frame of clip b sees all states ``cu_k[b]..cu_k[b+1]``; without any its result is 0.

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
        # training in the codec's own precision on ragged clips of up to 30 s at 25 Hz: half of each head turns,
        # forward and gradient
        dict(name="rotate_train", kind="rotate_train", type="fp32", clips=6, longest=750, ragged=True, past=0,
             q_heads=8, kv_heads=8, dim=64, rot=32, interleaved=True, factor=1.0),
        # four long recordings at once, positions stretched beyond the length that a model was trained on
        dict(name="rotate_long", kind="rotate", type="bf16", clips=4, longest=16384, ragged=False, past=45000,
             q_heads=16, kv_heads=4, dim=128, rot=128, interleaved=False, factor=8.0),
        # the next frame of many streams of uneven age, on its way into the cache; latency counts
        dict(name="append_step", kind="append", type="fp16", clips=96, cached=9000, ragged=True, fresh=1, mixed=False,
             q_heads=16, kv_heads=16, dim=64, page=32, rot=64, interleaved=False, factor=1.0),
        # clips join or continue with up to 750 frames each
        dict(name="append_prompt", kind="append", type="bf16", clips=64, cached=1500, ragged=True, fresh=750,
             mixed=False, q_heads=32, kv_heads=8, dim=128, page=16, rot=128, interleaved=False, factor=4.0),
        # a few drafted frames of some listeners are looked at together
        dict(name="chunk_draft", kind="chunk", type="bf16", clips=8, cached=1500, ragged=True, fresh=4, mixed=False,
             q_heads=16, kv_heads=8, dim=128, window=None, sinks=0, page=16),
        # two seconds at a time in the codec's own precision
        dict(name="chunk_fp32", kind="chunk", type="fp32", clips=6, cached=750, ragged=True, fresh=50, mixed=False,
             q_heads=8, kv_heads=8, dim=64, window=200, sinks=0, page=8),
        # streams that go on by one frame beside some that bring up to 500; bounded window with sinks, what left
        # the window has been given back
        dict(name="chunk_beside", kind="chunk", type="fp16", clips=32, cached=9000, ragged=True, fresh=500, mixed=True,
             q_heads=16, kv_heads=16, dim=64, window=1500, sinks=4, page=32),
        # the next piece of an hour-long recording (45000 frames at 12.5 Hz), whole history
        dict(name="chunk_long", kind="chunk", type="bf16", clips=1, cached=45000, ragged=False, fresh=2048, mixed=False,
             q_heads=32, kv_heads=8, dim=128, window=None, sinks=0, page=64),
        # the next frame of many clips looks at what it is conditioned on, some clips on nothing
        dict(name="cross_step", kind="cross", type="bf16", clips=64, longest=1, ragged=True, states=1500, empty=True,
             q_heads=16, kv_heads=16, dim=64),
        # whole clips over another modality's states, grouped heads
        dict(name="cross_clips", kind="cross", type="fp16", clips=12, longest=2000, ragged=True, states=750, empty=False,
             q_heads=16, kv_heads=4, dim=128),
        # training in the codec's own precision on short clips
        dict(name="cross_train_fp32", kind="cross_train", type="fp32", clips=6, longest=250, ragged=True, states=300,
             empty=True, q_heads=8, kv_heads=8, dim=64),
        # training on whole clips of up to 2000 frames
        dict(name="cross_train", kind="cross_train", type="bf16", clips=8, longest=2000, ragged=True, states=1500,
             empty=False, q_heads=16, kv_heads=8, dim=128),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate_train", "append", "chunk", "chunk", "cross", "cross_train"])
    kv_heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    dim, heads = rng.choice([64, 128]), kv_heads * group
    case = dict(kind=kind, type=rng.choice(["bf16", "fp16", "fp32"]), q_heads=heads, kv_heads=kv_heads, dim=dim,
                ragged=rng.random() < 0.7)
    clips = _log(rng, 1, 64)
    if kind in ("rotate", "rotate_train", "append"):
        case.update(rot=rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]),
                    interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 1.0, 4.0, 32.0]), clips=clips)
        most = max(2, int(4e7 / (clips * (heads + 2 * kv_heads) * dim)))
    if kind in ("rotate", "rotate_train"):
        case.update(longest=_log(rng, 1, min(16384, most)), past=rng.choice([0, _log(rng, 1, 500000)]))
    elif kind == "append":
        fresh = rng.choice([1, _log(rng, 2, min(2000, most))])
        case.update(fresh=fresh, mixed=rng.random() < 0.3, page=rng.choice([1, 8, 16, 24, 32, 64, 100]),
                    cached=_log(rng, 1, max(2, min(20000, most))))
    elif kind == "chunk":
        window = rng.choice([None, _log(rng, 1, 4096)])
        cached = _log(rng, 1, 20000)
        # the plain form holds every pair of frames of a head, and every clip's keys
        most = max(1, int(8e8 / (clips * heads * cached)))
        clips = max(1, min(clips, int(1.5e8 / (cached * kv_heads * dim))))
        case.update(clips=clips, cached=cached, fresh=min(1500, _log(rng, 1, min(1500, most))), mixed=rng.random() < 0.4,
                    window=window, sinks=0 if window is None else rng.choice([0, 1, 4, _log(rng, 5, 100)]),
                    page=rng.choice([1, 8, 16, 24, 32, 64, 100]))
    else:
        # a gradient through a softmax over one state is nothing but rounding
        states = _log(rng, 8 if kind == "cross_train" else 1, 3000)
        most = max(1, int((2e8 if kind == "cross_train" else 6e8) / (clips * heads * states)))
        case.update(clips=clips, states=states, longest=rng.choice([1, _log(rng, 1, min(4096, most))]),
                    empty=rng.random() < 0.4)
    return case


# ---------------------------------------------------------------- shapes that a case stands for

def _shape_rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(n, top, ragged, rng):
    """n lengths, the longest among them."""
    if not ragged:
        return [top] * n
    got = [rng.randint(max(1, top // 8), top) for _ in range(n)]
    got[rng.randrange(n)] = top
    return got


def _meta(case):
    """Host-side description of a case: lengths, and the page table where there is one."""
    rng, n = _shape_rng(case), case["clips"]
    if case["kind"] in ("rotate", "rotate_train"):
        return dict(fresh=_lengths(n, case["longest"], case["ragged"], rng), past=[rng.randint(0, case["past"]) for _ in range(n)])
    if case["kind"] in ("cross", "cross_train"):
        states = _lengths(n, case["states"], case["ragged"], rng)
        if case["empty"]:
            states = [0 if b % 5 == 4 else s for b, s in enumerate(states)]
        return dict(fresh=_lengths(n, case["longest"], case["ragged"], rng), states=states)
    past, fresh = _lengths(n, case["cached"], case["ragged"], rng), _lengths(n, case["fresh"], case["ragged"], rng)
    if case["mixed"]:
        keep = max(range(n), key=fresh.__getitem__)
        fresh = [f if b == keep or rng.random() < 0.25 else 1 for b, f in enumerate(fresh)]
    lens = [p + f for p, f in zip(past, fresh)]
    page, window, sinks = case["page"], case.get("window"), case.get("sinks", 0)
    table = np.full((n, -(-max(lens) // page) + 1), -1, dtype=np.int32)
    for b in range(n):
        for e in range(-(-lens[b] // page)):
            # a page behind the window of the first new frame, and so of every later one, has been given back
            if window is None or e * page < sinks or (e + 1) * page > past[b] + 1 - window:
                table[b, e] = 1
    held = int((table > 0).sum())
    order = list(range(held + 4))
    rng.shuffle(order)
    table[table > 0] = order[:held]
    return dict(past=past, fresh=fresh, lens=lens, table=table, pages=held + 4)


def _frequencies(case):
    """base^(-2 i / rot); with a factor, those of waves that turn rarely within the length known so far are slower."""
    f = 10000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
    if case["factor"] == 1.0:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    return f * (keep + (1 - keep) / case["factor"]), 0.1 * math.log(case["factor"]) + 1


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kind, typ, dim, hq, hk = case["kind"], TYPES[case["type"]], case["dim"], case["q_heads"], case["kv_heads"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(typ)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    m = _meta(case)
    total = sum(m["fresh"])
    state = dict(case, scale=1 / math.sqrt(dim), fresh_lens=m["fresh"], cu=ints([0] + list(np.cumsum(m["fresh"]))))
    if "rot" in case:
        f, state["amplitude"] = _frequencies(case)
        state["frequencies"] = torch.from_numpy(f).to(dev)
    if kind in ("cross", "cross_train"):
        state.update(states_lens=m["states"], cu_k=ints([0] + list(np.cumsum(m["states"]))))
        # one projection of the states makes keys and values
        kv = normal(sum(m["states"]), 2 * hk, dim)
        state.update(q=normal(total, hq, dim), k=kv[:, :hk], v=kv[:, hk:])
        if kind == "cross_train":
            state["dout"] = normal(total, hq, dim)
        return state
    if kind == "chunk":
        state["q"] = normal(total, hq, dim)
    else:
        # one projection makes all three
        qkv = normal(total, hq + 2 * hk, dim)
        state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    state["past"] = ints(m["past"])
    if kind == "rotate_train":
        state["dq"], state["dk"] = normal(total, hq, dim), normal(total, hk, dim)
    if kind in ("append", "chunk"):
        state.update(lens=ints(m["lens"]), lens_list=m["lens"], table=ints(m["table"]))
        state["k_pool"], state["v_pool"] = (torch.empty(m["pages"], hk, case["page"], dim, device=dev, dtype=typ)
                                            .normal_(generator=gen) for _ in range(2))
    return state


def work(case):
    m, size, dim, hq, hk = _meta(case), BYTES[case["type"]], case["dim"], case["q_heads"], case["kv_heads"]
    kind, total = case["kind"], sum(m["fresh"])
    nq = total * hq * dim
    if kind in ("rotate", "rotate_train"):
        n = total * (hq + hk) * dim * (2 if kind == "rotate_train" else 1)
        return {"bytes": 2 * n * size, "flops": 3 * n * case["rot"] // dim}
    if kind == "append":
        n = total * (hq + 2 * hk) * dim
        return {"bytes": 2 * n * size + 4 * m["table"].size, "flops": 3 * total * (hq + hk) * case["rot"]}
    if kind == "chunk":
        pairs, rows = 0, 0
        for past, n in zip(m["past"], m["fresh"]):
            p = np.arange(past, past + n, dtype=np.int64)
            w = p + 1 if case["window"] is None else np.minimum(p + 1, case["window"])
            s = np.minimum(case["sinks"], p + 1 - w)
            pairs += int((w + s).sum())
            first = 0 if case["window"] is None else max(0, past + 1 - case["window"])
            rows += past + n - first + min(case["sinks"], first)
        return {"bytes": 2 * nq * size + 2 * rows * hk * dim * size + 4 * m["table"].size + 4 * total * hq,
                "flops": 4 * pairs * hq * dim}
    nk = sum(m["states"]) * hk * dim
    pairs = sum(a * b for a, b in zip(m["fresh"], m["states"])) * hq
    if kind == "cross":
        return {"bytes": size * (2 * nq + 2 * nk) + 4 * total * hq, "flops": 4 * pairs * dim}
    # forward (scores, values) and backward (scores again, and the four gradient products)
    return {"bytes": size * (4 * nq + 4 * nk), "flops": 14 * pairs * dim}


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"rotate": _plain_rotate, "rotate_train": _plain_rotate_train, "append": _plain_append, "chunk": _plain_chunk,
            "cross": _plain_cross, "cross_train": _plain_cross_train}[s["kind"]](s)


def _run_own(s):
    import residual_vector_quantization_amd as rvq
    kind = s["kind"]
    if kind in ("rotate", "rotate_train"):
        how = dict(cu=s["cu"], first=s["past"], interleaved=s["interleaved"], amplitude=s["amplitude"])
        out = rvq.rvq_rotary(s["q"], s["k"], s["frequencies"], **how)
        if kind == "rotate":
            return out
        return (*out, *rvq.rvq_rotary(s["dq"], s["dk"], s["frequencies"], inverse=True, **how))
    if kind == "append":
        q = rvq.rvq_rotary_append(s["q"], s["k"], s["v"], s["frequencies"], s["k_pool"], s["v_pool"], s["table"],
                                  s["past"], s["cu"], interleaved=s["interleaved"], amplitude=s["amplitude"])
        return q, s["k_pool"], s["v_pool"]
    if kind == "chunk":
        return rvq.rvq_cache_chunk_attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"],
                                             window=s["window"], sinks=s["sinks"], scale=s["scale"])
    out, lse = rvq.rvq_cross_attention(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], scale=s["scale"])
    if kind == "cross":
        return out, lse
    return (out, *rvq.rvq_cross_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu"], s["cu_k"],
                                                   scale=s["scale"]))


# ---------------------------------------------------------------- plain forms

def _clip_of(cu, total):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(total, device=cu.device).int(), right=True)


def _positions(s):
    """Each packed frame's position in its clip, in 64 bits."""
    total = s["q"].shape[0]
    clip = _clip_of(s["cu"], total)
    return torch.arange(total, device=clip.device) - s["cu"].long()[clip] + s["past"].long()[clip], clip


def _turned(x, position, s, way):
    """x [T, H, D] with its first rot values turned by way * position * frequencies."""
    angle = position.double()[:, None] * s["frequencies"]
    c = (torch.cos(angle) * s["amplitude"]).float()[:, None]
    d = (torch.sin(angle) * (s["amplitude"] * way)).float()[:, None]
    rot = s["rot"]
    y = x.float()
    if s["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _plain_rotate(s):
    p, _ = _positions(s)
    return _turned(s["q"], p, s, 1), _turned(s["k"], p, s, 1)


def _plain_rotate_train(s):
    p, _ = _positions(s)
    return (_turned(s["q"], p, s, 1), _turned(s["k"], p, s, 1), _turned(s["dq"], p, s, -1), _turned(s["dk"], p, s, -1))


def _plain_append(s):
    p, clip = _positions(s)
    page = s["table"][clip, p // s["page"]].long()
    s["k_pool"][page, :, p % s["page"]] = _turned(s["k"], p, s, 1)
    s["v_pool"][page, :, p % s["page"]] = s["v"]
    return _turned(s["q"], p, s, 1), s["k_pool"], s["v_pool"]


def _padded(x, cu, longest):
    """[T, H, D] packed -> [B, H, longest, D] in 32 bits, zeros behind each clip's end."""
    at = torch.arange(longest, device=x.device)
    n = (cu[1:] - cu[:-1]).long()
    if x.shape[0] == 0:
        return torch.zeros(n.shape[0], x.shape[1], longest, x.shape[2], device=x.device)
    index = (cu[:-1].long()[:, None] + at).clamp(max=x.shape[0] - 1)
    y = x[index].float() * (at < n[:, None])[..., None, None]
    return y.transpose(1, 2).contiguous()


def _packed(y, cu, total):
    """[B, H, L, D] -> [T, H, D]: each clip's own rows."""
    clip = _clip_of(cu, total)
    return y[clip, :, torch.arange(total, device=y.device) - cu[clip].long()]


def _softmax(x):
    """Weights and log of the sum of exponentials; 0 and -inf for rows that are all -inf. Works in x's memory."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    return x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse[..., 0]


def _plain_chunk(s):
    table, lens, page, hk = s["table"], s["lens"].long(), s["page"], s["kv_heads"]
    most, longest = max(s["fresh_lens"]), max(s["lens_list"])
    q = _padded(s["q"], s["cu"], most)
    b, hq, n, d = q.shape
    at = torch.arange(longest, device=q.device)
    where = table.long()[:, at // page].clamp(min=0)
    k = s["k_pool"][where, :, at % page].float().permute(0, 2, 3, 1).contiguous()     # [B, Hk, D, L]
    v = s["v_pool"][where, :, at % page].float().transpose(1, 2).contiguous()         # [B, Hk, L, D]
    fresh = (s["cu"][1:] - s["cu"][:-1]).long()
    p = torch.arange(n, device=q.device) + (lens - fresh)[:, None]
    sees = (at <= p[..., None]) & (at < lens[:, None, None])
    if s["window"] is not None:
        sees &= (p[..., None] - at < s["window"]) | (at < s["sinks"])
    x = torch.matmul(q.view(b, hk, hq // hk * n, d), k).view(b, hk, hq // hk, n, longest).mul_(s["scale"])
    w, lse = _softmax(x.masked_fill_(~sees[:, None, None], -math.inf))
    out = torch.matmul(w.view(b, hk, hq // hk * n, longest), v).view(b, hq, n, d)
    total = s["q"].shape[0]
    lse = _packed(lse.reshape(b, hq, n, 1), s["cu"], total)[..., 0]
    return _packed(out, s["cu"], total).to(s["q"].dtype), lse.t().contiguous()


def _cross_weights(s):
    lq, lk, group = max(s["fresh_lens"]), max(1, max(s["states_lens"])), s["q_heads"] // s["kv_heads"]
    q, k, v = _padded(s["q"], s["cu"], lq), _padded(s["k"], s["cu_k"], lk), _padded(s["v"], s["cu_k"], lk)
    b, d = q.shape[0], q.shape[3]
    q = q.view(b, s["kv_heads"], group * lq, d)
    sees = torch.arange(lk, device=q.device) < (s["cu_k"][1:] - s["cu_k"][:-1])[:, None]
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    w, lse = _softmax(x.masked_fill_(~sees[:, None, None], -math.inf))
    return q, k, v, w, lse.view(b, s["q_heads"], lq, 1)


def _plain_cross(s):
    q, _, v, w, lse = _cross_weights(s)
    out = torch.matmul(w, v).view(q.shape[0], s["q_heads"], -1, q.shape[3])
    total = s["q"].shape[0]
    return _packed(out, s["cu"], total).to(s["q"].dtype), _packed(lse, s["cu"], total)[..., 0].t().contiguous()


def _plain_cross_train(s):
    q, k, v, w, _ = _cross_weights(s)
    b, heads, rows, d = q.shape
    typ, nq, nk = s["q"].dtype, s["q"].shape[0], s["k"].shape[0]
    out = torch.matmul(w, v)
    do = _padded(s["dout"], s["cu"], max(s["fresh_lens"])).view(b, heads, rows, d)
    dv = torch.matmul(w.transpose(2, 3).contiguous(), do)
    dx = torch.matmul(do, v.transpose(2, 3).contiguous())
    dx = dx.sub_((do * out).sum(-1, keepdim=True)).mul_(w)
    dq = torch.matmul(dx, k) * s["scale"]
    dk = torch.matmul(dx.transpose(2, 3).contiguous(), q) * s["scale"]
    out, dq = out.view(b, s["q_heads"], -1, d), dq.view(b, s["q_heads"], -1, d)
    return (_packed(out, s["cu"], nq).to(typ), _packed(dq, s["cu"], nq).to(typ), _packed(dk, s["cu_k"], nk).to(typ),
            _packed(dv, s["cu_k"], nk).to(typ))


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("cross", "cross_train"):
        return _exact_cross(s, case["kind"] == "cross_train")
    if case["kind"] == "chunk":
        return _exact_chunk(s)
    return _exact_rotary(s)


def _exact_rotary(s):
    q, past = s["q"], s["past"].tolist()
    position = torch.cat([torch.arange(n, device=q.device, dtype=torch.float64) + p for n, p in zip(s["fresh_lens"], past)])
    unit = torch.polar(torch.full_like(s["frequencies"], s["amplitude"])[None].expand(position.shape[0], -1).contiguous(),
                       torch.outer(position, s["frequencies"]))[:, None]

    def turn(x, by):
        y, rot = x.double().clone(), s["rot"]
        if s["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2).contiguous()) * by
            y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:2], rot)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * by
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    if s["kind"] == "append":
        k, page = turn(s["k"], unit), s["page"]
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
        at = 0
        for b, (n, p) in enumerate(zip(s["fresh_lens"], past)):
            j = torch.arange(p, p + n, device=q.device)
            where = s["table"][b].long()[j // page]
            k_pool[where, :, j % page] = k[at:at + n]
            v_pool[where, :, j % page] = s["v"][at:at + n].double()
            at += n
        return turn(q, unit), k_pool, v_pool
    got = (turn(q, unit), turn(s["k"], unit))
    if s["kind"] == "rotate_train":
        got += (turn(s["dq"], unit.conj()), turn(s["dk"], unit.conj()))
    return got


def _softmax64(x):
    top = x.max(-1, keepdim=True).values
    x = (x - top).exp()
    return x / x.sum(-1, keepdim=True), top[..., 0] + x.sum(-1).log()


def _exact_chunk(s):
    q, group = s["q"].double(), s["q_heads"] // s["kv_heads"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[1::-1], -math.inf, dtype=torch.float64, device=q.device)
    start = 0
    for b, (n, total) in enumerate(zip(s["fresh_lens"], s["lens_list"])):
        j = torch.arange(total, device=q.device)
        if s["window"] is not None:
            j = j[(j > total - n - s["window"]) | (j < s["sinks"])]
        pages = s["table"][b].long()[j // s["page"]]
        k, v = (s[p][pages, :, j % s["page"]].double() for p in ("k_pool", "v_pool"))
        p = torch.arange(total - n, total, device=q.device)[:, None]
        hidden = j > p
        if s["window"] is not None:
            hidden |= (j <= p - s["window"]) & (j >= s["sinks"])
        rows = slice(start, start + n)
        for h in range(s["q_heads"]):
            x = (q[rows, h] @ k[:, h // group].t() * s["scale"]).masked_fill(hidden, -math.inf)
            w, lse[h, rows] = _softmax64(x)
            out[rows, h] = w @ v[:, h // group]
        start += n
    return out, lse


def _exact_cross(s, train):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    group = s["q_heads"] // s["kv_heads"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[1::-1], -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    q0 = k0 = 0
    for nq, nk in zip(s["fresh_lens"], s["states_lens"]):
        a, e = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(s["q_heads"] if nk else 0):
            kh, vh = k[e, h // group], v[e, h // group]
            w, lse[h, a] = _softmax64(q[a, h] @ kh.t() * s["scale"])
            out[a, h] = w @ vh
            if train:
                g = s["dout"][a, h].double()
                dw = g @ vh.t()
                dx = w * (dw - (w * dw).sum(-1, keepdim=True)) * s["scale"]
                dq[a, h] = dx @ kh
                dk[e, h // group] += dx.t() @ q[a, h]
                dv[e, h // group] += w.t() @ g
        q0, k0 = q0 + nq, k0 + nk
    return (out, dq, dk, dv) if train else (out, lse)
