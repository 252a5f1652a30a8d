"""Rotary positions on the GPU, alone and on the way into the cache, against float64 on the CPU.

Bounds, with f = 2^-24 and u half a step of the inputs' type: the part of the angle that goes through the series is
known to 2 f of an eighth of a turn, the series and its roundings add 2 f, the amplitude (given in float64, used in
float32) and its product 2 f: sine and cosine are off by 6 f of the amplitude. The angle in float64 is off by 2^-51 of
itself and the oracle's by as much. Then come two products and a sum in float32 and one rounding to the type.
"""

import math
import random

import pytest
import torch

from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, ints, offsets
from test_gpu_cache import cache

pytestmark = [pytest.mark.gpu, needs_gpu]

F32 = 2.0 ** -24


def turned(x, position, frequencies, interleaved, amplitude, way=1):
    """(value, bound) in float64 on the CPU."""
    typ, x = x.dtype, x.double().cpu()
    n, u = len(frequencies), torch.finfo(typ).eps / 2
    angle = position.double()[:, None, None] * frequencies
    c, s = torch.cos(angle) * amplitude, torch.sin(angle) * amplitude * way
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., one], x[..., two]
    value, bound = x.clone(), torch.zeros_like(x)
    value[..., one], value[..., two] = a * c - b * s, b * c + a * s
    size = a.abs() + b.abs()
    off = size * abs(amplitude) * (8 * F32 + angle.abs() * 2.0 ** -50)
    for at in (one, two):
        y = value[..., at].abs()
        bound[..., at] = off + u * (y + off) + F32 * y + torch.finfo(typ).tiny * torch.finfo(typ).eps
    return value, bound


def close(name, got, want):
    value, bound = want
    off = ((got.double().cpu() - value).abs() - bound).max().item() if value.numel() else 0.0
    assert off <= 0, f"{name}: over the bound by {off}"


def waves(rot, factor=1.0):
    return rvq().rvq_rotary_frequencies(rot, scaling=None if factor == 1.0 else "ramp", factor=factor, context=4096)


def make(typ, tokens, hq, hk, dim, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, hq + hk, dim, generator=g).to(TYPES[typ]).to(DEV)
    return x[:, :hq], x[:, hq:]


def check(typ, dim, hq, hk, rot, lens, first=None, interleaved=False, amplitude=1.0, seed=0):
    m = rvq()
    announce("rotary", typ=typ, dim=dim, heads=(hq, hk), rot=rot, lens=lens, first=first, interleaved=interleaved)
    q, k = make(typ, sum(lens), hq, hk, dim, seed)
    f = waves(rot)
    at = torch.tensor([i + (first[b] if first else 0) for b, n in enumerate(lens) for i in range(n)], dtype=torch.int64)
    for inverse in (False, True):
        args = dict(interleaved=interleaved, amplitude=amplitude, inverse=inverse)
        got = m.rvq_rotary(q, k, f.to(DEV), cu=ints(offsets(lens)), first=ints(first) if first else None, **args)
        again = m.rvq_rotary(q, k, f.to(DEV), positions=at.to(torch.int32).to(DEV), **args)
        torch.cuda.synchronize()
        for name, x, y, z in zip("qk", (q, k), got, again):
            close(name, y, turned(x, at, f, interleaved, amplitude, -1 if inverse else 1))
            assert torch.equal(y, z)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (64, 16), (64, 2), (64, 6), (64, 40), (128, 128), (128, 96), (128, 24), (128, 126)])
@pytest.mark.parametrize("typ", list(TYPES))
def test_layouts_and_parts_of_the_head(typ, dim, rot, interleaved):
    check(typ, dim, 3, 1, rot, [5, 0, 33, 1, 0], interleaved=interleaved)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (16, 4), (33, 7), (64, 64)])
@pytest.mark.parametrize("tokens", [1, 2, 31, 700])
def test_heads_and_tokens(hq, hk, tokens):
    check("bf16", 64, hq, hk, 64, [tokens], first=[7])
    check("fp32", 128, hq, hk, 64, [tokens], interleaved=True, amplitude=1.25)


@pytest.mark.parametrize("typ", list(TYPES))
def test_many_tokens(typ):
    """Enough for a thread to take several heads, and for the loop's last turn to be a part of one."""
    check(typ, 64, 9, 2, 64, [30000, 3, 9000], first=[0, 5, 100000])
    check(typ, 128, 4, 3, 20, [50000], interleaved=True)


def test_far_positions():
    check("fp32", 64, 1, 1, 64, [40, 40, 40, 40], first=[0, 999_990, 2 ** 24 + 1, 2 ** 31 - 41])
    check("fp32", 64, 1, 1, 64, [40], first=[-20])


def test_more_clips_than_are_staged():
    rng = random.Random(0)
    lens = [rng.choice([0, 1, 2, 5]) for _ in range(1500)]
    check("fp16", 64, 2, 1, 64, lens, first=[rng.randrange(5000) for _ in lens])


def test_queries_or_keys_alone():
    m = rvq()
    q, k = make("bf16", 20, 4, 2, 64)
    f, cu = waves(64).to(DEV), ints([0, 20])
    both = m.rvq_rotary(q, k, f, cu=cu)
    one, none = m.rvq_rotary(q, None, f, cu=cu)
    assert none is None and torch.equal(one, both[0])
    none, one = m.rvq_rotary(None, k, f, cu=cu)
    assert none is None and torch.equal(one, both[1])
    empty = m.rvq_rotary(q[:0], k[:0], f, cu=ints([0, 0]))
    assert empty[0].shape == (0, 4, 64) and empty[1].shape == (0, 2, 64)


@pytest.mark.parametrize("rot,interleaved", [(64, False), (32, True), (22, False)])
def test_in_place_and_rows_outside_clips(rot, interleaved):
    m = rvq()
    for typ in TYPES:
        q, k = make(typ, 50, 4, 2, 64)
        f, cu = waves(rot).to(DEV), ints([3, 10, 10, 41])
        out = tuple(torch.full_like(x, 7.0) for x in (q, k))
        m.rvq_rotary(q, k, f, cu=cu, interleaved=interleaved, out=out)
        was = q.clone(), k.clone()
        m.rvq_rotary(q, k, f, cu=cu, interleaved=interleaved, out=(q, k))
        for x, y, z in zip((q, k), was, out):
            assert torch.equal(x[3:41], z[3:41])
            assert torch.equal(x[:3], y[:3]) and torch.equal(x[41:], y[41:])
            assert (z[:3] == 7).all() and (z[41:] == 7).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """The operator is linear, so differences are exact but for roundings: 2^-24 each of sums of 2 * 64 products."""
    m = rvq()
    x, _ = make("fp32", 60, 3, 1, 64, 1)
    step, _ = make("fp32", 60, 3, 1, 64, 2)
    g, _ = make("fp32", 60, 3, 1, 64, 3)
    f, args = waves(48).to(DEV), dict(cu=ints([0, 60]), interleaved=interleaved, amplitude=1.5)
    lose = m.rvq_rotary(g, None, f, inverse=True, **args)[0].double()
    change = m.rvq_rotary(x + step, None, f, **args)[0].double() - m.rvq_rotary(x, None, f, **args)[0].double()
    actual = (x + step).double() - x.double()
    left, right = (lose * actual).sum((1, 2)), (g.double() * change).sum((1, 2))
    sizes = (g.abs().double().square().sum((1, 2)) * (x.abs() + step.abs()).double().square().sum((1, 2))).sqrt()
    assert ((left - right).abs() <= 1.5 * 24 * F32 * sizes).all()


def test_scores_depend_on_the_distance():
    m = rvq()
    q, k = make("fp32", 1, 1, 1, 64)
    f = waves(64).to(DEV)

    def score(a, b):
        x = m.rvq_rotary(q, None, f, positions=ints([a]))[0].double()
        y = m.rvq_rotary(None, k, f, positions=ints([b]))[1].double()
        return (x * y).sum().item()

    size = q.double().norm().item() * k.double().norm().item()
    for far in (100, 1_000_000, 2_000_000_000):
        assert abs(score(far + 13, far) - score(13, 0)) <= 24 * F32 * size


# ---------------------------------------------------------------- on the way into the cache

@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 50, False), (128, 10, True)])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [1, 7, 16])
def test_append_is_rotation_and_append(typ, dim, rot, interleaved, page):
    m = rvq()
    hq, hk, old, new = 6, 2, [0, 5, 16, 33, 2], [3, 1, 0, 20, 40]
    announce("rotary append", typ=typ, dim=dim, rot=rot, page=page)
    k_pool, v_pool, table, _ = cache(typ, dim, hk, page, [a + b for a, b in zip(old, new)])
    table[4][-(-30 // page)] = -1           # some frames of the last clip have no page
    q, kv = make(typ, sum(new), hq, 2 * hk, dim)
    k, v = kv[:, :hk], kv[:, hk:]
    f, cu = waves(rot).to(DEV), ints(offsets(new))
    args = dict(interleaved=interleaved, amplitude=0.75)
    want = tuple(p.clone() for p in (k_pool, v_pool))
    q_want, k_turned = m.rvq_rotary(q, k, f, cu=cu, first=ints(old), **args)
    m.rvq_cache_append(k_turned, v, *want, ints(table), ints(old), cu)
    got = m.rvq_rotary_append(q, k, v, f, k_pool, v_pool, ints(table), ints(old), cu, **args)
    torch.cuda.synchronize()
    assert torch.equal(got, q_want)
    for x, y in zip((k_pool, v_pool), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_one_frame_each():
    m = rvq()
    hq, hk, old = 4, 4, [0, 5, 16, 33, 2, 700]
    for queries in (True, False):
        k_pool, v_pool, table, _ = cache("bf16", 64, hk, 8, [n + 1 for n in old])
        q, kv = make("bf16", len(old), hq, 2 * hk, 64)
        k, v = kv[:, :hk], kv[:, hk:]
        f = waves(64).to(DEV)
        want = tuple(p.clone() for p in (k_pool, v_pool))
        q_want, k_turned = m.rvq_rotary(q, k, f, positions=ints(old))
        m.rvq_cache_append(k_turned, v, *want, ints(table), ints(old))
        got = m.rvq_rotary_append(q if queries else None, k, v, f, k_pool, v_pool, ints(table), ints(old))
        assert got is None if not queries else torch.equal(got, q_want)
        for x, y in zip((k_pool, v_pool), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_without_pages():
    m = rvq()
    pool = torch.empty(0, 2, 4, 64, device=DEV)
    q, kv = make("fp32", 3, 2, 4, 64)
    f, lens = waves(64).to(DEV), ints([4, 0, 9])
    table = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    got = m.rvq_rotary_append(q, kv[:, :2], kv[:, 2:], f, pool, pool.clone(), table, lens)
    assert torch.equal(got, m.rvq_rotary(q, None, f, positions=lens)[0])


# ---------------------------------------------------------------- graphs and streams

def test_captured_step_and_other_stream():
    m = rvq()
    old = [3, 40, 9]
    k_pool, v_pool, table, _ = cache("fp16", 64, 2, 16, [n + 8 for n in old])
    q, kv = make("fp16", 3, 4, 4, 64)
    q, kv = q.contiguous(), kv.contiguous()
    f, lens, table = waves(64).to(DEV), ints(old), ints(table)
    out = torch.empty_like(q)

    def step():
        m.rvq_rotary_append(q, kv[:, :2], kv[:, 2:], f, k_pool, v_pool, table, lens, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        lens.add_(1)
        q.normal_()
        kv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = tuple(p.clone() for p in (k_pool, v_pool))
        q_want, k_turned = m.rvq_rotary(q, kv[:, :2], f, positions=lens)
        m.rvq_cache_append(k_turned, kv[:, 2:].contiguous(), *want, table, lens)
        assert torch.equal(out, q_want)
        for x, y in zip((k_pool, v_pool), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
