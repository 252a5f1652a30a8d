"""The paged key-value cache on the GPU: attention of the newest frame against float64, and the pages' upkeep
against a page-by-page account on the CPU (attention_oracle)."""

import math
import random

import pytest
import torch

import attention_oracle as oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints

pytestmark = [pytest.mark.gpu, needs_gpu]


def cache(typ, dim, hk, page, lens, spare=3, seed=0, window=None, sinks=0, wide=0):
    """Pools with pages in random places, the table and the reference counts; pages behind the window are given
    back, and what no clip holds is NaN."""
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    cols = max([1] + [-(-n // page) for n in lens]) + wide
    table = [[-1] * cols for _ in lens]
    want = [(b, e) for b, n in enumerate(lens) for e in range(-(-n // page))
            if window is None or e * page < sinks or (e + 1) * page > n - window]
    pages = len(want) + spare
    order = list(range(pages))
    rng.shuffle(order)
    pools = [torch.full((pages, hk, page, dim), math.nan, dtype=TYPES[typ]) for _ in range(2)]
    refs = [0] * pages
    for (b, e), p in zip(want, order):
        table[b][e] = p
        refs[p] = 1
        held = min(page, lens[b] - e * page)
        for pool in pools:
            pool[p, :, :held] = torch.randn(hk, held, dim, generator=g).to(TYPES[typ])
    return pools[0].to(DEV), pools[1].to(DEV), table, refs


def check(typ, dim, hq, hk, page, lens, window=None, sinks=0, scale=None, seed=0):
    m = rvq()
    announce("cache attention", typ=typ, dim=dim, heads=(hq, hk), page=page, lens=lens, window=window, sinks=sinks)
    k, v, table, _ = cache(typ, dim, hk, page, lens, seed=seed, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), hq, dim, generator=g).to(TYPES[typ]).to(DEV)
    out = m.rvq_cache_attention(q, k, v, ints(table), ints(lens), window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    close("out", out, oracle.cache_attention(q, k, v, ints(table), ints(lens), window, sinks,
                                             1 / math.sqrt(dim) if scale is None else scale))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [1, 7, 16, 100])
def test_lengths_and_pages(typ, dim, page):
    check(typ, dim, 4, 2, page, [1, 0, 2, page, page + 1, 31, 32, 33, 63, 64, 65, 130])


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (5, 1), (16, 1), (17, 1), (24, 1), (40, 2), (6, 6), (32, 8)])
@pytest.mark.parametrize("typ", ["bf16", "fp32"])
def test_head_groups(typ, hq, hk):
    check(typ, 64, hq, hk, 16, [200, 3, 77])


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 2), (1, 0), (1, 4), (16, 3), (33, 40), (64, 64), (100, 1), (4000, 3)])
@pytest.mark.parametrize("typ", list(TYPES))
def test_windows_and_sinks(typ, window, sinks):
    check(typ, 64, 4, 2, 16, [300, 16, 1, 65, 0, 128], window=window, sinks=sinks)


@pytest.mark.parametrize("typ,dim", [("bf16", 128), ("fp16", 64), ("fp32", 128)])
def test_long_caches_are_split_and_joined(typ, dim):
    check(typ, dim, 4, 2, 32, [5000, 12, 4097, 2049])
    check(typ, dim, 8, 1, 24, [9001])


def test_other_scales():
    check("bf16", 64, 4, 2, 16, [300], scale=2.5)
    check("fp32", 64, 4, 2, 16, [300], scale=0.0)


def test_a_frame_without_a_page_gives_nan_and_only_there():
    m = rvq()
    lens = [100, 100, 100, 100, 100]
    k, v, table, _ = cache("bf16", 64, 2, 16, lens)
    q = torch.randn(5, 4, 64, device=DEV).bfloat16()
    good = m.rvq_cache_attention(q, k, v, ints(table), ints(lens), window=40, sinks=3)
    table[1][5], table[2][6], table[3][0] = -1, k.shape[0], -7
    table[0][1] = table[4][2] = 123456789      # behind the window: not looked at
    out = m.rvq_cache_attention(q, k, v, ints(table), ints(lens), window=40, sinks=3)
    assert torch.isnan(out[1:4]).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[4], good[4])
    # a count beyond the table
    out = m.rvq_cache_attention(q, k, v, ints(table), ints([100, 0, -5, 113, 2 ** 31 - 1]), window=40, sinks=3)
    assert torch.equal(out[0], good[0]) and (out[1:3] == 0).all() and torch.isnan(out[3:]).all()


@pytest.mark.parametrize("typ", list(TYPES))
def test_prefill_and_decode_agree(typ):
    """Frame by frame through the cache gives what the windowed attention gives at once."""
    m = rvq()
    n, hq, hk, dim, page, window, sinks = 70, 4, 2, 64, 8, 20, 3
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, h, dim, generator=g).to(TYPES[typ]).to(DEV) for h in (hq, hk, hk))
    want, _ = m.rvq_window_attention(q, k, v, ints([0, n]), window=window, sinks=sinks)
    pools = [torch.full((20, hk, page, dim), math.nan, dtype=TYPES[typ], device=DEV) for _ in range(2)]
    table, refs, lens = ints([[-1] * 10]), ints([0] * 20), ints([0])
    u = torch.finfo(TYPES[typ]).eps / 2
    size = v.double().abs().amax()
    for i in range(n):
        table, refs, missing = m.rvq_cache_reserve(table, lens, lens + 1, refs, page)
        m.rvq_cache_append(k[i:i + 1], v[i:i + 1], *pools, table, lens)
        lens = lens + 1
        out = m.rvq_cache_attention(q[i:i + 1], *pools, table, lens, window=window, sinks=sinks)
        table, lens, refs = m.rvq_cache_free(table, lens, refs, page, window=window, sinks=sinks)
        # each side rounds its weights and its result once, and sums in float32
        assert (out[0].double() - want[i].double()).abs().max() <= (4 * u + 600 * 2.0 ** -24) * size, i
        assert missing.item() == 0
    assert int((refs > 0).sum()) <= -(-window // page) + 2


def test_strided_queries_and_the_same_bits():
    m = rvq()
    lens = [3000, 40, 700]
    k, v, table, _ = cache("bf16", 128, 2, 16, lens)
    qkv = torch.randn(3, 12, 128, device=DEV).bfloat16()
    q = qkv[:, 2:10]
    args = (k, v, ints(table), ints(lens))
    one = m.rvq_cache_attention(q, *args)
    out = torch.zeros(3, 20, 128, dtype=torch.bfloat16, device=DEV)
    m.rvq_cache_attention(q.contiguous(), *args, out=out[:, 5:13])
    assert torch.equal(one, out[:, 5:13]) and (out[:, :5] == 0).all() and (out[:, 13:] == 0).all()
    for _ in range(3):
        assert torch.equal(one, m.rvq_cache_attention(q, *args))


def test_graph_of_a_decode_step():
    m = rvq()
    lens = [3000, 40]
    k, v, table, _ = cache("bf16", 64, 2, 16, lens, wide=1)
    q = torch.randn(2, 4, 64, device=DEV).bfloat16()
    table, counts = ints(table), ints(lens)

    def step():
        return m.rvq_cache_attention(q, k, v, table, counts, window=1000, sinks=4)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        q.normal_()
        counts.copy_(ints([3000 - 500 * turn, 40 - turn]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, step()), turn
        torch.cuda.synchronize()


# ---------------------------------------------------------------- pages

@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("fp32", 128)])
def test_append(typ, dim):
    m = rvq()
    hk, page = 3, 5
    lens, add = [0, 7, 5, 12, 3], [3, 11, 0, 1, 6]
    k_pool, v_pool, table, refs = cache(typ, dim, hk, page, [n + a for n, a in zip(lens, add)], seed=2)
    table[4][1] = -1                             # the last clip's frames from position 5 on have no page
    g = torch.Generator().manual_seed(8)
    new = [torch.randn(sum(add), hk, dim, generator=g).to(TYPES[typ]).to(DEV) for _ in range(2)]
    want = [p.clone() for p in (k_pool, v_pool)]
    at = 0
    for b, (n, a) in enumerate(zip(lens, add)):
        for j in range(n, n + a):
            p = table[b][j // page]
            if p >= 0:
                for w, x in zip(want, new):
                    w[p, :, j % page] = x[at]
            at += 1
    cu = [0] + torch.tensor(add).cumsum(0).tolist()
    m.rvq_cache_append(*new, k_pool, v_pool, ints(table), ints(lens), ints(cu))
    for w, x in zip(want, (k_pool, v_pool)):
        assert torch.equal(w.view(torch.uint8), x.view(torch.uint8))
    # one frame each, a position beyond the table and one before it
    before = k_pool.clone()
    one = new[0][:5]
    m.rvq_cache_append(one, one, k_pool, v_pool, ints(table), ints([10 ** 6, -1, 2 ** 31 - 1, 0, 5]))
    before[table[3][0], :, 0] = one[3]
    assert torch.equal(before.view(torch.uint8), k_pool.view(torch.uint8))


def random_tables(rng, clips, cols, pages, page):
    """Clips that share some full pages, and a partial page each of their own."""
    refs, table, lens = [0] * pages, [], []
    order = list(range(pages))
    rng.shuffle(order)
    for b in range(clips):
        row, n = [-1] * cols, rng.choice([0, page, rng.randrange(cols * page + 1)])
        for e in range(-(-n // page)):
            full = (e + 1) * page <= n
            if full and table and lens[-1] >= (e + 1) * page and rng.random() < 0.5 and table[-1][e] >= 0:
                row[e] = table[-1][e]
            elif order:
                row[e] = order.pop()
            else:
                n = e * page
                break
            refs[row[e]] += 1
        table.append(row)
        lens.append(n)
    return table, lens, refs


@pytest.mark.parametrize("clips,cols,pages,page", [(1, 1, 1, 1), (3, 4, 9, 16), (40, 7, 200, 8), (300, 9, 2100, 4),
                                                   (700, 20, 9000, 3), (5, 3, 70000, 2),
                                                   (4500, 2, 7000, 2)])
def test_reserve_free_fork_compact(clips, cols, pages, page):
    m = rvq()
    rng = random.Random(clips * 1000 + pages)
    for turn in range(3):
        announce("pages", clips=clips, cols=cols, pages=pages, page=page, turn=turn)
        table, lens, refs = random_tables(rng, clips, cols, pages, page)
        # reserve
        new = [n + rng.choice([0, 0, 1, rng.randrange(3 * page)]) for n in lens]
        got = m.rvq_cache_reserve(ints(table), ints(lens), ints(new), ints(refs), page)
        want = oracle.reserve(table, lens, new, refs, page)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].item() == want[2]
        # free
        drop = [int(rng.random() < 0.3) for _ in lens]
        for d, window, sinks in ((drop, None, 0), (None, 2 * page, 1), (drop, 3, page + 1), (None, 0, 0), (None, None, 0)):
            got = m.rvq_cache_free(ints(table), ints(lens), ints(refs), page, None if d is None else ints(d), window, sinks)
            want = oracle.free(table, lens, refs, page, d, window, sinks)
            assert all(a.tolist() == b for a, b in zip(got, want)), (window, sinks)
        # fork: all clips, and a few
        layers, dim, hk = 2, 64, 1
        pools = [torch.arange(layers * pages, device=DEV, dtype=torch.float32).view(layers, pages, 1, 1, 1).expand(
            layers, pages, hk, page, dim).contiguous() + x for x in (0, 0.25)]
        for count in (clips, min(2, clips)):
            children = rng.sample(range(clips), count)
            parents = [rng.randrange(clips) for _ in children]
            if count > 1:
                parents[0] = rng.choice([-1, clips, parents[0]])
            moved, copies = [p.clone() for p in pools], []
            got = m.rvq_cache_fork(ints(table), ints(lens), ints(refs), ints(parents), ints(children), *moved)
            want = oracle.fork(table, lens, refs, parents, children, page, copies)
            assert all(a.tolist() == b for a, b in zip(got[:3], want[:3])) and got[3].item() == want[3]
            for p, q in zip(pools, moved):
                p = p.clone()
                for s, d in copies:
                    p[:, d] = p[:, s]
                assert torch.equal(p, q)
        # compact what a free leaves
        freed = oracle.free(table, lens, refs, page, drop, page, 1)
        copies = []
        got = m.rvq_cache_compact(ints(freed[0]), ints(freed[2]), *pools)
        want = oracle.compact(freed[0], freed[2], copies)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].item() == want[2]
        src, dst = [s for s, _ in copies], [d for _, d in copies]
        for pool, x in zip(pools, (0, 0.25)):
            number = (pool[:, :, 0, 0, 0] - x).cpu()
            expect = torch.arange(layers * pages, dtype=torch.float32).view(layers, pages)
            expect[:, dst] = expect[:, src]
            assert torch.equal(number, expect)
            assert (pool == pool[..., :1, :1, :1]).all()


def test_a_fork_without_room():
    m = rvq()
    table, lens, refs = [[0, 1], [2, -1], [-1, -1]], [6, 3, 0], [1, 1, 1, 0]
    pools = [torch.arange(4.0, device=DEV).view(4, 1, 1, 1).expand(4, 1, 4, 64).contiguous() for _ in range(2)]
    got = m.rvq_cache_fork(ints(table), ints(lens), ints(refs), ints([1, 0, 0]), ints([2, 1, 0]), *pools)
    # the only free page goes to the first pair; pages let go of by this call are not handed out in it
    assert got[0].tolist() == [[0, -1], [0, -1], [3, -1]]
    assert got[1].tolist() == [6, 6, 3] and got[2].tolist() == [2, 0, 0, 1] and got[3].item() == 2
    assert pools[0][:, 0, 0, 0].tolist() == [0, 1, 2, 2]


@pytest.mark.parametrize("dims", [4, 5])
def test_copy(dims):
    m = rvq()
    shape = (9, 2, 3, 64) if dims == 4 else (4, 9, 2, 3, 64)
    k, v = torch.randn(shape, device=DEV), torch.randn(shape, device=DEV)
    src, dst = [0, 5, 7, -1, 9, 2], [1, 3, 8, 4, 4, 9]
    want = [k.clone(), v.clone()]
    for w in want:
        pages = w.movedim(-4, 0)
        for s, d in zip(src[:3], dst[:3]):
            pages[d] = pages[s]
    m.rvq_cache_copy(ints(src), ints(dst), k, v)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_wide_offsets():
    """Rows past 2^31 values into a pool are found."""
    m = rvq()
    pages, hk, page, dim = 17000, 8, 128, 128          # 2.2e9 values a pool
    pools = [torch.empty((pages, hk, page, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(40, hk, dim, generator=g).bfloat16().to(DEV) for _ in range(2)]
    table, lens = ints([[pages - 1, pages - 2]]), ints([100])
    old = [torch.randn(2, hk, page, dim, generator=g).bfloat16().to(DEV) for _ in range(2)]
    for pool, x in zip(pools, old):
        pool[pages - 1], pool[pages - 2] = x[0], x[1]
    m.rvq_cache_append(*new, *pools, table, lens, ints([0, 40]))
    m.rvq_cache_copy(ints([pages - 1, pages - 2]), ints([1, 0]), *pools)
    q = torch.randn(1, 16, dim, generator=g).bfloat16().to(DEV)
    small = [torch.stack([pool[0], pool[1]]).contiguous() for pool in pools]
    out = m.rvq_cache_attention(q, *pools, table, ints([140]))
    close("out", out, oracle.cache_attention(q, *small, ints([[1, 0]]), ints([140]), None, 0, 1 / math.sqrt(dim)))
    for pool, x in zip(small, new):
        assert torch.equal(pool[1][:, 100:].transpose(0, 1), x[:28]) and torch.equal(pool[0][:, :12].transpose(0, 1), x[28:])


def test_refusals():
    m = rvq()
    lens = [20, 5]
    k, v, table, refs = cache("bf16", 64, 2, 16, lens)
    table, lens, refs = ints(table), ints(lens), ints(refs)
    q = torch.randn(2, 4, 64, device=DEV).bfloat16()
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q[:, :3], k, v, table, lens)
    with pytest.raises(TypeError):
        m.rvq_cache_attention(q.float(), k, v, table, lens)
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q[:1], k, v, table, lens)
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q, k, v[:-1], table, lens)
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q, k, v, table, lens[:1])
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q, k, v, table, lens, window=-2)
    with pytest.raises(ValueError):
        m.rvq_cache_attention(q, k.transpose(1, 2), v.transpose(1, 2), table, lens)
    with pytest.raises(m.RVQError):
        m.rvq_cache_attention(q, k, v, table, lens, scale=math.nan)
    with pytest.raises(m.RVQError):
        m.rvq_cache_attention(q[..., :32], k[..., :32].contiguous(), v[..., :32].contiguous(), table, lens)
    with pytest.raises(TypeError):
        m.rvq_cache_append(q[:, :2].float(), q[:, :2].float(), k, v, table, lens)
    with pytest.raises(ValueError):
        m.rvq_cache_append(q[:1, :2], q[:1, :2], k, v, table, lens)
    with pytest.raises(ValueError):
        m.rvq_cache_append(q[:, :2], q[:, :2], k, v, table, lens, ints([0, 2]))
    with pytest.raises(m.RVQError):
        m.rvq_cache_reserve(table, lens, lens, refs, 0)
    with pytest.raises(ValueError):
        m.rvq_cache_reserve(table, lens, lens[:1], refs, 16)
    with pytest.raises(TypeError):
        m.rvq_cache_reserve(table.long(), lens, lens, refs, 16)
    with pytest.raises(ValueError):
        m.rvq_cache_fork(table, lens, refs, ints([0]), ints([0, 1]), k, v)
    with pytest.raises(ValueError):
        m.rvq_cache_fork(table, lens, refs, ints([0, 0, 0]), ints([0, 1, 0]), k, v)
    with pytest.raises(ValueError):
        m.rvq_cache_fork(table, lens, refs[:-1], ints([0]), ints([1]), k, v)
    with pytest.raises(ValueError):
        m.rvq_cache_compact(table, refs[:-1], k, v)
    with pytest.raises(ValueError):
        m.rvq_cache_free(table, lens, refs, 16, drop=ints([1]))
    with pytest.raises(ValueError):
        m.rvq_cache_copy(ints([0, 1]), ints([2]), k, v)


def test_nothing_to_do():
    m = rvq()
    k = torch.zeros(0, 2, 16, 64, device=DEV)
    table, none = torch.zeros((0, 4), dtype=torch.int32, device=DEV), ints([])
    assert m.rvq_cache_attention(torch.zeros(0, 4, 64, device=DEV), k, k, table, none).shape == (0, 4, 64)
    m.rvq_cache_append(torch.zeros(0, 2, 64, device=DEV), torch.zeros(0, 2, 64, device=DEV), k, k, table, none)
    assert m.rvq_cache_reserve(table, none, none, none, 16)[2].item() == 0
    assert m.rvq_cache_compact(table, none, k, k)[2].item() == 0
    # clips without pages in an empty pool
    table, lens = ints([[-1], [-1]]), ints([0, 0])
    out = m.rvq_cache_attention(torch.ones(2, 4, 64, device=DEV), k, k, table, lens)
    assert (out == 0).all()
    assert m.rvq_cache_reserve(table, lens, ints([1, 17]), none, 16)[2].item() == 3
