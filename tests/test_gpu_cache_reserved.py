"""Upkeep of cache pages on the GPU where a table is not the plainest one: pages reserved ahead, pages that are not
there, no clips at all. Accounts are written out by hand; after every operation a page's count is the number of
table entries that name it."""

import math

import pytest
import torch

from gpu_util import DEV, announce, needs_gpu, rvq

pytestmark = [pytest.mark.gpu, needs_gpu]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def counted(table, pages):
    """How many entries name each page."""
    named = torch.tensor(table).flatten()
    return torch.bincount(named[(named >= 0) & (named < pages)].long(), minlength=pages).tolist()


# ---------------------------------------------------------------- free

@pytest.mark.parametrize("pages", [0, 5, 65536, 70000])
def test_free_without_clips(pages):
    m = rvq()
    announce("free of no clips", pages=pages)
    table, none = torch.zeros((0, 4), dtype=torch.int32, device=DEV), ints([])
    refs = (torch.arange(pages, device=DEV) % 3).int()
    got = m.rvq_cache_free(table, none, refs, 16)
    assert got[0].shape == (0, 4) and got[1].shape == (0,) and torch.equal(got[2], refs)


# ---------------------------------------------------------------- reserve

def reserved(table, lens, new_lens, refs, page):
    """The account of a reserve: in the columns of positions lens .. new_lens - 1, entries that name no page get one."""
    table, refs = [list(r) for r in table], list(refs)
    pages = len(refs)
    free, missing = [p for p, n in enumerate(refs) if n <= 0], 0
    for row, had, want in zip(table, lens, new_lens):
        for e in range(-(-max(had, 0) // page), -(-max(want, 0) // page)):
            if e < len(row) and 0 <= row[e] < pages:
                continue
            if e >= len(row) or not free:
                missing += 1
                continue
            row[e] = free.pop(0)
            refs[row[e]] = 1
    return table, refs, missing


def test_pages_reserved_ahead_stay():
    m = rvq()
    table, lens = [[0, -1, -1, -1], [-1, -1, -1, -1], [1, 2, -1, -1]], ints([3, 0, 8])
    refs = ints(counted(table, 12))
    held = [[0, 3, 4, -1], [5, 6, -1, -1], [1, 2, -1, -1]]
    table, refs, missing = m.rvq_cache_reserve(ints(table), lens, ints([9, 5, 8]), refs, 4)
    assert table.tolist() == held and refs.tolist() == counted(held, 12) and missing.item() == 0
    # the same again, before any frame has been written
    table, refs, missing = m.rvq_cache_reserve(table, lens, ints([9, 5, 8]), refs, 4)
    assert table.tolist() == held and refs.tolist() == counted(held, 12) and missing.item() == 0
    # and further ahead
    held = [[0, 3, 4, 7], [5, 6, -1, -1], [1, 2, 8, 9]]
    table, refs, missing = m.rvq_cache_reserve(table, lens, ints([13, 5, 16]), refs, 4)
    assert table.tolist() == held and refs.tolist() == counted(held, 12) and missing.item() == 0


def test_a_reserve_that_found_too_few_pages_is_taken_up_again():
    m = rvq()
    table, lens, new = [[-1, -1, -1], [-1, -1, -1], [1, 4, -1]], ints([0, 0, 8]), ints([12, 8, 8])
    refs = ints(counted(table, 6))
    table, refs, missing = m.rvq_cache_reserve(ints(table), lens, new, refs, 4)
    assert table.tolist() == [[0, 2, 3], [5, -1, -1], [1, 4, -1]] and missing.item() == 1
    table, lens, refs = m.rvq_cache_free(table, lens, refs, 4, drop=ints([0, 0, 1]))
    held = [[0, 2, 3], [5, 1, -1], [-1, -1, -1]]
    table, refs, missing = m.rvq_cache_reserve(table, lens, ints([12, 8, 0]), refs, 4)
    assert table.tolist() == held and refs.tolist() == counted(held, 6) and missing.item() == 0


@pytest.mark.parametrize("clips,cols,pages,page", [(1, 1, 1, 1), (1, 700, 900, 3), (7, 5, 40, 16), (300, 9, 2100, 4),
                                                   (20, 130, 70000, 2), (4500, 4, 9000, 2)])
def test_reserve_among_pages_that_are_there(clips, cols, pages, page):
    """Some columns beyond the count already name a page, some name none or something that is no page."""
    m = rvq()
    g = torch.Generator().manual_seed(clips + pages)
    for turn in range(3):
        announce("reserve", clips=clips, cols=cols, pages=pages, page=page, turn=turn)
        lens = torch.randint(0, cols * page + 1, (clips,), generator=g)
        new = lens + torch.randint(0, 2 * page * min(cols, 8), (clips,), generator=g) * torch.randint(0, 2, (clips,), generator=g)
        order = torch.randperm(pages, generator=g).tolist()
        table, there = [], torch.rand(clips, cols, generator=g).tolist()
        for b in range(clips):
            row = []
            for e in range(cols):
                inside = e * page < lens[b]
                if (inside or there[b][e] < 0.3) and order:
                    row.append(order.pop())
                else:
                    row.append(-1 if there[b][e] < 0.8 else (pages, -5, 2 ** 31 - 1)[e % 3])
            table.append(row)
        refs = counted(table, pages)
        want = reserved(table, lens.tolist(), new.tolist(), refs, page)
        got = m.rvq_cache_reserve(ints(table), lens.int().to(DEV), new.int().to(DEV), ints(refs), page)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].item() == want[2]
        assert want[1] == counted(want[0], pages)


# ---------------------------------------------------------------- fork

@pytest.mark.parametrize("gone", [-1, 7, 2 ** 31 - 1, -2 ** 31])
def test_a_fork_of_a_clip_whose_partial_page_is_not_there(gone):
    """The child has no page there either: it does not get one with another clip's old frames."""
    m = rvq()
    page, pages = 4, 7
    table, lens = [[1, gone, -1], [2, -1, -1], [-1, -1, -1], [-1, -1, -1]], [6, 3, 0, 0]
    refs = counted(table, pages)
    g = torch.Generator().manual_seed(1)
    pools = [torch.randn(pages, 1, page, 64, generator=g).to(DEV) for _ in range(2)]
    table, lens, refs, missing = m.rvq_cache_fork(ints(table), ints(lens), ints(refs), ints([0, 1]), ints([2, 3]), *pools)
    held = [[1, gone, -1], [2, -1, -1], [1, -1, -1], [0, -1, -1]]
    assert table.tolist() == held and refs.tolist() == counted(held, pages)
    assert lens.tolist() == [6, 3, 6, 3] and missing.item() == 0
    out = m.rvq_cache_attention(torch.ones(4, 1, 64, device=DEV), *pools, table, lens)
    assert torch.isnan(out[0]).all() and torch.isnan(out[2]).all()
    assert torch.isfinite(out[1]).all() and torch.equal(out[1], out[3])


def test_a_fork_does_not_share_pages_that_were_reserved_ahead():
    m = rvq()
    page, pages = 4, 9
    table, lens = [[0, 1, 2], [3, 4, -1], [5, -1, -1], [-1, -1, -1]], [6, 4, 0, 0]
    refs = counted(table, pages)
    pools = [torch.full((pages, 1, page, 64), math.nan, device=DEV) for _ in range(2)]
    for b, n in enumerate(lens):                    # frame j of clip b holds 100 b + j
        for j in range(n):
            for pool in pools:
                pool[table[b][j // page], :, j % page] = 100 * b + j
    table, lens, refs, missing = m.rvq_cache_fork(ints(table), ints(lens), ints(refs), ints([0, 1, 0]), ints([2, 3, 1]), *pools)
    held = [[0, 1, 2], [0, 7, -1], [0, 6, -1], [3, -1, -1]]
    assert table.tolist() == held and refs.tolist() == counted(held, pages)
    assert lens.tolist() == [6, 6, 6, 4] and missing.item() == 0
    # every clip goes on by four frames of its own
    table, refs, missing = m.rvq_cache_reserve(table, lens, lens + 4, refs, page)
    assert missing.item() == 0 and refs.tolist() == counted(table.tolist(), pages)
    new = (1000 + torch.arange(16.0, device=DEV)).view(16, 1, 1).expand(16, 1, 64).contiguous()
    m.rvq_cache_append(new, new, *pools, table, lens, ints([0, 4, 8, 12, 16]))
    was = [[0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], [100, 101, 102, 103]]
    rows = table.tolist()
    for pool in pools:
        for b, before in enumerate(was):
            want = before + [1000 + 4 * b + i for i in range(4)]
            assert [pool[rows[b][j // page], 0, j % page, 0].item() for j in range(len(want))] == want, b


@pytest.mark.parametrize("clips,cols,pages,page", [(2, 3, 9, 1), (30, 9, 400, 4), (300, 5, 70000, 3), (4500, 3, 20000, 2)])
def test_forks_of_tables_with_pages_ahead_and_pages_gone(clips, cols, pages, page):
    m = rvq()
    g = torch.Generator().manual_seed(clips)
    for turn in range(2):
        announce("fork", clips=clips, cols=cols, pages=pages, page=page, turn=turn)
        lens = torch.randint(0, cols * page + 1, (clips,), generator=g).tolist()
        order, luck = torch.randperm(pages, generator=g).tolist(), torch.rand(clips, cols, generator=g).tolist()
        table = [[order.pop() if luck[b][e] < (0.8 if e * page < lens[b] else 0.4) else (-1, pages, -9)[e % 3]
                  for e in range(cols)] for b in range(clips)]
        refs = counted(table, pages)
        parents = torch.randint(0, clips, (clips,), generator=g).tolist()
        children = torch.randperm(clips, generator=g).tolist()
        pools = [torch.arange(float(pages), device=DEV).view(pages, 1, 1, 1).expand(pages, 1, page, 64).contiguous() + x
                 for x in (0, 0.25)]
        before = [p.clone() for p in pools]
        got = m.rvq_cache_fork(ints(table), ints(lens), ints(refs), ints(parents), ints(children), *pools)
        free, want, copies, missing = [p for p, n in enumerate(refs) if n <= 0], [list(r) for r in table], [], 0
        for p, c in zip(parents, children):
            full, part = divmod(lens[p], page)
            row = table[p][:full] + [-1] * (cols - full)
            if part and 0 <= table[p][full] < pages:
                if free:
                    row[full] = free.pop(0)
                    copies.append((table[p][full], row[full]))
                else:
                    missing += 1
            want[c] = row
        assert got[0].tolist() == want and got[1].tolist() == [lens[parents[children.index(c)]] for c in range(clips)]
        assert got[2].tolist() == counted(want, pages) and got[3].item() == missing
        for pool, old in zip(pools, before):
            for s, t in copies:
                old[t] = old[s]
            assert torch.equal(pool, old)
