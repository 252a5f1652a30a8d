"""A paged cache through many steps of reserve, append, fork, free and compact, in a pool that is often too small: every
clip's pages hold its own frames, shared ones are full, and a page's count is the number of entries that name it."""

import random

import pytest
import torch

from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_cache_reserved import counted, ints

pytestmark = [pytest.mark.gpu, needs_gpu]


class Streams:
    """A cache and, on the host, the frames that each of its clips should find there (a number each)."""

    def __init__(self, clips, cols, pages, page):
        self.m, self.page, self.pages, self.cols = rvq(), page, pages, cols
        self.table, self.lens, self.refs = ints([[-1] * cols] * clips), ints([0] * clips), ints([0] * pages)
        self.pools = [torch.full((pages, 1, page, 64), -1.0, device=DEV) for _ in range(2)]
        self.frames, self.next = [[] for _ in range(clips)], 0

    def reserve(self, ahead):
        new = [len(f) + a for f, a in zip(self.frames, ahead)]
        before = self.table.tolist()
        self.table, self.refs, missing = self.m.rvq_cache_reserve(self.table, self.lens, ints(new), self.refs, self.page)
        after = self.table.tolist()
        wanted = 0
        for b, (old, now) in enumerate(zip(before, after)):
            for e in range(max(self.cols, -(-new[b] // self.page))):
                asked = -(-len(self.frames[b]) // self.page) <= e < -(-new[b] // self.page)
                if e >= self.cols or (asked and now[e] < 0):
                    wanted += asked
                elif not asked or old[e] >= 0:
                    assert now[e] == old[e]
        assert missing.item() == wanted

    def append(self, counts):
        x = self.next + torch.arange(float(sum(counts)), device=DEV)
        rows = torch.stack([x, x + 0.5], 1)[:, :, None].expand(-1, -1, 64).contiguous()
        cu = [0] + torch.tensor(counts).cumsum(0).tolist()
        self.m.rvq_cache_append(rows[:, :1], rows[:, 1:], *self.pools, self.table, self.lens, ints(cu))
        for f, n in zip(self.frames, counts):
            f.extend(range(self.next, self.next + n))
            self.next += n
        self.lens = ints([len(f) for f in self.frames])

    def fork(self, parents, children):
        self.table, self.lens, self.refs, _ = self.m.rvq_cache_fork(self.table, self.lens, self.refs, ints(parents),
                                                                    ints(children), *self.pools)
        old = [list(f) for f in self.frames]
        for p, c in zip(parents, children):
            self.frames[c] = list(old[p])

    def free(self, drop, window, sinks):
        self.table, self.lens, self.refs = self.m.rvq_cache_free(self.table, self.lens, self.refs, self.page, ints(drop),
                                                                 window, sinks)
        self.frames = [[] if d else f for f, d in zip(self.frames, drop)]

    def compact(self):
        self.table, self.refs, live = self.m.rvq_cache_compact(self.table, self.refs, *self.pools)
        assert live.item() == (self.refs > 0).sum() and (self.refs[live.item():] == 0).all()

    def check(self):
        table, refs, page = self.table.tolist(), self.refs.tolist(), self.page
        assert refs == counted(table, self.pages) and self.lens.tolist() == [len(f) for f in self.frames]
        held = [pool[:, 0, :, 63].tolist() for pool in self.pools]
        for row, f in zip(table, self.frames):
            for e, p in enumerate(row):
                if p < 0:
                    continue
                mine = f[e * page:(e + 1) * page]
                assert held[0][p][:len(mine)] == mine and held[1][p][:len(mine)] == [x + 0.5 for x in mine]
                assert refs[p] == 1 or len(mine) == page


@pytest.mark.parametrize("clips,cols,pages,page,seed", [(4, 6, 14, 4, 1), (9, 5, 60, 3, 2), (6, 12, 30, 1, 3), (3, 40, 50, 16, 4),
                                                        (40, 8, 150, 2, 5)])
def test_many_steps(clips, cols, pages, page, seed):
    announce("cache steps", clips=clips, cols=cols, pages=pages, page=page)
    rng, s = random.Random(seed), Streams(clips, cols, pages, page)
    window = rng.choice([2 * page, 3])
    for step in range(80):
        room = [cols * page - len(f) for f in s.frames]
        what = rng.choice(["reserve", "append", "append", "fork", "free", "window", "compact"])
        if what == "reserve":
            s.reserve([rng.choice([0, 1, page, rng.randrange(3 * page)]) for _ in range(clips)])
        elif what == "append":
            counts = [min(r, rng.choice([0, 1, 1, rng.randrange(2 * page + 1)])) for r in room]
            s.reserve(counts)
            s.append(counts)
        elif what == "fork":
            children = rng.sample(range(clips), rng.randint(1, clips))
            s.fork([rng.randrange(clips) for _ in children], children)
        elif what == "compact":
            s.compact()
        else:
            s.free([int(rng.random() < 0.25) for _ in range(clips)], window if what == "window" else None, 1)
        s.check()
