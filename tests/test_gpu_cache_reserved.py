"""Upkeep of cache pages on the GPU where a table is not the plainest one: pages reserved ahead, pages that are not
there, no clips at all. Accounts are written out by hand; after every operation a page's count is the number of
table entries that name it."""

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
