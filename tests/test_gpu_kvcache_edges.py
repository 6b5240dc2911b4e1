"""Edges of the cache's operators: page numbers, lengths, windows, scales and terms at the ends of their ranges."""
import math

import pytest
import torch

from means_clustering_amd import kvcache

from .test_gpu_kvcache import BF, DEV, E, FP, U, Case

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------------ tables ----

@pytest.mark.parametrize("p", [16, 64, 1 << 20])
def test_tables_pages_that_no_cache_can_have(p):
    """A page of 2^31 / page_size or more has no slot: its first slots would wrap to those of page 0."""
    last = 2 ** 31 // p - 1
    pages = [last, last + 1, 2 * last + 2, 2 ** 31 - 1, 2, -5]
    pages = [min(x, 2 ** 31 - 1) for x in pages]
    want = [x * p + 3 if 0 <= x <= last else -1 for x in pages]
    R = len(pages)
    # held pages, read from the table
    t = kvcache.tables(_i32([3] * R), _i32([1] * R), _i32(pages).view(R, 1), _i32([0]), p, R)
    assert t.slots.tolist() == want
    # new pages, from the free list
    table = torch.full((R, 1), -7, dtype=torch.int32, device=DEV)
    t = kvcache.tables(_i32([0] * R), _i32([4] * R), table, _i32(pages), p, 4 * R)
    assert t.slots.tolist()[3::4] == want
    assert table.view(-1).tolist() == pages
    # and nothing is appended for them
    if p == 16:
        cache = torch.zeros(4, p, 1, 16, dtype=BF, device=DEV)
        kvcache.append(None, torch.ones(4 * R, 1, 16, dtype=BF, device=DEV), None, cache, None, t.slots)
        assert bool((cache[2, :4] == 1).all()) and float(cache.float().sum()) == 4 * 16


# ------------------------------------------------------------------------------------------------------ attend ----

def _check(c, **changes):
    """The call against Case.reference, its tolerances and its rule for rows that see nothing."""
    out, lse = kvcache.attend(**dict(c.device(), **changes), lse=True)
    torch.cuda.synchronize()
    ro, rl, to, tl = c.reference()
    got, gl = out.double().cpu(), lse.double().cpu()
    assert bool(((got - ro).abs() <= to).all()), ((got - ro).abs() - to).max()
    empty = rl == -math.inf
    assert bool((gl[empty] == -math.inf).all()) and bool((got[empty] == 0).all())
    assert bool(((gl[~empty] - rl[~empty]).abs() <= tl[~empty]).all())


@pytest.mark.parametrize("n", [1, 12, 60])
@pytest.mark.parametrize("window", [63, 64, 65, 80, 100, 5000, 2 ** 31 - 1])
def test_attend_window_over_a_row_shorter_than_its_request(n, window):
    """100 slots, of which the table row holds 64: the last query stands at slot 99 and sees those after 99 - window."""
    c = Case([(100, n), (70, 1)], 4, 2, 64, BF, window=window)
    c.table[:, 4:] = -1
    print(f"[attend] n={n} window={window}", flush=True)
    _check(c, block_table=c.table[:, :4].contiguous().to(DEV))
