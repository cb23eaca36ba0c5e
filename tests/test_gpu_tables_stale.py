"""Tables on the device whose manager has changed under them are refused: their list of free blocks is a copy."""
import numpy as np
import pytest
import torch

from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300.engine import DeviceTables, PagedKVCache

pytestmark = pytest.mark.gpu


def made(nb=40, **kw):
    cache = PagedKVCache(pkv.make_desc("f16", 1, nb, 4, 2, 64))
    for x, n in ((1, 20), (2, 16), (3, 0)):
        cache.add_sequence(x, n)
    return cache, DeviceTables(cache, [1, 2, 3], 8, **kw)


@pytest.mark.parametrize("change", [
    lambda c: c.add_sequence(9, 5), lambda c: c.fork(1, 9), lambda c: c.mgr.free_seq(2), lambda c: c.mgr.append_slot(3),
    lambda c: c.mgr.extend(1, 40)])
@pytest.mark.parametrize("steps", [0, 2])
def test_a_manager_that_changed_makes_tables_stale(change, steps):
    cache, tables = made()
    for _ in range(steps):
        tables.extend()
        assert tables.follow() == 3
    change(cache)
    was = [x.clone() for x in (tables.tables, tables.lens, tables.slots, tables.totals)]
    with pytest.raises(ValueError, match="stale"):
        tables.extend()
    with pytest.raises(ValueError, match="stale"):
        tables.follow()
    for x, y in zip(was, (tables.tables, tables.lens, tables.slots, tables.totals)):
        assert torch.equal(x, y)


def test_blocks_that_moved_in_the_free_list_are_found_by_follow():
    """Added and freed again: as many free blocks as before, in another order."""
    cache, tables = made()
    cache.add_sequence(9, 64)
    cache.mgr.free_seq(9)
    tables.extend()
    with pytest.raises(ValueError, match="blocks"):
        tables.follow()


def test_blocks_that_others_free_are_not_seen():
    """A sequence beside the batch ends, or a row whose blocks are full is forked: the tables go on, with the blocks they know."""
    cache, _ = made(nb=9)
    cache.add_sequence(9, 60)                          # 2 + 1 + 0 + 4 blocks of 9
    tables = DeviceTables(cache, [1, 2, 3], 8, max_tokens=100)
    cache.mgr.free_seq(9)
    for counts, served in (([13, 0, 2], 3), ([0, 1, 0], 1), ([0, 0, 14], 3), ([0, 0, 1], 2)):
        tables.extend(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        assert tables.totals[1].item() == served == tables.follow(counts)
        rc, host, lens = cache.mgr.pack_tables([1, 2, 3], 8)
        assert np.array_equal(tables.tables.cpu().numpy(), host) and np.array_equal(tables.lens.cpu().numpy(), lens)
    cache.fork(2, 10)                                  # 16 tokens: a whole block
    tables.extend(torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"))
    assert tables.follow([1, 0, 0]) == 3
    cache.fork(1, 11)                                  # 34 tokens
    with pytest.raises(ValueError, match="stale"):
        tables.extend()


def test_rows_that_do_not_fit_leave_the_tables_usable():
    cache, tables = made(nb=6, max_tokens=100)
    counts = [[1, 1, 1], [20, 20, 20], [3, 1, 2]]
    for c in counts:
        tables.extend(torch.tensor(c, dtype=torch.int32, device="cuda"))
        assert tables.follow(c) == tables.totals[1].item()
        rc, host, lens = cache.mgr.pack_tables([1, 2, 3], 8)
        assert np.array_equal(tables.tables.cpu().numpy(), host) and np.array_equal(tables.lens.cpu().numpy(), lens)


def test_several_steps_ahead():
    cache, tables = made()
    for _ in range(20):
        tables.extend()
    for _ in range(20):
        assert tables.follow() == 3
    rc, host, lens = cache.mgr.pack_tables([1, 2, 3], 8)
    assert np.array_equal(tables.tables.cpu().numpy(), host) and list(lens) == [40, 36, 20]
