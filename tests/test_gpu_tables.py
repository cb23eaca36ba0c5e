"""Tables, slots and lengths built on the GPU, against the host block manager row after row."""
import numpy as np
import pytest
import torch

from paged_kv_cache_258_gb300 import pkv

pytestmark = pytest.mark.gpu
BLOCK = 16


def up(x):
    return -(-int(x) // BLOCK)


def expect(nb, free, used, tables, lens, new, max_tokens):
    """Row after row and token after token."""
    tables, lens = tables.copy(), lens.copy()
    mb = tables.shape[1]
    start, slots, served, is_open = [0], [], 0, True
    for i, m in enumerate(new):
        if lens[i] < 0 or lens[i] > mb * BLOCK or m < 0:
            m = 0
        need = up(lens[i] + m) - up(lens[i])
        fits = used + need <= len(free) and len(slots) + m <= max_tokens and up(lens[i] + m) <= mb
        is_open = is_open and (fits or m == 0)
        if is_open:
            served += 1
            for p in range(lens[i], lens[i] + m):
                if p % BLOCK == 0:
                    tables[i, p // BLOCK] = free[used]
                    used += 1
                b = tables[i, p // BLOCK]
                slots.append(b * BLOCK + p % BLOCK if 0 <= b < nb else -1)
            lens[i] += m
        start.append(len(slots))
    return tables, slots + [-1] * (max_tokens - len(slots)), start, lens, [used, served, start[-1]]


def run(nb, free, used, tables, lens, new, max_tokens, in_place=False):
    dev = lambda x, t=torch.int32: torch.tensor(np.asarray(x), dtype=t, device="cuda")
    tt, tl = dev(tables).reshape(tables.shape), dev(lens)
    totals = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    tu = totals[:1] if in_place else dev([used])
    tu.fill_(used)
    out = tl if in_place else torch.full_like(tl, -9)
    slots = torch.full((max_tokens + 1,), -5, dtype=torch.int64, device="cuda")
    start = torch.full((len(lens) + 1,), -3, dtype=torch.int32, device="cuda")
    pkv.pkv_extend_tables(nb, dev(free), tu, tt, tl, None if new is None else dev(new), slots[:max_tokens], start, out, totals)
    assert slots[-1].item() == -5
    return [x.cpu().numpy() for x in (tt, slots[:-1], start, out, totals)]


def case(n, lo, hi, new_lo, new_hi, seed, spare=3, share=1.0, width=2):
    rng = np.random.default_rng(seed)
    lens = rng.integers(lo, hi + 1, n).astype(np.int64)
    new = rng.integers(new_lo, new_hi + 1, n).astype(np.int64)
    held = -(-lens // BLOCK)
    need = -(-(lens + new) // BLOCK) - held
    mb = max(int((held + need).max(initial=0)) + width, 1)
    n_free = int(need.sum() * share)
    nb = int(held.sum()) + n_free + spare
    ids = rng.permutation(nb)
    tables, at = np.full((n, mb), -1, dtype=np.int64), 0
    for i, b in enumerate(held):
        tables[i, :b] = ids[at:at + b]
        at += b
    return nb, ids[at:at + n_free + spare], spare, tables, lens, new


def same(got, want):
    for g, w, name in zip(got, want, ("tables", "slots", "start", "lens", "totals")):
        assert np.array_equal(g, np.asarray(w)), name


@pytest.mark.parametrize("n,lo,hi,new_lo,new_hi", [
    (1, 0, 0, 1, 1), (1, 15, 15, 1, 1), (1, 16, 16, 1, 1), (1, 17, 17, 0, 0), (3, 0, 40, 0, 5), (64, 0, 300, 1, 1),
    (33, 0, 100, 0, 40), (1, 0, 0, 5000, 5000), (2, 7, 7, 4099, 4111), (1000, 0, 0, 0, 70), (1023, 0, 50, 0, 3),
    (1025, 0, 50, 0, 9), (2500, 0, 33, 0, 4), (5000, 0, 20, 1, 1),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches(n, lo, hi, new_lo, new_hi, in_place):
    c = case(n, lo, hi, new_lo, new_hi, seed=n + hi)
    most = int(c[5].sum()) + 5
    same(run(*c, most, in_place=in_place), expect(*c, most))
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("n,share,short,width", [(50, 0.5, 0, 1), (50, 1.0, 31, 1), (3000, 0.6, 0, 1), (3000, 1.0, 900, 1),
                                                 (40, 1.0, 0, -1), (2100, 1.0, 0, -1), (40, 0.0, 0, 1)])
def test_rows_that_do_not_fit(n, share, short, width):
    """Too few blocks, places for tokens, or table entries: rows up to the first that does not fit are served."""
    c = case(n, 0, 60, 0, 30, seed=n, share=share, width=width)
    most = int(c[5].sum()) - short
    got, want = run(*c, most), expect(*c, most)
    same(got, want)
    assert want[4][1] < n  # (a first row that does not fit leaves none)
    assert pkv.pkv_get_device_status() == 0


def test_one_token_each_by_default():
    c = case(70, 0, 90, 1, 1, seed=5)
    same(run(*c[:5], None, 70), expect(*c, 70))


def test_nothing_to_do():
    t = np.zeros((0, 4), dtype=np.int64)
    same(run(9, [1, 2], 1, t, np.zeros(0, dtype=np.int64), np.zeros(0, dtype=np.int64), 3), (t, [-1] * 3, [0], [], [1, 0, 0]))
    c = case(4, 3, 30, 0, 0, seed=1)
    same(run(*c, 0), expect(*c, 0))


def test_bad_values_are_skipped_and_flagged():
    nb, free, used, tables, lens, new = case(12, 5, 60, 1, 30, seed=3)
    lens[2], lens[3], new[5] = -4, tables.shape[1] * BLOCK + 1, -2
    most = int(new.clip(0).sum())
    same(run(nb, free, used, tables, lens, new, most), expect(nb, free, used, tables, lens, new, most))
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_CONTEXT_LEN | pkv.PKV_DEV_BAD_QUERY_RANGE
    c = list(case(12, 5, 60, 20, 30, seed=4))
    c[1] = c[1].copy()
    c[1][c[2] + 3] = nb + 1000                          # a fresh id that is not in the pool
    same(run(*c, 400), expect(*c, 400))
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_FREE_LIST
    c = list(case(3, 5, 5, 2, 2, seed=4))
    c[3] = c[3].copy()
    c[3][1, 0] = -8                                     # an old one
    same(run(*c, 6), expect(*c, 6))
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_BLOCK_ID
    for bad in (-1, 1000):
        c = list(case(3, 5, 5, 2, 2, seed=4))
        got = run(c[0], c[1], bad, *c[3:], 6)
        assert got[4].tolist() == [bad, 3, 6]           # no new block is needed
        c = list(case(3, 5, 5, 20, 20, seed=4))
        got = run(c[0], c[1], bad, *c[3:], 60)
        assert got[4].tolist() == [bad, 0, 0] and (got[1] == -1).all()
        assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_FREE_LIST


def test_huge_counts_saturate():
    """Sums past 32 bits: a row of 2^31 - 1 tokens, and rows behind it."""
    nb, free, used, tables, lens, new = case(8, 0, 9, 1, 3, seed=9)
    for i in (3, 4, 6):
        new[i] = 2 ** 31 - 1
    got = run(nb, free, used, tables, lens, new, 50)
    same(got, expect(nb, free, used, tables, lens, np.array([*new[:3], 10 ** 6, *[0] * 4]), 50))
    assert got[4][1] == 3 and pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("n", [5, 60])
def test_the_block_manager_gives_the_same(n):
    """Steps of the device and of the manager side by side, from the manager's free list."""
    rng = np.random.default_rng(n)
    nb = 40 * n
    mgr = pkv.BlockManager(nb, free_order=rng.permutation(nb).astype(np.int32))
    lens = rng.integers(1, 100, n)
    for i, c in enumerate(lens):
        mgr.add_seq(i, int(c))
    ids, mb = np.arange(n, dtype=np.int64), 40
    rc, tables, lens = mgr.pack_tables(ids, mb)
    tt, tl = torch.from_numpy(tables.copy()).cuda(), torch.from_numpy(lens.copy()).cuda()
    free = torch.tensor(mgr.free_list(), dtype=torch.int32, device="cuda")
    totals = torch.zeros(3, dtype=torch.int32, device="cuda")
    start = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    for step in range(6):
        new = rng.integers(0, 60, n).astype(np.int32)
        slots = torch.empty(int(new.sum()) + 2, dtype=torch.int64, device="cuda")
        pkv.pkv_extend_tables(nb, free, totals[:1], tt, tl, torch.from_numpy(new).cuda(), slots, start, tl, totals)
        want = []
        for i in range(n):
            rc, s, _, _ = mgr.extend(i, int(new[i]))
            assert rc == pkv.PKV_OK
            want.extend(s.tolist())
        rc, tables, lens = mgr.pack_tables(ids, mb)
        assert np.array_equal(tt.cpu().numpy(), tables) and np.array_equal(tl.cpu().numpy(), lens)
        assert slots.tolist() == want + [-1, -1] and totals[1].item() == n


def test_replayed_from_a_graph():
    """A captured step, replayed: lengths, tables and the count of blocks go on from replay to replay."""
    c = case(20, 0, 50, 1, 1, seed=8)
    n, mb = c[3].shape
    free = np.random.default_rng(0).permutation(500)
    tables = np.concatenate([c[3], np.full((n, 10), -1)], 1)
    tt, tl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (tables, c[4]))
    tf = torch.tensor(free, dtype=torch.int32, device="cuda")
    totals = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    start = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_extend_tables(500, tf, totals[:1], tt, tl, None, slots, start, tl, totals)
    want = (tables, None, None, c[4], [0])
    for _ in range(40):
        graph.replay()
        want = expect(500, free, want[4][0], want[0], want[3], np.ones(n, dtype=np.int64), n)
        same([x.cpu().numpy() for x in (tt, slots, start, tl, totals)], want)


def test_calls_behind_one_another():
    """Many tokens a call, lengths and the count of blocks in place, without waiting between the calls: what a call's
    launches read must still be there although the next ones write it."""
    n, steps = 300, 6
    rng = np.random.default_rng(9)
    tables = np.full((n, 30), -1, dtype=np.int64)
    free = rng.permutation(n * 20)
    new = [rng.integers(20, 70, n) for _ in range(steps)]
    most = 70 * n
    tt = torch.tensor(tables, dtype=torch.int32, device="cuda")
    tf = torch.tensor(free, dtype=torch.int32, device="cuda")
    tn = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in new]
    tl, totals = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (n, 3))
    slots = [torch.empty(most, dtype=torch.int64, device="cuda") for _ in range(steps)]
    start = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    launches = [pkv.extend_tables_launcher(n * 20, tf, totals[:1], tt, tl, x, s, start, tl, totals) for x, s in zip(tn, slots)]
    for launch in launches:
        launch()
    want = (tables, None, None, np.zeros(n, dtype=np.int64), [0])
    for x, s in zip(new, slots):
        want = expect(n * 20, free, want[4][0], want[0], want[3], x, most)
        assert np.array_equal(s.cpu().numpy(), np.asarray(want[1]))
    same([x.cpu().numpy() for x in (tt, slots[-1], start, tl, totals)], want)
    assert pkv.pkv_get_device_status() == 0
