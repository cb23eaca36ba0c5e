"""The cache-shrinking calls together, as a serving loop uses them: prompts by chunked prefill, scored decode
steps with prefix sharing and copy-on-write, eviction, more steps -- over 8-bit and 16-bit caches. Host
mirrors of the pools follow every step through 64-bit restatements and the slots and tables that the block
manager gave."""
import numpy as np
import pytest
import torch

import shrink_oracle as R
from helpers import NP_STORAGE, as_f64, to_host, to_torch
from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300 import workloads as W
from paged_kv_cache_258_gb300.engine import DecodeBatch, PagedKVCache, PrefillStep, StepExecutor
from paged_kv_cache_258_gb300.scheduler import Request, Scheduler, serve
from test_scheduler import MirroredManager, VirtualClock

pytestmark = pytest.mark.gpu


class Mirror:
    """The pools on the host: codes and scales, or rows of the storage type; advanced by the restatements."""

    def __init__(self, desc, dtype, q8):
        self.dtype, self.q8 = dtype, q8
        shape = pkv.pool_shape(desc)
        self.pools = [np.zeros(shape, np.uint8 if q8 else NP_STORAGE[dtype]) for _ in range(2)]
        self.scales = [np.zeros(shape[:3], np.float32) for _ in range(2)] if q8 else None

    def copy(self, pairs):
        for src, dst in pairs:
            for a in self.pools + (self.scales or []):
                a[:, dst] = a[:, src]

    def append(self, rows, slots):
        """rows: (k, v) storage arrays [L, n_tok, n_kv, d]"""
        for i, x in enumerate(rows):
            for layer in range(x.shape[0]):
                if self.q8:
                    f = as_f64(to_torch(x[layer], self.dtype, device="cpu"))
                    R.append(f, slots, self.pools[i][layer], self.scales[i][layer], self.dtype)
                else:
                    for t, slot in enumerate(slots):
                        self.pools[i][layer, slot // 16, :, slot % 16] = x[layer, t]

    def wide(self, layer):
        if self.q8:
            return [R.widen(p[layer], s[layer]) for p, s in zip(self.pools, self.scales)]
        return [as_f64(to_torch(p[layer], self.dtype, device="cpu")) for p in self.pools]

    def check(self, cache, tables, lens):
        """Every referenced row of the device pools equals the mirror's, bit for bit."""
        dev = [cache.k_pool, cache.v_pool]
        for i in range(2):
            got = dev[i].view(torch.uint8).cpu().numpy() if self.q8 else to_host(dev[i], self.dtype)
            for s, c in enumerate(lens):
                for j in range(int(c)):
                    b = tables[s, j // 16]
                    assert np.array_equal(got[:, b, :, j % 16], self.pools[i][:, b, :, j % 16]), (i, s, j)
            if self.q8:
                sc = [cache.k_scales, cache.v_scales][i].cpu().numpy()
                used = np.unique(np.concatenate([tables[s, :-(-int(c) // 16)] for s, c in enumerate(lens)]))
                assert np.array_equal(sc[:, used], self.scales[i][:, used])


def io(rng, L, n, n_q, n_kv, d, dtype):
    q = W.normal_values(rng, (L, n, n_q, d), dtype)
    k, v = (W.normal_values(rng, (L, n, n_kv, d), dtype) for _ in range(2))
    out = torch.full((L, n, n_q, d), float("nan"), dtype=pkv.torch_dtype(dtype), device="cuda")
    return q, k, v, out


@pytest.mark.parametrize("dtype,q8,n_q,n_kv,d", [("bf16", True, 4, 2, 64), ("f16", True, 8, 1, 128), ("f16", False, 4, 2, 64),
                                                 ("bf16", False, 4, 4, 128)])
def test_serving_with_eviction(dtype, q8, n_q, n_kv, d):
    rng = np.random.default_rng(5)
    L, nb, mb = 2, 120, 24
    desc = pkv.make_desc(dtype, L, nb, n_q, n_kv, d)
    cache = PagedKVCache(desc, free_order=W.free_order(nb, 3), storage="q8" if q8 else None)
    assert cache.kv_bytes_per_token_layer() == 2 * n_kv * d * (1 if q8 else 2)
    mirror = Mirror(desc, dtype, q8)
    scale = 1 / np.sqrt(d)
    p_step = 2.0 ** -11 if q8 else R.HALF_STEP[dtype]

    def check_rows(got, q, tables, lens, half):
        w = np.zeros((L, len(lens), n_kv, mb * 16))
        for layer in range(L):
            k, v = mirror.wide(layer)
            want, tol, w[layer], w_tol = R.decode(as_f64(to_torch(q[layer], dtype, device="cpu")), k, v, tables, lens, scale,
                                                  dtype, half)
            assert np.all(np.abs(got[layer] - want) <= 2 * tol)
        return w

    # prompts: two chunks for one of them, then a child that shares a partly filled block
    pre = PrefillStep(cache, max_tokens=160, max_seqs=3, max_blocks=mb)
    for chunks in ([(1, 90, True), (2, 37, True)], [(1, 71, False), (3, 5, True)]):
        T = sum(c[1] for c in chunks)
        q, k, v, out = io(rng, L, T, n_q, n_kv, d, dtype)
        st = pre.step(chunks, to_torch(q, dtype), to_torch(k, dtype), to_torch(v, dtype), out, scale)
        slots = st["np"][: 2 * pre.max_tokens].view(np.int64)[:T].copy()
        torch.cuda.synchronize()
        mirror.append((k, v), slots)
        _, tables, lens = cache.mgr.pack_tables([c[0] for c in chunks], mb)
        got = as_f64(out)
        row = 0
        for i, (_, n, _) in enumerate(chunks):
            for t in range(n):
                p = int(lens[i]) - n + t
                check_rows(got[:, row + t:row + t + 1], q[:, row + t:row + t + 1], tables[i:i + 1], np.array([p + 1]),
                           R.HALF_STEP[dtype])
            row += n
    cache.fork(1, 4)
    ids = [1, 2, 3, 4]
    batch = DecodeBatch(cache, ids, max_blocks=mb, scored=True)
    sums = np.zeros((L, 4, n_kv, mb * 16))

    def steps(count):
        nonlocal sums
        for _ in range(count):
            q, k, v, out = io(rng, L, 4, n_q, n_kv, d, dtype)
            st = batch.step(to_torch(q, dtype), to_torch(k, dtype), to_torch(v, dtype), out, scale)
            torch.cuda.synchronize()
            mirror.copy(st["pairs"].numpy()[: st["npairs"]].tolist())
            mirror.append((k, v), st["slots"].numpy())
            tables, lens = st["tables"].numpy(), st["lens"].numpy()
            sums += check_rows(as_f64(out), q, tables, lens, p_step)
        mirror.check(cache, tables, lens)
        # per step and head a weight is off by less than 2^-12 of itself (a logit by 2^-13); see decode()
        assert np.allclose(batch.scores.double().cpu().numpy(), sums, rtol=2.0 ** -11, atol=1e-7)

    def evict(keep, recent):
        nonlocal sums
        _, src, lens = cache.mgr.pack_tables(batch.seq_ids, mb)
        scores = batch.scores.cpu().numpy()
        kept = batch.evict(keep, recent)
        _, dst, new_lens = cache.mgr.pack_tables(batch.seq_ids, mb)
        torch.cuda.synchronize()
        keep = np.broadcast_to(keep, (4,))
        assert np.array_equal(new_lens, np.minimum(keep, lens))
        want_kept = np.full(tuple(kept.shape), -1, dtype=np.int32)
        new = scores.copy()
        R.evict(mirror.pools, mirror.scales, src, dst, lens, keep, recent, scores, new, want_kept)
        assert np.array_equal(kept.cpu().numpy(), want_kept)
        assert np.array_equal(batch.scores.cpu().numpy(), new)
        sums = new.astype(np.float64)
        mirror.check(cache, dst, new_lens)

    steps(3)
    evict(60, 8)                       # sequences 1 and 4 share ten blocks: both get rows of their own
    assert not set(cache.mgr.block_table(1)[1]) & set(cache.mgr.block_table(4)[1])
    steps(14)
    batch.set_sequences([4, 2, 3, 1])  # sums follow their sequences
    sums = sums[:, [3, 1, 2, 0]]
    steps(2)
    evict([20, 31, 1000, 1], 4)        # one untouched, one down to a single position
    steps(3)
    assert batch.total_cow >= 1
    assert pkv.pkv_get_device_status() == 0
    # a sequence outside the batch that shares a member's blocks keeps its rows
    cache.fork(2, 9)
    _, t9, l9 = cache.mgr.pack_tables([9], mb)
    before = [np.stack([p[:, t9[0, j // 16], :, j % 16] for j in range(l9[0])]) for p in mirror.pools]
    evict(10, 3)
    after = [np.stack([p[:, t9[0, j // 16], :, j % 16] for j in range(l9[0])]) for p in mirror.pools]
    assert all(np.array_equal(a, b) for a, b in zip(before, after))
    _, t9b, l9b = cache.mgr.pack_tables([9], mb)
    assert np.array_equal(t9, t9b) and np.array_equal(l9, l9b)
    mirror.check(cache, t9b, l9b)


def test_evict_refusals():
    desc = pkv.make_desc("bf16", 1, 4, 2, 1, 64)
    cache = PagedKVCache(desc, storage="q8")
    cache.add_sequence(1, 64)
    with pytest.raises(ValueError, match="scored"):
        DecodeBatch(cache, [1], max_blocks=4).evict(10, 2)
    batch = DecodeBatch(cache, [1], max_blocks=4, scored=True)
    with pytest.raises(ValueError):
        batch.evict(-1, 2)
    with pytest.raises(ValueError):
        batch.evict(4, -2)
    cache.fork(1, 2)                   # every block is shared and none is free
    before = cache.mgr.save()
    with pytest.raises(pkv.PkvError, match="NO_BLOCKS"):
        batch.evict(10, 2)
    assert cache.mgr.block_table(1) == cache.mgr.block_table(2) and cache.mgr.stats()["alloc_failures"] == 1
    assert len(before) == len(cache.mgr.save())
    twice = DecodeBatch(cache, [2, 2], max_blocks=4, scored=True)
    with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
        twice.evict(10, 2)
    with pytest.raises(ValueError):
        PagedKVCache(pkv.make_desc("f32", 1, 4, 2, 1, 64), storage="q8")
    with pytest.raises(ValueError):
        PagedKVCache(desc, storage="q4")
    f32 = PagedKVCache(pkv.make_desc("f32", 1, 4, 2, 1, 64))
    with pytest.raises(ValueError, match="scored"):
        DecodeBatch(f32, [1], max_blocks=4, scored=True)


@pytest.mark.parametrize("overlap", [True, False])
def test_continuous_batching_over_an_8_bit_cache(overlap):
    """The scheduler's iterations through StepExecutor on an 8-bit cache: chunks, decodes, shared prefixes."""
    dtype, L, n_q, n_kv, d, nb, mb = "bf16", 2, 4, 2, 64, 70, 30
    rng = np.random.default_rng(9)
    order = W.free_order(nb, 7)
    desc = pkv.make_desc(dtype, L, nb, n_q, n_kv, d)
    cache = PagedKVCache(desc, free_order=order, storage="q8")
    mm = MirroredManager(nb, order)
    cache.mgr = mm.c
    sched = Scheduler(mm, max_batch_tokens=64, chunk=32, max_running=6, max_blocks=mb)
    sched.add_prefix(3, 21)
    reqs = [Request(rid=i, klass="a", prompt=int(rng.integers(25, 90)), response=int(rng.integers(2, 12)),
                    arrival=float(i), priority=0, prefix=3 if i % 2 else None) for i in range(6)]
    ex = StepExecutor(cache, max_decode=6, max_tokens=64, max_chunks=8, max_blocks=mb)
    ex.overlap = overlap
    mirror = Mirror(desc, dtype, True)
    scale = 1 / np.sqrt(d)
    clock = VirtualClock()
    seen = {"dec": 0, "pre": 0, "pairs": 0}

    def rows(ids):
        _, tables, lens = mm.c.pack_tables(ids, mb)
        return tables, lens

    def execute(plan):
        nd, nt = plan.n_dec, plan.n_pre_tokens
        dq, dk, dv, d_out = io(rng, L, max(nd, 1), n_q, n_kv, d, dtype)
        pq, pk, pv, p_out = io(rng, L, max(nt, 1), n_q, n_kv, d, dtype)
        ex.run(plan, tuple(to_torch(x, dtype)[:, :nd] for x in (dq, dk, dv)) + (d_out[:, :nd],),
               tuple(to_torch(x, dtype)[:, :nt] for x in (pq, pk, pv)) + (p_out[:, :nt],), scale)
        torch.cuda.synchronize()
        mirror.copy(plan.pairs.tolist() if len(plan.pairs) else [])
        if nt:
            mirror.append((pk[:, :nt], pv[:, :nt]), plan.pre_slots)
        if nd:
            mirror.append((dk[:, :nd], dv[:, :nd]), plan.dec_slots)
        got_d, got_p = as_f64(d_out), as_f64(p_out)
        for layer in range(L):
            k, v = mirror.wide(layer)
            if nd:
                tables, lens = rows([int(s) for s in plan.dec_seq])
                want, tol, _, _ = R.decode(as_f64(to_torch(dq[layer, :nd], dtype, device="cpu")), k, v, tables, lens, scale,
                                           dtype, 2.0 ** -11)
                assert np.all(np.abs(got_d[layer, :nd] - want) <= tol)
            at = 0
            for o, n in plan.pre_chunks:
                tables, lens = rows([int(o.seq)])
                for t in (0, n - 1):
                    qf = as_f64(to_torch(pq[layer, at + t:at + t + 1], dtype, device="cpu"))
                    want, tol, _, _ = R.decode(qf, k, v, tables, np.array([int(lens[0]) - n + t + 1]), scale, dtype,
                                               R.HALF_STEP[dtype])
                    assert np.all(np.abs(got_p[layer, at + t] - want[0]) <= 2 * tol)
                at += n
        seen["dec"] += nd
        seen["pre"] += nt
        seen["pairs"] += len(plan.pairs)
        clock.t += 1.0

    serve(sched, reqs, execute, clock, clock.wait_until)
    assert all(r.state == "done" for r in reqs)
    assert seen["dec"] > 0 and seen["pre"] > 0 and seen["pairs"] > 0
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("dtype,q8,scored", [("bf16", True, True), ("f16", True, False), ("f16", False, True)])
def test_launchers_equal_the_calls(dtype, q8, scored):
    """A step's launchers over views of larger buffers against the call for each layer, bit for bit."""
    L, n, n_q, n_kv, d, nb, mb = 3, 3, 8, 2, 128, 40, 9
    desc = pkv.make_desc(dtype, L, nb, n_q, n_kv, d)
    rng = np.random.default_rng(21)
    got = []
    big = [to_torch(x, dtype) for x in io(rng, L, n + 2, n_q, n_kv, d, dtype)[:3]]
    rows = [to_torch(x, dtype) for x in io(rng, L, 90, n_q, n_kv, d, dtype)[:3]]
    q, k, v = (x[:, 1:n + 1] for x in big)
    for launchers in (False, True):
        cache = PagedKVCache(desc, storage="q8" if q8 else None)
        slots = torch.from_numpy(np.concatenate([cache.add_sequence(i, c) for i, c in enumerate((60, 29, 1))])).cuda()
        _, tables, lens = cache.mgr.pack_tables([0, 1, 2], mb)
        tables, lens = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
        starts = torch.tensor([0, 60, 89, 90], dtype=torch.int32, device="cuda")
        last = slots[torch.tensor([59, 88, 89], device="cuda")]
        out = torch.zeros((L, n + 1, n_q, d), device="cuda", dtype=pkv.torch_dtype(dtype))[:, :n]
        p_out = torch.zeros((L, 90, n_q, d), device="cuda", dtype=pkv.torch_dtype(dtype))
        scores = torch.zeros((L, n, n_kv, mb * 16 + 1), device="cuda") if scored else None
        ws = cache.decode_workspace(n, mb, scored)
        p_ws = pkv.alloc_q8_prefill_workspace(desc) if q8 else None
        if launchers:
            fill = cache.append_launcher(rows[1], rows[2], slots)
            append = cache.append_launcher(k, v, last)
            decode = cache.decode_launcher(q, tables, lens, 0.1, out, ws, scores)
            prefill = pkv.q8_prefill_launcher(desc, rows[0], *cache._arrays(), tables, lens, starts, 60, 0.1, p_out,
                                              p_ws) if q8 else None
        for layer in range(L):
            if launchers:
                fill(layer), append(layer), decode(layer)
                if q8:
                    prefill(layer)
            else:
                cache.append(layer, rows[1][layer], rows[2][layer], slots)
                cache.append(layer, k[layer], v[layer], last)
                cache.decode(layer, q[layer], tables, lens, 0.1, out[layer], ws, None if scores is None else scores[layer])
                if q8:
                    pkv.pkv_q8_prefill_attention(desc, layer, rows[0][layer], *cache._arrays(), tables, lens, starts, 60, 0.1,
                                                 p_out[layer], p_ws)
        assert pkv.pkv_get_device_status() == 0
        got.append([x.contiguous().view(torch.uint8).cpu() for x in (*cache._arrays(), out, p_out, *([scores] if scored else []))])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][-1].any()
    with pytest.raises(ValueError):
        cache.decode_launcher(q[:2], tables, lens, 0.1, out, ws, scores)
    with pytest.raises(ValueError):
        cache.append_launcher(k[:, :, :1], v, last)
    with pytest.raises(ValueError):
        cache.decode_launcher(q, tables, lens, 0.1, out, ws, torch.zeros((L, n, n_kv, 16), device="cuda"))
    if not q8:
        with pytest.raises(ValueError, match="scores"):
            cache.decode_launcher(q, tables, lens, 0.1, out, ws)


@pytest.mark.parametrize("q8", [True, False])
def test_steps_reuse_their_buffers(q8):
    """Steps into the same tensors (checked once) equal steps into new ones, also behind a change of scores."""
    L, n, n_q, n_kv, d = 2, 3, 4, 2, 64
    desc = pkv.make_desc("bf16", L, 60, n_q, n_kv, d)
    got = []
    for reuse in (True, False):
        rng = np.random.default_rng(31)
        cache = PagedKVCache(desc, storage="q8" if q8 else None)
        for i in range(n):
            cache.add_sequence(i, 20 + i)
        batch = DecodeBatch(cache, range(n), max_blocks=8, scored=True)
        keep = [to_torch(x, "bf16") for x in io(rng, L, n, n_q, n_kv, d, "bf16")[:3]]
        out = torch.zeros_like(keep[0])
        outs = []
        for step in range(7):
            fresh = [to_torch(x, "bf16") for x in io(rng, L, n, n_q, n_kv, d, "bf16")[:3]]
            if reuse:
                for a, b in zip(keep, fresh):
                    a.copy_(b)
            if step == 4:
                batch.scores = batch.scores.clone()
            batch.step(*(keep if reuse else fresh), out if reuse else (out := torch.zeros_like(out)), 0.125)
            outs.append(out.clone())
        got.append(outs + [batch.scores, *cache._arrays()])
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(*got))
    assert pkv.pkv_get_device_status() == 0


def test_evict_on_a_stream_of_its_own(monkeypatch):
    """A batch on a side stream whose first eviction comes while the current stream is busy: what the eviction
    needs is allocated on the batch's stream, and its codes and scores are those of the restatement."""
    dtype, L, n, n_q, n_kv, d, nb, mb = "bf16", 2, 3, 4, 2, 64, 64, 16
    rng = np.random.default_rng(41)
    desc = pkv.make_desc(dtype, L, nb, n_q, n_kv, d)
    cache = PagedKVCache(desc, storage="q8")
    mirror = Mirror(desc, dtype, True)
    slots = np.concatenate([cache.add_sequence(i, c) for i, c in enumerate((200, 77, 31))])
    _, k, v, _ = io(rng, L, len(slots), n_q, n_kv, d, dtype)
    for layer in range(L):
        cache.append(layer, to_torch(k[layer], dtype), to_torch(v[layer], dtype), torch.from_numpy(slots).cuda())
    mirror.append((k, v), slots)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    batch = DecodeBatch(cache, range(n), max_blocks=mb, scored=True, stream=side)
    q, k, v, out = io(rng, L, n, n_q, n_kv, d, dtype)
    torch.cuda.synchronize()
    st = batch.step(to_torch(q, dtype), to_torch(k, dtype), to_torch(v, dtype), out, 0.125)
    torch.cuda.synchronize()
    mirror.append((k, v), st["slots"].numpy())
    scores = batch.scores.cpu().numpy()
    _, src, lens = cache.mgr.pack_tables(batch.seq_ids, mb)
    seen, empty = [], torch.empty

    def recorded(*a, **kw):
        if "cuda" in str(kw.get("device")):
            seen.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    torch.cuda._sleep(100_000_000)                     # some 50 ms of the current stream
    monkeypatch.setattr(torch, "empty", recorded)
    kept = batch.evict([50, 20, 31], 4)
    monkeypatch.undo()
    assert len(seen) == 2 and all(s == side for s in seen)
    torch.cuda.synchronize()
    _, dst, new_lens = cache.mgr.pack_tables(batch.seq_ids, mb)
    want_kept = np.full(tuple(kept.shape), -1, dtype=np.int32)
    new = scores.copy()
    R.evict(mirror.pools, mirror.scales, src, dst, lens, np.array([50, 20, 31]), 4, scores, new, want_kept)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(batch.scores.cpu().numpy(), new)
    mirror.check(cache, dst, new_lens)
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("scores", ["half", "narrow", "host", "layers"])
def test_a_refused_eviction_changes_nothing(q8, scores):
    """Scores that the call cannot take are refused before any table is shortened or block released."""
    desc = pkv.make_desc("bf16", 2, 12, 4, 2, 64)
    cache = PagedKVCache(desc, storage="q8" if q8 else None)
    cache.add_sequence(1, 60)
    cache.add_sequence(2, 33)
    cache.fork(1, 3)
    batch = DecodeBatch(cache, [1, 2], max_blocks=4, scored=True)
    good = batch.scores
    batch.scores = {"half": good.half(), "narrow": good[..., :-1].contiguous(), "host": good.cpu(), "layers": good[:1]}[scores]
    before = cache.mgr.save()
    launches = pkv.pkv_launch_count()
    with pytest.raises(ValueError):
        batch.evict(10, 2)
    assert cache.mgr.save() == before and pkv.pkv_launch_count() == launches
    batch.scores = good
    batch.evict(10, 2)                                  # and the batch is still good
    assert [cache.mgr.block_table(i)[2] for i in (1, 2, 3)] == [10, 10, 60]
    assert pkv.pkv_get_device_status() == 0


def test_overlapped_decode_behind_an_eviction_and_a_scored_layer():
    """A layer's append + decode that may overlap the scored decode of the layer before it, right behind an
    eviction of both layers: it reads its pool at once, which the eviction must have left by then."""
    dtype, L, n, n_q, n_kv, d, c, k = "bf16", 2, 8, 16, 8, 128, 6000, 2900
    mb = -(-c // 16)
    nb = n * mb
    desc = pkv.make_desc(dtype, L, nb, n_q, n_kv, d)
    g = torch.Generator(device="cuda").manual_seed(7)
    pools = [torch.randn(pkv.pool_shape(desc), device="cuda", generator=g).bfloat16() for _ in range(2)]
    tables = torch.randperm(nb, device="cuda", generator=g).int().view(n, mb).contiguous()
    lens, keep, grown = (torch.full((n,), x, dtype=torch.int32, device="cuda") for x in (c, k, k + 1))
    scores = torch.rand((L, n, n_kv, mb * 16), device="cuda", generator=g)
    q, knew, vnew = (torch.randn((L, n, h, d), device="cuda", generator=g).bfloat16() for h in (n_q, n_kv, n_kv))
    ws, sws = pkv.alloc_workspace(desc, n, mb), pkv.alloc_scored_workspace(desc, n, mb)
    kept = torch.empty((L, n, n_kv, k), dtype=torch.int32, device="cuda")
    want = None
    for overlap in [False] + [True] * 12:
        work, sums = [p.clone() for p in pools], scores.clone()
        out = torch.zeros_like(q)
        evict = pkv.evict_launcher(desc, *work, tables, tables, lens, keep, 64, sums, sums, kept)
        first = pkv.scored_decode_launcher(desc, q, *work, tables, keep, 0.09, out, sums, sws)
        second = pkv.decode_append_launcher(desc, q, knew, vnew, *work, tables, grown, 0.09, out, ws)
        torch.cuda.synchronize()
        evict()
        first(0)
        second(1, overlap)
        torch.cuda.synchronize()
        got = [out, sums, *work]
        if want is None:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pkv.pkv_get_device_status() == 0


def test_a_planned_step_is_launched_before_sequences_change():
    """Between a step's plan and its launch a scored batch refuses to shorten or reorder its sequences: the
    step's slots and tables are of the plan's time."""
    desc = pkv.make_desc("bf16", 1, 16, 4, 2, 64)
    cache = PagedKVCache(desc, storage="q8")
    for i in range(2):
        cache.add_sequence(i, 40 + i)
    batch = DecodeBatch(cache, [0, 1], max_blocks=4, scored=True)
    q, k, v, out = (torch.zeros((1, 2, h, 64), device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2, 4))
    st = batch.plan()
    before = cache.mgr.save()
    with pytest.raises(ValueError, match="planned"):
        batch.evict(10, 2)
    with pytest.raises(ValueError, match="planned"):
        batch.set_sequences([1, 0])
    batch.set_sequences([0, 1])                         # no change
    assert cache.mgr.save() == before
    batch.upload(st)
    batch.run_device(st, q, k, v, out, 0.1)
    batch.set_sequences([1, 0])
    batch.evict(10, 2)
    assert [cache.mgr.block_table(i)[2] for i in (0, 1)] == [10, 10]
    plain = DecodeBatch(cache, [0, 1], max_blocks=4)   # without scores its rows may be reordered at any time
    plain.plan()
    plain.set_sequences([1, 0])
    assert pkv.pkv_get_device_status() == 0
