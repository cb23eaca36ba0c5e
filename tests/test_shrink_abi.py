"""8-bit pools, summed weights and eviction without a GPU: sizes, refusals before any launch, the shortening
of sequences in the block manager."""
import ctypes
from pathlib import Path

import numpy as np
import pytest
import torch

import shrink_oracle as R
from paged_kv_cache_258_gb300 import pkv

PTR, MIS, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), ctypes.c_void_p(0)


def desc_of(dtype="bf16", layers=2, nb=16, n_q=4, n_kv=2, d=64):
    return pkv.make_desc(dtype, layers, nb, n_q, n_kv, d)


def test_sizes():
    d = desc_of()
    assert pkv.pkv_q8_pool_bytes(d) == 2 * 16 * 2 * 16 * 64 == pkv.pkv_pool_bytes(d) // 2
    assert pkv.pkv_q8_scale_bytes(d) == 2 * 16 * 2 * 4
    # counters, the partial results of 640 runs (2 x 32, 16 or 8 rows of d + 2 floats), one layer of K and V in 16 bits
    for dim, rows in ((64, 32), (128, 16), (256, 8)):
        x = pkv.make_desc("f16", 2, 16, 4, 2, dim)
        assert pkv.pkv_q8_prefill_workspace_bytes(x) == 8192 + 640 * 2 * rows * (dim + 2) * 4 + 2 * pkv.pkv_pool_bytes(x) // 2
    assert pkv.pkv_evict_workspace_bytes(d, 3, 7, True) == 2 * 2 * 3 * 2 * 7 * 4
    assert pkv.pkv_evict_workspace_bytes(d, 3, 7, False) == 0
    f32 = desc_of("f32")
    assert pkv.pkv_q8_pool_bytes(f32) == pkv.pkv_q8_scale_bytes(f32) == pkv.pkv_q8_prefill_workspace_bytes(f32) == 0
    assert pkv.pkv_q8_decode_workspace_bytes(d, 0, 4) == pkv.pkv_scored_workspace_bytes(d, 4, 0) == 0


def append(d, layer=0, n=3, k=PTR, v=PTR, slots=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR):
    return pkv.lib().pkv_q8_append(ctypes.byref(d), layer, k, v, slots, n, kc, vc, ks, vs, NULL)


def decode(d, layer=0, n=2, mb=4, q=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR, tables=PTR, lens=PTR, out=PTR, scores=NULL, stride=0):
    return pkv.lib().pkv_q8_decode_attention(ctypes.byref(d), layer, q, kc, vc, ks, vs, tables, mb, lens, n, 0.1, out,
                                             scores, stride, NULL, 0, NULL)


def scored(d, layer=0, n=2, mb=4, q=PTR, kp=PTR, vp=PTR, tables=PTR, lens=PTR, out=PTR, scores=PTR, stride=64):
    return pkv.lib().pkv_paged_decode_attention_scored(ctypes.byref(d), layer, q, kp, vp, tables, mb, lens, n, 0.1, out,
                                                       scores, stride, NULL, 0, NULL)


def prefill(d, layer=0, n=2, tok=5, mq=3, mb=4, q=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR, out=PTR, ws=PTR, ws_bytes=1 << 30):
    return pkv.lib().pkv_q8_prefill_attention(ctypes.byref(d), layer, q, kc, vc, ks, vs, PTR, mb, PTR, PTR, n, tok, mq,
                                              0.1, out, ws, ws_bytes, NULL)


def evict(d, n=2, mb=4, recent=1, kp=PTR, vp=PTR, ks=NULL, vs=NULL, src=PTR, dst=PTR, lens=PTR, keep=PTR, scores=PTR,
          new=PTR, stride=64, kept=PTR, max_keep=8, ws=NULL, ws_bytes=0):
    return pkv.lib().pkv_evict_tokens(ctypes.byref(d), kp, vp, ks, vs, src, dst, mb, lens, keep, n, recent, scores, new,
                                      stride, kept, max_keep, ws, ws_bytes, NULL)


def copy(d, n=1, kc=PTR, vc=PTR, ks=PTR, vs=PTR, pairs=PTR):
    return pkv.lib().pkv_q8_copy_blocks(ctypes.byref(d), kc, vc, ks, vs, pairs, n, NULL)


@pytest.mark.parametrize("call", [append, decode, scored, prefill, copy])
def test_fp32_and_unsupported_shapes_are_refused(call):
    assert call(desc_of("f32")) == pkv.PKV_ERR_UNSUPPORTED
    assert call(desc_of(d=96)) == pkv.PKV_ERR_UNSUPPORTED
    assert call(desc_of(n_q=6)) == pkv.PKV_ERR_UNSUPPORTED
    assert call(desc_of(layers=0)) == pkv.PKV_ERR_INVALID_ARG


def test_evict_takes_fp32_pools_but_no_fp32_codes():
    assert evict(desc_of("f32"), ks=PTR, vs=PTR) == pkv.PKV_ERR_UNSUPPORTED
    assert evict(desc_of("f32"), stride=63) == pkv.PKV_ERR_INVALID_ARG      # past the check of the type


@pytest.mark.parametrize("call,kw", [
    (append, dict(layer=2)), (append, dict(layer=-1)), (append, dict(n=-1)), (append, dict(k=NULL)), (append, dict(v=MIS)),
    (append, dict(slots=NULL)), (append, dict(kc=MIS)), (append, dict(vc=NULL)), (append, dict(ks=NULL)),
    (append, dict(vs=ctypes.c_void_p(0x10002))),
    (decode, dict(layer=2)), (decode, dict(n=-1)), (decode, dict(mb=0)), (decode, dict(mb=(1 << 24) + 1)),
    (decode, dict(q=NULL)), (decode, dict(q=MIS)), (decode, dict(kc=MIS)), (decode, dict(ks=NULL)), (decode, dict(vs=NULL)),
    (decode, dict(tables=NULL)), (decode, dict(lens=NULL)), (decode, dict(out=MIS)),
    (decode, dict(scores=PTR, stride=63)), (decode, dict(scores=ctypes.c_void_p(0x10002), stride=64)),
    (scored, dict(scores=NULL)), (scored, dict(stride=63)), (scored, dict(layer=3)), (scored, dict(kp=MIS)),
    (prefill, dict(layer=2)), (prefill, dict(n=-1)), (prefill, dict(tok=-1)), (prefill, dict(mq=6)), (prefill, dict(mb=0)),
    (prefill, dict(ws=NULL)), (prefill, dict(ws_bytes=100)), (prefill, dict(ws=MIS)), (prefill, dict(q=NULL)),
    (prefill, dict(ks=NULL)),
    (evict, dict(n=-1)), (evict, dict(recent=-1)), (evict, dict(mb=0)), (evict, dict(max_keep=0)), (evict, dict(kp=NULL)),
    (evict, dict(src=NULL)), (evict, dict(dst=NULL)), (evict, dict(lens=NULL)), (evict, dict(keep=NULL)),
    (evict, dict(scores=NULL)), (evict, dict(new=NULL)), (evict, dict(kept=NULL)), (evict, dict(stride=63)),
    (evict, dict(ks=PTR)), (evict, dict(ks=PTR, vs=PTR)), (evict, dict(ks=PTR, vs=PTR, ws=PTR, ws_bytes=7)),
    (evict, dict(vp=MIS)),
    (copy, dict(n=-1)), (copy, dict(pairs=NULL)), (copy, dict(kc=MIS)), (copy, dict(vs=NULL)),
])
def test_bad_arguments_are_refused(call, kw):
    assert call(desc_of(), **kw) == pkv.PKV_ERR_INVALID_ARG


def test_sizes_past_the_limits_are_refused():
    d = desc_of()
    assert decode(d, n=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert scored(d, n=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert prefill(d, n=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert evict(d, n=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert evict(desc_of(layers=65536)) == pkv.PKV_ERR_UNSUPPORTED
    wide = desc_of(nb=(1 << 26), n_kv=2)                                    # 2^31 rows a layer
    assert decode(wide) == scored(wide) == prefill(wide) == pkv.PKV_ERR_UNSUPPORTED


def test_empty_calls_do_nothing():
    d, L = desc_of(), pkv.pkv_launch_count()
    assert append(d, n=0, k=NULL) == decode(d, n=0, q=NULL) == scored(d, n=0, q=NULL, scores=NULL) == pkv.PKV_OK
    assert prefill(d, n=0) == prefill(d, mq=0) == evict(d, n=0) == copy(d, n=0) == pkv.PKV_OK
    assert pkv.pkv_launch_count() == L


def test_the_binding_refuses_host_and_misshaped_tensors():
    d = desc_of()
    codes = torch.zeros(pkv.pool_shape(d), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(pkv.scale_shape(d))
    pool = torch.zeros(pkv.pool_shape(d), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    tables, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    scores = torch.zeros((2, 2, 64))
    all_scores = torch.zeros((2, 2, 2, 64))
    kept = torch.zeros((2, 2, 2, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.pkv_q8_append(d, 0, k, k, torch.zeros(2, dtype=torch.int64), codes, codes, scales, scales)
    with pytest.raises(ValueError):
        pkv.pkv_q8_copy_blocks(d, codes, codes, scales, scales, torch.zeros((1, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        pkv.pkv_q8_decode_attention(d, 0, q, codes, codes, scales, scales, tables, lens, 0.1, q)
    with pytest.raises(ValueError):
        pkv.pkv_q8_prefill_attention(d, 0, q, codes, codes, scales, scales, tables, lens, lens, 1, 0.1, q, pool)
    with pytest.raises(ValueError):
        pkv.pkv_paged_decode_attention_scored(d, 0, q, pool, pool, tables, lens, 0.1, q, scores, pool)
    with pytest.raises(ValueError, match="at least 64"):
        pkv.pkv_paged_decode_attention_scored(d, 0, q, pool, pool, tables, lens, 0.1, q, scores[..., :63], pool)
    with pytest.raises(ValueError):
        pkv.pkv_evict_tokens(d, pool, pool, tables, tables, lens, lens, 1, all_scores, all_scores, kept)
    with pytest.raises(ValueError, match="block_tables"):
        pkv.pkv_q8_decode_attention(d, 0, q, codes, codes, scales, scales, lens, lens, 0.1, q)


# ---- pkv_mgr_compact -------------------------------------------------------------------------------

class PlainManager:
    """Tables, reference counts and free list as plain lists; only what compact needs."""

    def __init__(self, mgr, ids):
        self.tables = {i: mgr.block_table(i)[1] for i in ids}
        self.ctx = {i: mgr.block_table(i)[2] for i in ids}
        self.free = mgr.free_list()
        self.ref = mgr.refcounts()

    def compact(self, ids, lens):
        keep = {i: -(-n // 16) for i, n in zip(ids, lens)}
        shared = [(i, b) for i, n in zip(ids, lens) if n != self.ctx[i] for b in range(keep[i]) if self.ref[self.tables[i][b]] > 1]
        if len(shared) > len(self.free):
            return False
        fresh = [self.free.pop(0) for _ in shared]
        dropped = []
        for (i, b), f in zip(shared, fresh):
            dropped.append(self.tables[i][b])
            self.tables[i][b] = f
            self.ref[f] = 1
        tails = []
        for i, n in zip(ids, lens):
            if n != self.ctx[i]:
                tails += self.tables[i][keep[i]:]
                self.tables[i] = self.tables[i][:keep[i]]
                self.ctx[i] = n
        for b in tails + dropped:
            self.ref[b] -= 1
            if self.ref[b] == 0:
                self.free.append(b)
        return True

    def check(self, mgr):
        for i, t in self.tables.items():
            assert mgr.block_table(i)[1:] == (t, self.ctx[i])
        assert mgr.free_list() == self.free and mgr.refcounts() == self.ref


@pytest.mark.parametrize("seed", range(8))
def test_compact_matches_a_plain_restatement(seed):
    rng = np.random.default_rng(seed)
    nb = 60
    m = pkv.BlockManager(nb, free_order=rng.permutation(nb))
    ids = []
    for step in range(60):
        op = rng.integers(4)
        if op == 0 and len(ids) < 8:
            sid = 100 + step
            if m.add_seq(sid, int(rng.integers(0, 90)))[0] == pkv.PKV_OK:
                ids.append(sid)
        elif op == 1 and ids and len(ids) < 8:
            sid = 100 + step
            if m.fork(int(rng.choice(ids)), sid) == pkv.PKV_OK:
                ids.append(sid)
        elif op == 2 and ids:
            m.extend(int(rng.choice(ids)), int(rng.integers(0, 20)))
        elif ids:
            some = [int(x) for x in rng.permutation(ids)[:rng.integers(1, len(ids) + 1)]]
            plain = PlainManager(m, ids)
            lens = [int(rng.integers(0, plain.ctx[i] + 1)) for i in some]
            failures = m.stats()["alloc_failures"]
            ok = plain.compact(some, lens)
            rc = m.compact(some, lens)
            assert rc == (pkv.PKV_OK if ok else pkv.PKV_ERR_NO_BLOCKS)
            assert m.stats()["alloc_failures"] == failures + (not ok)
            plain.check(m)
    image = m.save()
    assert pkv.BlockManager.load(image).save() == image


def test_compact_refusals_change_nothing():
    m = pkv.BlockManager(8)
    m.add_seq(1, 40)
    m.fork(1, 2)
    m.add_seq(3, 60)
    before = m.save()
    for ids, lens, rc in [([1, 1], [3, 3], pkv.PKV_ERR_INVALID_ARG), ([9], [0], pkv.PKV_ERR_INVALID_ARG),
                          ([1], [41], pkv.PKV_ERR_INVALID_ARG), ([1], [-1], pkv.PKV_ERR_INVALID_ARG)]:
        assert m.compact(ids, lens) == rc
        assert m.save() == before
    assert m.compact([1, 2], [39, 39]) == pkv.PKV_ERR_NO_BLOCKS       # six fresh blocks, one free
    assert m.stats()["alloc_failures"] == 1
    assert m.block_table(1)[1] == m.block_table(2)[1] and len(m.free_list()) == 1
    m.inject_alloc_failure(0)
    assert m.compact([1], [10]) == pkv.PKV_ERR_NO_BLOCKS              # rolled back
    assert m.block_table(1)[2] == 40 and m.free_list() == [7]
    assert m.compact([1], [10]) == pkv.PKV_OK
    assert m.block_table(1)[1:] == ([7], 10) and m.block_table(2)[1] == [0, 1, 2]
    assert m.compact([], []) == pkv.PKV_OK
    with pytest.raises(ValueError):
        m.compact([1], [1, 2])


def test_compact_takes_fresh_blocks_before_it_releases_any():
    """A block released by one sequence is never another's destination in the same call: its rows are
    still to be read."""
    m = pkv.BlockManager(6)
    m.add_seq(1, 48)
    m.fork(1, 2)
    m.add_seq(3, 32)
    assert m.free_list() == [5]
    assert m.compact([3, 1], [16, 16]) == pkv.PKV_OK
    assert m.block_table(1)[1] == [5] and m.block_table(3)[1] == [3] and m.free_list() == [4]


# ---- the restatement itself --------------------------------------------------------------------------

def test_codes_match_another_implementation():
    """The e4m3 table and rounding of the restatement against torch's conversions."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, R.VALUES, equal_nan=True)
    x = np.clip(np.random.default_rng(0).standard_normal(50000) * 100, -448, 448).astype(np.float32)
    ties = (R.VALUES[:126] + R.VALUES[1:127]) / 2
    x = np.concatenate([x, ties, -ties, R.VALUES[:127]]).astype(np.float32)
    assert np.array_equal(R.to_codes(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scales_are_the_least_that_fit(dtype):
    for amax in (0.0, 1e-9, 447.9, 448.0, 448.1, 896.0, 65504.0, 2.0 ** -24):
        s = R.least_scale(amax, dtype)
        assert amax <= 448 * s and (s == 2.0 ** R.MIN_EXP[dtype] or amax > 448 * s / 2)


def test_an_eviction_workspace_is_not_written_when_it_is_allocated(monkeypatch):
    """It holds saved scales, not counters: a fill queued behind the eviction's first launch would wipe them."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(5.0))
    assert torch.all(pkv.alloc_evict_workspace(desc_of(), 3, 700, device="cpu") == 5.0)
    counted = pkv.alloc_q8_prefill_workspace(desc_of(), device="cpu")      # this one holds counters
    words = pkv.PKV_ARRIVAL_BYTES // 4
    assert not counted[:words].any() and torch.all(counted[words:] == 5.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_the_range_that_keeps_full_precision(dtype):
    """Elements down to 1 / 14,336 of a block's largest are held within 2^-4 of themselves: the least scale S has
    224 S < largest <= 448 S, and codes are normal from 2^-6 S on. A factor of 2^14 would be too much."""
    rng = np.random.default_rng(0)
    worst = {14336.0: 0.0, 2.0 ** 14: 0.0}
    for amax in np.concatenate([[224.001, 225.0, 256.0, 300.0, 447.9, 448.0], rng.uniform(224.1, 448, 200)]) * 2.0 ** 3:
        s = R.least_scale(amax, dtype)
        assert 224 * s < amax <= 448 * s
        for factor in worst:
            x = amax / np.exp(rng.uniform(0, np.log(factor), 4000))
            x = np.append(x, amax / factor)
            worst[factor] = max(worst[factor], np.max(np.abs(R.VALUES[R.to_codes(x / s)] * s / x - 1)))
    assert worst[14336.0] <= 2.0 ** -4 < worst[2.0 ** 14]
    assert "factor 14,336" in (Path(__file__).resolve().parents[1] / "include" / "pkv.h").read_text()


def test_more_heads_than_a_grid_holds_are_refused():
    many = desc_of(nb=1, n_q=65536, n_kv=65536)
    assert decode(many) == scored(many) == prefill(many) == pkv.PKV_ERR_UNSUPPORTED
    # the append has a CTA for every 16 tokens, head, K and V: 2^31 - 1 at most
    assert append(desc_of(nb=1, n_q=1 << 30, n_kv=1 << 30), n=1) == pkv.PKV_ERR_UNSUPPORTED
    assert append(desc_of(nb=1, n_q=1 << 27, n_kv=1 << 27), n=8 * 16) == pkv.PKV_ERR_UNSUPPORTED
