"""Decode with summed weights over 16-bit pools, and eviction, on the GPU against 64-bit restatements."""
import numpy as np
import pytest
import torch

import shrink_oracle as R
from helpers import NP_STORAGE, as_f64, paged_case, to_host, to_torch
from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BLOCK = 16
COUNTERS = 2048  # words at the front of a decode workspace that are zero between calls


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_scored_decode_matches(dtype, d, G):
    lens = [0, 1, 16, 17, 100, 1500 if G == 4 else 47]
    q, kp, vp, tables, lens, nb = paged_case(dtype, lens, 2 * G, 2, d, seed=d + G)
    desc = pkv.make_desc(dtype, 1, nb, 2 * G, 2, d)
    f64 = [as_f64(to_torch(x, dtype, device="cpu")) for x in (q, kp[0], vp[0])]
    scale = 1 / np.sqrt(d)
    want, tol, w, w_tol = R.decode(f64[0], np.nan_to_num(f64[1]), np.nan_to_num(f64[2]), tables, lens, scale, dtype,
                                   R.HALF_STEP[dtype])
    n, mb = tables.shape
    start = torch.rand((n, 2, mb * BLOCK + 3), device="cuda")
    scores = start.clone()
    tq = to_torch(q, dtype)
    out = torch.full_like(tq, float("nan"))
    ws = pkv.alloc_scored_workspace(desc, n, mb)
    if ws is not None:
        ws[COUNTERS:].fill_(float("nan"))
    pkv.pkv_paged_decode_attention_scored(desc, 0, tq, to_torch(kp, dtype), to_torch(vp, dtype),
                                          torch.from_numpy(np.ascontiguousarray(tables)).cuda(),
                                          torch.from_numpy(lens).cuda(), scale, out, scores, ws)
    assert pkv.pkv_get_device_status() == 0
    assert np.all(np.abs(as_f64(out) - want) <= tol)
    got, was = scores.double().cpu().numpy(), start.double().cpu().numpy()
    total = was[:, :, :w.shape[2]] + w
    assert np.all(np.abs(got[:, :, :w.shape[2]] - total) <= w_tol + 2.0 ** -23 * total)
    for s, c in enumerate(lens):
        assert np.array_equal(got[s, :, c:], was[s, :, c:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G", [1, 4])
def test_scored_decode_of_many_small_weights(dtype, G):
    """One key outweighs each of 40,000 others by 2^23.5, below fp16's last subnormal's half step at 1, and
    only the others have values: each of their weights still rounds by half a step of its own."""
    d, c = 64, 40000
    nb = c // BLOCK
    k, v = np.zeros((nb, 1, BLOCK, d), dtype=np.float32), np.full((nb, 1, BLOCK, d), 8.0, dtype=np.float32)
    k[nb // 2, 0, 3], v[nb // 2, 0, 3] = 2.03125, 0.0     # logit 64 * 2.03125 / 8 = 16.25 = 23.44 ln 2
    tk, tv = (torch.from_numpy(x[None]).cuda().to(pkv.torch_dtype(dtype)) for x in (k, v))
    q = np.ones((1, G, d))
    tables, lens = np.arange(nb, dtype=np.int32)[None], np.array([c], dtype=np.int32)
    want, tol, w, w_tol = R.decode(q, k.astype(np.float64), v.astype(np.float64), tables, lens, 0.125, dtype,
                                   R.HALF_STEP[dtype])
    desc = pkv.make_desc(dtype, 1, nb, G, 1, d)
    tq = torch.ones((1, G, d), device="cuda", dtype=pkv.torch_dtype(dtype))
    out, scores = torch.empty_like(tq), torch.zeros((1, 1, c), device="cuda")
    pkv.pkv_paged_decode_attention_scored(desc, 0, tq, tk, tv, torch.from_numpy(tables).cuda(),
                                          torch.from_numpy(lens).cuda(), 0.125, out, scores,
                                          pkv.alloc_scored_workspace(desc, 1, nb))
    assert np.all(np.abs(as_f64(out) - want) <= tol) and np.all(tol < 0.02 * want)
    assert np.all(np.abs(scores.double().cpu().numpy() - w) <= w_tol + 2.0 ** -23 * w)


def evict_case(dtype, lens, keep, n_kv, d, layers, seed, in_place, q8, max_blocks=None, stride_more=0):
    rng = np.random.default_rng(seed)
    lens, keep = np.asarray(lens, dtype=np.int32), np.asarray(keep, dtype=np.int32)
    n = len(lens)
    nbs = -(-lens.astype(np.int64) // BLOCK)
    mb = max_blocks or max(1, int(nbs.max()))
    k = np.minimum(np.maximum(keep, 0), lens)
    fresh = -(-k // BLOCK)
    nb = int(nbs.sum() + fresh.sum()) + 2
    order = rng.permutation(nb)
    src, at = np.full((n, mb), -1, dtype=np.int32), 0
    for s in range(n):
        src[s, :nbs[s]] = order[at:at + nbs[s]]
        at += int(nbs[s])
    dst = np.full((n, mb), -1, dtype=np.int32)
    for s in range(n):
        for b in range(fresh[s]):
            own = in_place is True or (in_place == "mixed" and rng.random() < 0.6)
            dst[s, b] = src[s, b] if own else order[at]
            at += 1
    shape = (layers, nb, n_kv, BLOCK, d)
    if q8:
        pools = [rng.integers(0, 256, size=shape, dtype=np.uint8) for _ in range(2)]
        scales = [(2.0 ** rng.integers(-8, 9, size=shape[:3])).astype(np.float32) for _ in range(2)]
    else:
        pools = [W.normal_values(rng, shape, dtype) for _ in range(2)]
        scales = None
    scores = rng.random((layers, n, n_kv, mb * BLOCK + stride_more), dtype=np.float32)
    desc = pkv.make_desc(dtype, layers, nb, n_kv, n_kv, d)
    return desc, pools, scales, src, dst, lens, keep, scores


def run_evict(desc, pools, scales, src, dst, lens, keep, scores, recent, dtype, same_scores, max_keep=None, stream=None):
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    if scales:
        tp = [c(p).view(torch.float8_e4m3fn) for p in pools]
        ts = [c(s) for s in scales]
        more = dict(k_scales=ts[0], v_scales=ts[1], workspace=pkv.alloc_evict_workspace(desc, *src.shape))
    else:
        tp, ts, more = [to_torch(p, dtype) for p in pools], None, {}
    sc = c(scores)
    new = sc if same_scores else torch.full_like(sc, 9.0)
    top = max_keep or max(1, int(np.minimum(keep, lens).max()))
    kept = torch.full((*scores.shape[:3], top), -7, dtype=torch.int32, device="cuda")
    pkv.pkv_evict_tokens(desc, tp[0], tp[1], c(src), c(dst), c(lens), c(keep), recent, sc, new, kept, stream=stream, **more)
    torch.cuda.synchronize()
    host = [p.view(torch.uint8).cpu().numpy() if scales else to_host(p, dtype) for p in tp]
    return host, [s.cpu().numpy() for s in ts] if ts else None, new.cpu().numpy(), kept.cpu().numpy(), sc.cpu().numpy()


def nan_blind(a):
    return np.where(a & 127 == 127, 127, a)


def check_evict(case, recent, dtype, same_scores, **more):
    desc, pools, scales, src, dst, lens, keep, scores = case
    got = run_evict(desc, pools, scales, src, dst, lens, keep, scores, recent, dtype, same_scores, **more)
    new = scores.copy() if same_scores else np.full_like(scores, 9.0)
    kept = np.full(got[3].shape, -7, dtype=np.int32)
    want = [p.copy() for p in pools]
    want_s = [s.copy() for s in scales] if scales else None
    R.evict(want, want_s, src, dst, lens, keep, recent, scores, new, kept)
    assert np.array_equal(got[3], kept)
    assert np.array_equal(got[2], new, equal_nan=True)
    if not same_scores:
        assert np.array_equal(got[4], scores, equal_nan=True)
    for a, b in zip(got[0], want):
        if scales:
            # rows the call moves compare as codes, the two NaN codes as one
            assert np.array_equal(nan_blind(a), nan_blind(b))
        else:
            assert np.array_equal(a, b)
    if scales:
        for a, b in zip(got[1], want_s):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("in_place", [True, False, "mixed"])
@pytest.mark.parametrize("dtype,d,q8", [("f32", 64, False), ("f16", 128, False), ("bf16", 256, False), ("f16", 64, True),
                                        ("bf16", 128, True), ("bf16", 256, True)])
def test_evict_matches(in_place, dtype, d, q8):
    lens = [0, 1, 16, 40, 333, 100, 257]
    keep = [0, 1, 3, 40, 90, 0, 256]
    case = evict_case(dtype, lens, keep, 2, d, 2, seed=d, in_place=in_place, q8=q8, stride_more=5)
    check_evict(case, 7, dtype, same_scores=in_place is True)
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("recent", [0, 1, 50, 10 ** 6, 2 ** 40])
def test_evict_recent_window(recent):
    case = evict_case("bf16", [700, 64], [300, 33], 3, 64, 1, seed=2, in_place=True, q8=False)
    check_evict(case, recent, "bf16", same_scores=True)


def test_evict_long_sequence_in_place():
    """Many chunks of the sweep and of the move; few (sequence, head) pairs, so columns are cut finely."""
    case = evict_case("f16", [9001], [4321], 1, 256, 1, seed=3, in_place=True, q8=False)
    check_evict(case, 100, "f16", same_scores=True)
    case = evict_case("f16", [9001], [8999], 1, 128, 1, seed=4, in_place=True, q8=True)
    check_evict(case, 0, "f16", same_scores=True)


def test_evict_ties_zeros_and_special_scores():
    """Equal scores keep the lower positions; zeros of both signs are equal; +inf and NaN stay first;
    negative scores go last."""
    case = list(evict_case("bf16", [600, 600, 600], [200, 31, 590], 2, 64, 1, seed=5, in_place=False, q8=False))
    sc = case[7]
    sc[0, 0] = 0.25
    sc[0, 1] = np.where(np.arange(sc.shape[-1]) % 3 == 0, -0.0, 0.0)
    sc[0, 2] = np.round(sc[0, 2] * 4) - 2
    sc[0, 2, :, 17], sc[0, 2, :, 300], sc[0, 2, :, 301] = np.inf, np.nan, -np.inf
    sc[0, 1, :, 500], sc[0, 1, :, 499] = np.nan, np.inf
    check_evict(tuple(case), 4, "bf16", same_scores=False)


def test_evict_long_8_bit_sequence_in_pieces():
    """More positions than the selection's registers hold, and more blocks than its threads."""
    case = evict_case("bf16", [17000, 20000], [5000, 16001], 1, 64, 1, seed=9, in_place="mixed", q8=True)
    check_evict(case, 33, "bf16", same_scores=False)
    sc = case[7]
    sc[...] = np.round(sc * 8) / 8                        # few different scores: ties across the pieces
    check_evict(case, 33, "bf16", same_scores=True)


def test_evict_everything_or_nothing():
    case = evict_case("f16", [50, 50, 50], [0, 50, 77], 1, 64, 2, seed=6, in_place=True, q8=True)
    check_evict(case, 5, "f16", same_scores=True)


def test_evict_skips_and_flags_bad_device_values():
    desc, pools, scales, src, dst, lens, keep, scores = evict_case("f16", [100, 100, 100], [40, 50, 60], 2, 64, 1, seed=7,
                                                                   in_place=False, q8=False)
    bad = keep.copy()
    bad[1] = -2
    host, _, new, kept, _ = run_evict(desc, pools, scales, src, dst, lens, bad, scores, 3, "f16", False, max_keep=50)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_KEEP    # negative, and 60 > max_keep
    assert np.all(kept[:, 1:] == -7) and np.all(new[:, 1:] == 9.0) and np.all(kept[:, 0, :, :40] >= 0)
    for s in (1, 2):
        for b in dst[s][dst[s] >= 0]:
            assert np.array_equal(host[0][0, b], pools[0][0, b])
    lens2 = lens.copy()
    lens2[2] = 16 * src.shape[1] + 1
    run_evict(desc, pools, scales, src, dst, lens2, keep, scores, 3, "f16", False)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_CONTEXT_LEN
    src2 = src.copy()
    src2[0, 1] = desc.num_blocks
    host, _, _, kept, _ = run_evict(desc, pools, scales, src2, dst, lens, keep, scores, 3, "f16", False)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_BLOCK_ID
    for g in range(2):
        for i in range(40):
            j = int(kept[0, 0, g, i])
            row = host[0][0, dst[0, i // 16], g, i % 16]
            same = pools[0][0, dst[0, i // 16], g, i % 16] if j // 16 == 1 else pools[0][0, src[0, j // 16], g, j % 16]
            assert np.array_equal(row, same)


def test_evict_on_another_stream_and_in_a_graph():
    case = evict_case("bf16", [200, 90], [64, 20], 2, 128, 2, seed=8, in_place=False, q8=True)
    check_evict(case, 6, "bf16", same_scores=False, stream=torch.cuda.current_stream())
    desc, pools, scales, src, dst, lens, keep, scores = case
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    tp, ts = [c(p).view(torch.float8_e4m3fn) for p in pools], [c(s) for s in scales]
    sc, new = c(scores), c(np.full_like(scores, 9.0))
    kept = torch.full((*scores.shape[:3], 64), -7, dtype=torch.int32, device="cuda")
    ws = pkv.alloc_evict_workspace(desc, *src.shape)
    args = (desc, tp[0], tp[1], c(src), c(dst), c(lens), c(keep), 6, sc, new, kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_evict_tokens(*args, k_scales=ts[0], v_scales=ts[1], workspace=ws)
    g.replay()
    g.replay()  # out of place: the same again
    torch.cuda.synchronize()
    got = run_evict(desc, pools, scales, src, dst, lens, keep, scores, 6, "bf16", False)
    assert np.array_equal(tp[0].view(torch.uint8).cpu().numpy(), got[0][0])
    assert np.array_equal(new.cpu().numpy(), got[2]) and np.array_equal(kept.cpu().numpy(), got[3])


@pytest.mark.parametrize("q8", [False, True])
def test_evict_offsets_past_32_bits(q8):
    """Pools of over 2^32 bytes, the sequence in the last blocks, moved in place and apart."""
    d, n_kv, c, k = 256, 8, 150, 61
    nb = 140_000 if q8 else 70_000
    desc = pkv.make_desc("f16", 1, nb, n_kv, n_kv, d)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.arange(nb - 20, nb, device="cuda")[torch.randperm(20, generator=torch.Generator().manual_seed(1))].int()
    for in_place in (True, False):
        if q8:
            pools = [torch.zeros(pkv.pool_shape(desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
            for p in pools:
                p[0, nb - 20:] = torch.randint(0, 120, (20, n_kv, 16, d), device="cuda", generator=g, dtype=torch.uint8)
            sc = [torch.ones(pkv.scale_shape(desc), device="cuda") for _ in range(2)]
            more = dict(k_scales=sc[0], v_scales=sc[1], workspace=pkv.alloc_evict_workspace(desc, 1, 10))
            calls = [p.view(torch.float8_e4m3fn) for p in pools]
        else:
            pools = [torch.zeros(pkv.pool_shape(desc), dtype=torch.float16, device="cuda") for _ in range(2)]
            for p in pools:
                p[0, nb - 20:] = torch.randn((20, n_kv, 16, d), device="cuda", generator=g).half()
            calls, more = pools, {}
        src = ids[:10].contiguous()
        dst = src if in_place else ids[10:].contiguous()
        scores = torch.rand((1, 1, n_kv, 160), device="cuda", generator=g)
        kept = torch.empty((1, 1, n_kv, k), dtype=torch.int32, device="cuda")
        rows = [p[0, src.long()].transpose(0, 1).reshape(n_kv, 160, d).clone() for p in pools]
        pkv.pkv_evict_tokens(desc, calls[0], calls[1], src[None], dst[None], torch.tensor([c], dtype=torch.int32, device="cuda"),
                             torch.tensor([k], dtype=torch.int32, device="cuda"), 9, scores, torch.zeros_like(scores), kept, **more)
        assert pkv.pkv_get_device_status() == 0
        at = kept[0, 0].long()
        for p, r in zip(pools, rows):
            moved = p[0, dst.long()].transpose(0, 1).reshape(n_kv, 160, d)[:, :k]
            assert torch.equal(moved, r.gather(1, at[..., None].expand(-1, -1, d)))
        del pools, calls
        torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [100, 256, 257, 400])
def test_evict_of_many_sequences(n):
    """As many sequences as the move ranks by what they keep, and more; some equal, some empty."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 90, size=n)
    keep = np.minimum(rng.integers(0, 70, size=n), rng.integers(0, 70, size=n))
    case = evict_case("bf16", lens, keep, 1, 64, 1, seed=10, in_place="mixed", q8=True)
    check_evict(case, 3, "bf16", same_scores=False)
    assert pkv.pkv_get_device_status() == 0
