"""8-bit pools on the GPU: quantising append, block copies, decode (with and without summed weights) and
prefill, against 64-bit restatements."""
import numpy as np
import pytest
import torch

import shrink_oracle as R
from helpers import as_f64, to_host, to_torch
from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300 import workloads as W

pytestmark = pytest.mark.gpu
BLOCK = 16
COUNTERS = 2048  # words at the front of a decode workspace that are zero between calls


def codes_to_torch(c):
    return torch.from_numpy(np.ascontiguousarray(c)).cuda().view(torch.float8_e4m3fn)


def codes_to_host(t):
    return t.view(torch.uint8).cpu().numpy()


def values(rng, shape, dtype):
    """(storage array, the same in float64)"""
    x = W.normal_values(rng, shape, dtype)
    return x, as_f64(to_torch(x, dtype, device="cpu"))


def same_codes(a, b):
    """Equal codes; the two NaN codes count as one."""
    return np.array_equal(np.where(a & 127 == 127, 127, a), np.where(b & 127 == 127, 127, b))


def filled_pools(rng, nb, n_kv, d, spread=3):
    """Random codes (no NaN) and power-of-two scales over 2 * spread binades."""
    c = rng.integers(0, 256, size=(1, nb, n_kv, BLOCK, d), dtype=np.uint8)
    c[c & 127 == 127] ^= 1
    s = 2.0 ** rng.integers(-spread, spread + 1, size=(1, nb, n_kv)).astype(np.float64) / 64
    return c, s.astype(np.float32)


def gpu_append(desc, x, y, slots, kc, vc, ks, vs, dtype):
    t = [codes_to_torch(kc), codes_to_torch(vc), torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()]
    pkv.pkv_q8_append(desc, 0, to_torch(x, dtype), to_torch(y, dtype), torch.from_numpy(slots).cuda(), *t)
    return codes_to_host(t[0]), codes_to_host(t[1]), t[2].cpu().numpy(), t[3].cpu().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_kv", [1, 3, 8])
def test_append_is_bit_exact(dtype, d, n_kv):
    """Whole blocks, blocks continued (their scale grows or not), blocks started, padding in between."""
    rng = np.random.default_rng(d + n_kv)
    nb = 12
    kc, ks = filled_pools(rng, nb, n_kv, d)
    vc, vs = filled_pools(rng, nb, n_kv, d)
    ks[0, 7], vs[0, 7] = 64.0, 64.0                 # large enough: stays
    ks[0, 8], vs[0, 8] = 2.0 ** -12, 2.0 ** -12     # far too small: old rows fall below the grid
    slots = [3 * 16 + i for i in range(16)]          # a whole block
    slots += [7 * 16 + i for i in (5, 6, 7)]         # a block continued
    slots += [8 * 16 + 15]
    slots += [-1, 2 * 16 + 0, -1, 2 * 16 + 1]        # a block started, padding inside
    slots += [9 * 16 + i for i in (9, 4, 12)]        # not in order
    slots = np.array(slots, dtype=np.int64)
    x, xf = values(rng, (len(slots), n_kv, d), dtype)
    y, yf = values(rng, (len(slots), n_kv, d), dtype)
    desc = pkv.make_desc(dtype, 1, nb, n_kv, n_kv, d)
    got = gpu_append(desc, x, y, slots, kc, vc, ks, vs, dtype)
    assert pkv.pkv_get_device_status() == 0
    R.append(xf, slots, kc[0], ks[0], dtype)
    R.append(yf, slots, vc[0], vs[0], dtype)
    assert np.array_equal(got[2], ks) and np.array_equal(got[3], vs)
    assert same_codes(got[0], kc) and same_codes(got[1], vc)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_of_special_values(dtype):
    """Zeros, subnormals, the largest finite value, infinities and NaN; a scale's borders."""
    rng = np.random.default_rng(1)
    d, nb = 64, 8
    big = 65504.0 if dtype == "f16" else 3.3895313892515355e38
    tiny = 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    rows = np.zeros((7, 1, d))
    rows[1, 0, :4] = [tiny, -tiny, 3 * tiny, 0]
    rows[2, 0, :4] = [big, -big, 1.0, -1.0]
    rows[3] = rng.standard_normal(d)
    rows[3, 0, :3] = [np.inf, -np.inf, np.nan]
    rows[4, 0, :3] = [448.0, 447.0, 1.0]             # exactly the border of a scale
    rows[5, 0, :3] = [450.0 if dtype == "bf16" else 448.25, 1.0, -0.0]  # just above it
    rows[6, 0, :2] = [np.inf, np.nan]                # nothing finite but zeros
    x = torch.from_numpy(rows).to(pkv.torch_dtype(dtype))
    xf = x.double().numpy()
    slots = np.arange(7, dtype=np.int64) * 16        # each starts a block of its own
    kc, vc = np.full((2, 1, nb, 1, BLOCK, d), 0x55, dtype=np.uint8)
    ks, vs = np.full((2, 1, nb, 1), 8.0, dtype=np.float32)
    desc = pkv.make_desc(dtype, 1, nb, 1, 1, d)
    t = [codes_to_torch(kc), codes_to_torch(vc), torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()]
    pkv.pkv_q8_append(desc, 0, x.cuda(), (2 * x).clamp(-big, big).cuda(), torch.from_numpy(slots).cuda(), *t)
    R.append(xf, slots, kc[0], ks[0], dtype)
    assert np.array_equal(t[2].cpu().numpy(), ks)
    assert same_codes(codes_to_host(t[0]), kc)
    assert np.array_equal(t[3].cpu().numpy()[0, 7], vs[0, 7])  # untouched


def test_append_skips_bad_slots_and_flags_them():
    rng = np.random.default_rng(2)
    d, nb = 128, 4
    kc, ks = filled_pools(rng, nb, 2, d)
    vc, vs = filled_pools(rng, nb, 2, d)
    slots = np.array([-5, nb * 16, 17, nb * 16 + 3, -1], dtype=np.int64)
    x, xf = values(rng, (5, 2, d), "bf16")
    desc = pkv.make_desc("bf16", 1, nb, 2, 2, d)
    got = gpu_append(desc, x, x, slots, kc, vc, ks, vs, "bf16")
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_SLOT
    R.append(xf, slots, kc[0], ks[0], "bf16")
    assert np.array_equal(got[2], ks) and same_codes(got[0], kc)


@pytest.mark.parametrize("d,n_kv", [(64, 1), (128, 4), (256, 3)])
def test_token_by_token_equals_the_definition(d, n_kv):
    """A block filled one row at a time, its scale growing on the way; then started anew."""
    rng = np.random.default_rng(3)
    dtype, nb = "bf16", 2
    kc, ks = filled_pools(rng, nb, n_kv, d)
    vc, vs = filled_pools(rng, nb, n_kv, d)
    desc = pkv.make_desc(dtype, 1, nb, n_kv, n_kv, d)
    t = [codes_to_torch(kc), codes_to_torch(vc), torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()]
    for step in range(20):
        rows = rng.standard_normal((1, n_kv, d)) * 2.0 ** rng.integers(-6, 7)
        x = torch.from_numpy(rows).to(torch.bfloat16)
        slots = np.array([16 + step % 16], dtype=np.int64)
        pkv.pkv_q8_append(desc, 0, x.cuda(), (-x).cuda(), torch.from_numpy(slots).cuda(), *t)
        R.append(x.double().numpy(), slots, kc[0], ks[0], dtype)
        R.append(-x.double().numpy(), slots, vc[0], vs[0], dtype)
        assert np.array_equal(t[2].cpu().numpy(), ks) and np.array_equal(t[3].cpu().numpy(), vs), step
        assert same_codes(codes_to_host(t[0]), kc) and same_codes(codes_to_host(t[1]), vc), step


def test_copy_blocks_moves_codes_and_scales():
    rng = np.random.default_rng(4)
    L, nb, n_kv, d = 3, 9, 5, 64
    c = rng.integers(0, 256, size=(2, L, nb, n_kv, BLOCK, d), dtype=np.uint8)
    s = rng.random((2, L, nb, n_kv), dtype=np.float32)
    t = [codes_to_torch(c[0]), codes_to_torch(c[1]), torch.from_numpy(s[0].copy()).cuda(), torch.from_numpy(s[1].copy()).cuda()]
    desc = pkv.make_desc("f16", L, nb, n_kv, n_kv, d)
    pairs = np.array([[0, 4], [8, 2], [3, 99], [-1, 5]], dtype=np.int32)
    pkv.pkv_q8_copy_blocks(desc, *t, torch.from_numpy(pairs).cuda())
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_PAIR
    for a, b in pairs[:2]:
        c[:, :, b], s[:, :, b] = c[:, :, a], s[:, :, a]
    assert np.array_equal(codes_to_host(t[0]), c[0]) and np.array_equal(codes_to_host(t[1]), c[1])
    assert np.array_equal(t[2].cpu().numpy(), s[0]) and np.array_equal(t[3].cpu().numpy(), s[1])


def q8_case(dtype, lens, n_q, n_kv, d, seed, spread=3, slack=3, max_blocks=None):
    """Pools whose unused rows hold NaN codes and whose unused blocks have NaN scales."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    nbs = -(-lens.astype(np.int64) // BLOCK)
    nb = int(nbs.sum()) + slack
    tables = W.shuffled_tables(lens, nb, seed, max_blocks=max_blocks or max(1, int(nbs.max())))
    kc, ks = filled_pools(rng, nb, n_kv, d, spread)
    vc, vs = filled_pools(rng, nb, n_kv, d, spread)
    used = np.zeros((nb, BLOCK), dtype=bool)
    for s, c in enumerate(lens):
        for j in range(int(c)):
            used[tables[s, j // BLOCK], j % BLOCK] = True
    for c in (kc, vc):
        c[0] = np.where(used[:, None, :, None], c[0], 0x7F)
    for s in (ks, vs):
        s[0, ~used.any(1)] = np.nan
    q, qf = values(rng, (len(lens), n_q, d), dtype)
    desc = pkv.make_desc(dtype, 1, nb, n_q, n_kv, d)
    dev = dict(q=to_torch(q, dtype), k=codes_to_torch(kc), v=codes_to_torch(vc), ks=torch.from_numpy(ks).cuda(),
               vs=torch.from_numpy(vs).cuda(), tables=torch.from_numpy(np.ascontiguousarray(tables)).cuda(),
               lens=torch.from_numpy(lens).cuda())
    return desc, dev, qf, R.widen(kc[0], ks[0]), R.widen(vc[0], vs[0]), tables, lens


def run_decode(desc, t, scale, scores=None, stream=None, ws=True):
    out = torch.full_like(t["q"], float("nan"))
    w = pkv.alloc_q8_workspace(desc, t["q"].shape[0], t["tables"].shape[1], scored=scores is not None) if ws else None
    if w is not None:
        w[COUNTERS:].fill_(float("nan"))
    pkv.pkv_q8_decode_attention(desc, 0, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["lens"], scale, out, w,
                                scores=scores, stream=stream)
    return out


def check_decode(desc, t, qf, kf, vf, tables, lens, dtype, scale, scored=True):
    want, tol, w, w_tol = R.decode(qf, np.nan_to_num(kf), np.nan_to_num(vf), tables, lens, scale, dtype, 2.0 ** -11)
    out = run_decode(desc, t, scale)
    assert pkv.pkv_get_device_status() == 0
    err = np.abs(as_f64(out) - want)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()),)
    if scored:
        S = tables.shape[1] * BLOCK + 5                      # a stride of its own, not a multiple of anything
        start = torch.rand((len(lens), desc.n_kv_heads, S), device="cuda")
        scores = start.clone()
        out2 = run_decode(desc, t, scale, scores)
        assert torch.equal(out2, out)                        # summing weights does not change the output
        got, was = scores.double().cpu().numpy(), start.double().cpu().numpy()
        total = was[:, :, :w.shape[2]] + w
        e = np.abs(got[:, :, :w.shape[2]] - total)
        assert np.all(e <= w_tol + 2.0 ** -23 * total)
        j = np.arange(S)[None, None] >= lens[:, None, None]
        assert np.array_equal(got[np.broadcast_to(j, got.shape)], was[np.broadcast_to(j, was.shape)])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_matches(dtype, d, G):
    lens = [0, 1, 15, 16, 17, 33, 100, 511]
    case = q8_case(dtype, lens, 2 * G, 2, d, seed=d + G)
    check_decode(*case, dtype, 1 / np.sqrt(d) / 16)


@pytest.mark.parametrize("d,G,n_kv,lens", [(128, 4, 1, [5000, 3, 0, 1024, 1025]), (256, 8, 2, [2049, 4097]),
                                           (64, 1, 3, [9000]), (128, 1, 32, [700, 1300, 64, 2048])])
def test_decode_of_split_contexts(d, G, n_kv, lens):
    case = q8_case("bf16", lens, G * n_kv, n_kv, d, seed=7, max_blocks=max(lens) // 16 + 9)
    check_decode(*case, "bf16", 1 / np.sqrt(d) / 16)


def test_decode_keeps_small_blocks_beside_huge_ones():
    """Scales 2^60 apart: a block of tiny V that holds all the weight is not lost beside a huge one that
    holds none. The huge block's keys point away from the query."""
    dtype, d = "bf16", 128
    desc, t, qf, kf, vf, tables, lens = q8_case(dtype, [64], 1, 1, d, seed=11, spread=0)
    first, last = int(tables[0, 0]), int(tables[0, 3])
    t["vs"][0, first], t["vs"][0, last] = 2.0 ** 30, 2.0 ** -30
    q = torch.ones_like(t["q"])
    codes = t["k"].view(torch.uint8)
    codes[0] = 0x38                                      # 1.0
    codes[0, first] = 0xB8                               # -1.0
    codes[0, int(tables[0, 1])] = codes[0, int(tables[0, 2])] = 0xB8
    t["q"], t["ks"][:] = q, 1.0
    k = R.VALUES[codes_to_host(t["k"])[0]]
    v = R.VALUES[codes_to_host(t["v"])[0]] * t["vs"][0].double().cpu().numpy()[..., None, None]
    want, tol, _, _ = R.decode(np.ones((1, 1, d)), k, v, tables, lens, 1.0, dtype, 2.0 ** -11)
    out = run_decode(desc, t, 1.0)
    # exp(-256) of 2^30-sized rows is far below the rest: both terms of the tolerance are the small block's
    assert np.all(np.abs(as_f64(out) - want) <= tol) and np.abs(want).max() < 2.0 ** -20


def test_decode_reads_any_scale_and_zero():
    """Scales that are no powers of two, and zero (its rows read as zeros)."""
    desc, t, qf, kf, vf, tables, lens = q8_case("f16", [50, 20], 4, 2, 64, seed=12)
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in ("ks", "vs"):
        t[n].copy_(torch.rand(t[n].shape, device="cuda", generator=g) / 32)
    t["vs"][0, int(tables[0, 1])] = 0.0
    t["ks"][0, int(tables[0, 2])] = 0.0
    pools = [R.widen(codes_to_host(t[a])[0], t[b][0].double().cpu().numpy()) for a, b in (("k", "ks"), ("v", "vs"))]
    check_decode(desc, t, qf, pools[0], pools[1], tables, lens, "f16", 0.125)


def test_decode_nan_and_infinite_inputs_reach_the_row_only():
    desc, t, qf, kf, vf, tables, lens = q8_case("bf16", [1500, 40, 300], 8, 2, 64, seed=13)
    t["k"].view(torch.uint8)[0, int(tables[0, 3]), 0, 2, 5] = 0x7F      # a NaN key of sequence 0, head 0
    t["q"][1, 6, 3] = float("nan")                                      # query head 6 of sequence 1
    out = run_decode(desc, t, 0.02)
    scores = torch.zeros((3, 2, tables.shape[1] * BLOCK), device="cuda")
    again = run_decode(desc, t, 0.02, scores)
    assert torch.equal(torch.isnan(out), torch.isnan(again))
    nan = torch.isnan(out).cpu().numpy()
    assert nan[0, :4].all() and not nan[0, 4:].any()
    assert nan[1, 6].all() and not nan[1, :6].any() and not nan[1, 7].any()
    assert not nan[2].any()
    assert torch.isnan(scores[0, 0, :1500]).all() and not torch.isnan(scores[0, 1]).any()
    assert torch.isnan(scores[1, 1, :40]).all() and not torch.isnan(scores[2]).any()


def test_decode_of_large_queries():
    """bf16 queries past fp16's range, and far below it."""
    for size in (2.0 ** 40, 2.0 ** -60, 2.0 ** -130):
        desc, t, qf, kf, vf, tables, lens = q8_case("bf16", [100, 7], 2, 1, 128, seed=14)
        t["q"] = (t["q"].double() * size).to(torch.bfloat16)
        # a scale that brings the logits back; 2^120 twice for the smallest
        scale = float(np.float32(min(1 / size, 2.0 ** 120))) / 200
        want, tol, _, _ = R.decode(as_f64(t["q"]), np.nan_to_num(kf), np.nan_to_num(vf), tables, lens, scale, "bf16",
                                   2.0 ** -11)
        assert np.all(np.abs(as_f64(run_decode(desc, t, scale)) - want) <= tol), size


def test_decode_skips_and_flags_bad_device_values():
    desc, t, qf, kf, vf, tables, lens = q8_case("f16", [64, 30], 2, 1, 128, seed=15)
    t["tables"][0, 2] = desc.num_blocks + 7
    scores = torch.zeros((2, 1, tables.shape[1] * BLOCK), device="cuda")
    out = run_decode(desc, t, 0.1, scores)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_BLOCK_ID
    live = [j for j in range(64) if j // 16 != 2]
    k, v = R.rows_of(kf, tables[0], 64, 0)[live], R.rows_of(vf, tables[0], 64, 0)[live]
    for h in range(2):
        want, w = R.attend(qf[0, h], k, v, 0.1)
        assert np.allclose(as_f64(out)[0, h], want, rtol=0, atol=2.0 ** -9 * np.abs(v).max())
    got = scores[0, 0].cpu().numpy()
    assert np.all(got[32:48] == 0) and abs(got.sum() - 2) < 1e-4
    t["lens"][1] = 16 * tables.shape[1] + 1                 # clamped to the table's width
    t["tables"][0, 2] = int(tables[0, 2])
    t["tables"][1] = t["tables"][0]
    out = run_decode(desc, t, 0.1)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_CONTEXT_LEN
    assert torch.isfinite(out).all()
    t["lens"][1] = -3
    out = run_decode(desc, t, 0.1)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_CONTEXT_LEN
    assert torch.all(out[1] == 0)


def test_decode_sequences_that_share_blocks_keep_their_own_scores():
    desc, t, qf, kf, vf, tables, lens = q8_case("bf16", [200, 200], 4, 2, 64, seed=16)
    t["tables"][1] = t["tables"][0]
    t["lens"][1] = 77
    tables = t["tables"].cpu().numpy()
    check_decode(desc, t, qf, kf, vf, tables, np.array([200, 77]), "bf16", 0.01)


def test_decode_in_a_graph_and_on_another_stream():
    desc, t, qf, kf, vf, tables, lens = q8_case("bf16", [1800, 40], 8, 2, 128, seed=17)
    scores = torch.zeros((2, 2, tables.shape[1] * BLOCK), device="cuda")
    want = run_decode(desc, t, 0.01, scores)
    once = scores.clone()
    side = torch.cuda.Stream()
    ws = pkv.alloc_q8_workspace(desc, 2, tables.shape[1], scored=True)
    out = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scores.zero_()
        args = (desc, 0, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["lens"], 0.01, out, ws)
        pkv.pkv_q8_decode_attention(*args, scores=scores)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pkv.pkv_q8_decode_attention(*args, scores=scores)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(scores, once)
        out.zero_()
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.allclose(scores, 4 * once, rtol=1e-6, atol=0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 8), (128, 4), (256, 2), (256, 4)])
def test_prefill_matches(dtype, d, G):
    """Chunks of 1 to 200 tokens, one over an empty cache, one inside a block; rows owned by no sequence."""
    lens, counts = [5, 200, 333, 40], [5, 63, 1, 40]
    n_kv = 2
    desc, t, _, kf, vf, tables, lens = q8_case(dtype, lens, G * n_kv, n_kv, d, seed=d * G)
    rng = np.random.default_rng(5)
    start = np.array([0, 5, 68, 69, 109], dtype=np.int32)
    q, qf = values(rng, (112, G * n_kv, d), dtype)
    out = torch.full((112, G * n_kv, d), 7.0, dtype=pkv.torch_dtype(dtype), device="cuda")
    ws = pkv.alloc_q8_prefill_workspace(desc)
    ws[COUNTERS:].fill_(float("nan"))
    scale = 1 / np.sqrt(d) / 16
    pkv.pkv_q8_prefill_attention(desc, 0, to_torch(q, dtype), t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["lens"],
                                 torch.from_numpy(start).cuda(), 63, scale, out, ws)
    assert pkv.pkv_get_device_status() == 0
    got = as_f64(out)
    assert np.all(got[109:] == 7.0)
    step = R.HALF_STEP[dtype]                               # the 16-bit prefill rounds its weights to the storage type
    for s in range(4):
        for i in range(counts[s]):
            p = int(lens[s]) - counts[s] + i
            row = start[s] + i
            want, tol, _, _ = R.decode(qf[row:row + 1], np.nan_to_num(kf), np.nan_to_num(vf), tables[s:s + 1],
                                       np.array([p + 1]), scale, dtype, step)
            # weights up to 2^8 of the running maximum's: their sum may be of unrounded ones (one more half step)
            assert np.all(np.abs(got[row] - want[0]) <= 2 * tol[0]), (s, i)


@pytest.mark.parametrize("n", [1, 2000])
def test_the_largest_halves_stay_finite(n):
    """65,504 is held as 65,536 in codes; attention gives 65,504 back: decode, short and long chunks."""
    d = 64
    nb = -(-n // 16)
    desc = pkv.make_desc("f16", 1, nb, 1, 1, d)
    kc = torch.zeros(pkv.pool_shape(desc), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.zeros(pkv.pool_shape(desc), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc, sv = torch.zeros((2, *pkv.scale_shape(desc)), device="cuda")
    x = torch.full((n, 1, d), 65504.0, dtype=torch.float16, device="cuda")
    pkv.pkv_q8_append(desc, 0, x, x, torch.arange(n, device="cuda"), kc, vc, sc, sv)
    assert torch.all(sv == 256.0)
    tables = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    lens = torch.full((1,), n, dtype=torch.int32, device="cuda")
    out = torch.empty((1, 1, d), dtype=torch.float16, device="cuda")
    pkv.pkv_q8_decode_attention(desc, 0, torch.zeros_like(out), kc, vc, sc, sv, tables, lens, 1.0, out,
                                pkv.alloc_q8_workspace(desc, 1, nb))
    assert torch.all(out == 65504.0)
    for m in {1, n}:
        out = torch.empty((m, 1, d), dtype=torch.float16, device="cuda")
        pkv.pkv_q8_prefill_attention(desc, 0, torch.zeros_like(out), kc, vc, sc, sv, tables, lens,
                                     torch.tensor([0, m], dtype=torch.int32).cuda(), m, 1.0, out,
                                     pkv.alloc_q8_prefill_workspace(desc))
        assert torch.all(out == 65504.0)


def prefill(desc, t, q, lens, counts, scale, dtype, extra_rows=0):
    """(outputs of a prefill call as float64, kernels launched)"""
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((int(start[-1]) + extra_rows, *q.shape[1:]), 7.0, dtype=pkv.torch_dtype(dtype), device="cuda")
    ws = pkv.alloc_q8_prefill_workspace(desc)
    ws[COUNTERS:].fill_(float("nan"))
    before = pkv.pkv_launch_count()
    pkv.pkv_q8_prefill_attention(desc, 0, to_torch(q, dtype), t["k"], t["v"], t["ks"], t["vs"], t["tables"],
                                 torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda(), torch.from_numpy(start).cuda(),
                                 int(max(counts)), scale, out, ws)
    torch.cuda.synchronize()
    return as_f64(out), pkv.pkv_launch_count() - before


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_short_chunks_over_long_contexts(dtype, d, G):
    """Chunks that go by passes of 8 rows or more (one launch): counts around the group's size, an empty
    chunk, contexts in runs and in partitions."""
    n_kv = 2
    for lens, counts in (([3000, 40, 9, 700], [11, 1, 9, 0]), ([130], [3])):
        desc, t, _, kf, vf, tables, lens = q8_case(dtype, lens, G * n_kv, n_kv, d, seed=3 * d + G)
        q, qf = values(np.random.default_rng(6), (sum(counts) + 2, G * n_kv, d), dtype)
        scale = 1 / np.sqrt(d) / 16
        got, launches = prefill(desc, t, q, lens, counts, scale, dtype, extra_rows=2)
        assert launches == 1 and pkv.pkv_get_device_status() == 0
        assert np.all(got[sum(counts):] == 7.0)
        row = 0
        for s, n in enumerate(counts):
            for i in range(n):
                want, tol, _, _ = R.decode(qf[row:row + 1], np.nan_to_num(kf), np.nan_to_num(vf), tables[s:s + 1],
                                           np.array([lens[s] - n + i + 1]), scale, dtype, 2.0 ** -11)
                assert np.all(np.abs(got[row] - want[0]) <= tol[0]), (s, i)
                row += 1


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_chunks_in_wide_passes(dtype, d, G):
    """Chunks of more rows than a column tile, tables wide enough that the passes take several tiles: chunks
    that end inside a pass, inside a tile, one token, none, and a whole context."""
    n_kv = 2
    tokens = 80 // G                                   # 80 rows: 2.5 passes of 32, 5 of 16
    lens, counts = [900, 300, tokens, 33, 17], [tokens, tokens - 3, tokens, 1, 0]
    desc, t, _, kf, vf, tables, lens = q8_case(dtype, lens, G * n_kv, n_kv, d, seed=5 * d + G, max_blocks=700)
    q, qf = values(np.random.default_rng(16), (sum(counts) + 2, G * n_kv, d), dtype)
    scale = 1 / np.sqrt(d) / 16
    got, launches = prefill(desc, t, q, lens, counts, scale, dtype, extra_rows=2)
    assert launches == 1 and pkv.pkv_get_device_status() == 0
    assert np.all(got[sum(counts):] == 7.0)
    row = 0
    for s, n in enumerate(counts):
        for i in range(n):
            want, tol, _, _ = R.decode(qf[row:row + 1], np.nan_to_num(kf), np.nan_to_num(vf), tables[s:s + 1],
                                       np.array([lens[s] - n + i + 1]), scale, dtype, 2.0 ** -11)
            assert np.all(np.abs(got[row] - want[0]) <= tol[0]), (s, i)
            row += 1


@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 2), (128, 8)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_wide_passes_are_causal_about_nan(d, G, where):
    """A NaN in the row of a new token, in the middle of a pass, reaches that token and the later ones only."""
    n_kv, length, tokens = 1, 2000, 48 // G
    desc, t, _, kf, vf, tables, lens = q8_case("bf16", [length], G, n_kv, d, seed=24, max_blocks=9000)
    at = tokens // 2 + 1
    bad = length - tokens + at
    t[where].view(torch.uint8)[0, int(tables[0, bad // 16]), 0, bad % 16, 41] = 0x7F
    q, _ = values(np.random.default_rng(17), (tokens, G, d), "bf16")
    got, launches = prefill(desc, t, q, lens, [tokens], 0.01, "bf16")
    assert launches == 1
    nan = np.isnan(got)
    assert not nan[:at].any()
    if where == "k":
        assert nan[at:].all()
    else:
        assert nan[at:, :, 41].all() and not np.delete(nan, 41, axis=2).any()


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("where", ["k", "v"])
def test_short_chunks_are_causal_about_nan(G, where):
    """A NaN in the row of one new token reaches that token and the later ones, not the earlier ones."""
    d, n_kv = 128, 1
    for length in (2000, 40):
        desc, t, _, kf, vf, tables, lens = q8_case("bf16", [length], G, n_kv, d, seed=21)
        bad = length - 3                                   # the third newest token
        t[where].view(torch.uint8)[0, int(tables[0, bad // 16]), 0, bad % 16, 77] = 0x7F
        q, _ = values(np.random.default_rng(7), (6, G, d), "bf16")
        got, launches = prefill(desc, t, q, lens, [6], 0.01, "bf16")
        assert launches == 1
        nan = np.isnan(got)
        assert not nan[:3].any()
        if where == "k":
            assert nan[3:].all()
        else:
            assert nan[3:, :, 77].all() and not np.delete(nan, 77, axis=2).any()


@pytest.mark.parametrize("wide", [0, 1000])
def test_short_chunks_skip_and_flag_bad_ranges(wide):
    """wide: table columns beyond the contexts (the launch takes runs then, not partitions)"""
    d, n_kv, G = 64, 2, 4
    desc, t, _, kf, vf, tables, lens = q8_case("f16", [900, 60, 60, 60], G * n_kv, n_kv, d, seed=22, max_blocks=57 + wide)
    q, qf = values(np.random.default_rng(8), (9, G * n_kv, d), "f16")
    out = torch.full((9, G * n_kv, d), 7.0, dtype=torch.float16, device="cuda")
    ws = pkv.alloc_q8_prefill_workspace(desc)
    lens = np.array([900, 1, 60, tables.shape[1] * 16 + 1], dtype=np.int32)  # two new tokens of one; too long
    start = np.array([0, 3, 5, 7, 9], dtype=np.int32)
    args = (t["k"], t["v"], t["ks"], t["vs"], t["tables"], torch.from_numpy(lens).cuda(), torch.from_numpy(start).cuda())
    pkv.pkv_q8_prefill_attention(desc, 0, to_torch(q, "f16"), *args, 3, 0.01, out, ws)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_QUERY_RANGE
    got = as_f64(out)
    assert np.all(got[3:5] == 7.0) and np.all(got[7:] == 7.0)
    for row, s, p in [(0, 0, 897), (2, 0, 899), (5, 2, 58), (6, 2, 59)]:
        want, tol, _, _ = R.decode(qf[row:row + 1], np.nan_to_num(kf), np.nan_to_num(vf), tables[s:s + 1], np.array([p + 1]),
                                   0.01, "f16", 2.0 ** -11)
        assert np.all(np.abs(got[row] - want[0]) <= tol[0])
    args[5].fill_(60)
    pkv.pkv_q8_prefill_attention(desc, 0, to_torch(q, "f16"), *args, 2, 0.01, out, ws)  # the first has three
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_QUERY_RANGE


def test_chunk_paths_agree():
    """The same rows as one long chunk (widened) and as short ones (by groups): equal within both roundings."""
    d, G, n_kv, length = 128, 4, 2, 600
    desc, t, _, kf, vf, tables, lens = q8_case("bf16", [length], G * n_kv, n_kv, d, seed=23)
    q, _ = values(np.random.default_rng(9), (500, G * n_kv, d), "bf16")
    whole, launches = prefill(desc, t, q, lens, [500], 0.01, "bf16")
    assert launches == 2
    for end in (length, length - 64):                     # the last tokens of a shorter context are the chunk
        at = 500 - (length - end) - 5
        part, launches = prefill(desc, t, q[at:at + 5], [end], [5], 0.01, "bf16")
        assert launches == 1
        # bf16 weights against fp16 ones, both outputs rounded to bf16
        size = np.abs(np.nan_to_num(vf)).max()
        assert np.all(np.abs(part - whole[at:at + 5]) <= (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -8) * size)


def test_the_largest_batch_and_one_more():
    """65,535 sequences of a token or two (every CTA scans their lengths), one refused beyond."""
    n, d, n_kv = 65535, 64, 1
    desc = pkv.make_desc("bf16", 1, n, 2, n_kv, d)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((2 * n, n_kv, d), device="cuda", generator=g).bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(pkv.pool_shape(desc), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = torch.zeros((2, *pkv.scale_shape(desc)), device="cuda")
    slots = (torch.arange(n, device="cuda") * 16)[:, None] + torch.arange(2, device="cuda")
    pkv.pkv_q8_append(desc, 0, k, v, slots.reshape(-1), kc, vc, ks, vs)
    lens = (torch.arange(n, device="cuda") % 3).int()
    tables = torch.arange(n, device="cuda").int()[:, None].contiguous()
    q = torch.randn((n, 2, d), device="cuda", generator=g).bfloat16()
    out = torch.full_like(q, float("nan"))
    scores = torch.zeros((n, n_kv, 16), device="cuda")
    ws = pkv.alloc_q8_workspace(desc, n, 1, scored=True)
    pkv.pkv_q8_decode_attention(desc, 0, q, kc, vc, ks, vs, tables, lens, 0.125, out, ws, scores=scores)
    assert pkv.pkv_get_device_status() == 0
    kf, vf = kc.float()[0] * ks[0][..., None, None], vc.float()[0] * vs[0][..., None, None]
    z = torch.einsum("nhd,njd->nhj", q.double(), kf[:, 0, :2].double()) * 0.125
    z = z.masked_fill(torch.arange(2, device="cuda") >= lens[:, None, None], -torch.inf)
    w = torch.nan_to_num(torch.softmax(z, -1))
    want = torch.einsum("nhj,njd->nhd", w, vf[:, 0, :2].double())
    # two terms: the weights' rounding and the output's (2^-11, 2^-8), relative to at most sum w |v|
    size = torch.einsum("nhj,njd->nhd", w, vf[:, 0, :2].double().abs())
    assert torch.all((out.double() - want).abs() <= (2.0 ** -11 + 2.0 ** -8 + 2.0 ** -16) * size)
    assert torch.allclose(scores[..., :2].double(), w.sum(1, keepdim=True), rtol=1e-5, atol=1e-7) and not scores[..., 2:].any()
    more = torch.zeros((n + 1, 2, d), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
        pkv.pkv_q8_decode_attention(desc, 0, more, kc, vc, ks, vs, torch.zeros((n + 1, 1), dtype=torch.int32, device="cuda"),
                                    torch.zeros(n + 1, dtype=torch.int32, device="cuda"), 1.0, more)


def test_offsets_past_32_bits():
    """Pools of over 2^32 bytes, the sequences in their last blocks: append, copy, decode and a chunk give
    what a small pool gives."""
    d, n_kv, G, n = 256, 8, 1, 2
    lens = np.array([100, 37], dtype=np.int32)
    small, big = 12, 140_000                              # 140,000 * 8 * 16 * 256 = 4.6e9 bytes
    rng = np.random.default_rng(4)
    x, y = (to_torch(W.normal_values(rng, (137, n_kv, d), "bf16"), "bf16") for _ in range(2))
    q = to_torch(W.normal_values(rng, (n, n_kv * G, d), "bf16"), "bf16")
    got = []
    for nb in (small, big):
        desc = pkv.make_desc("bf16", 1, nb, n_kv * G, n_kv, d)
        kc, vc = (torch.zeros(pkv.pool_shape(desc), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = torch.zeros((2, *pkv.scale_shape(desc)), device="cuda")
        ids = np.arange(nb - 12, nb)
        tables = np.full((n, 7), -1, dtype=np.int32)
        tables[0], tables[1, :3] = ids[[3, 1, 7, 11, 5, 0, 10]], ids[[2, 9, 4]]
        slots = np.concatenate([tables[s][np.arange(c) // 16].astype(np.int64) * 16 + np.arange(c) % 16 for s, c in enumerate(lens)])
        pkv.pkv_q8_append(desc, 0, x, y, torch.from_numpy(slots).cuda(), kc, vc, ks, vs)
        pkv.pkv_q8_copy_blocks(desc, kc, vc, ks, vs, torch.tensor([[ids[4], ids[6]]], dtype=torch.int32, device="cuda"))
        tables[1, 2] = ids[6]
        tt, tl = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
        out = torch.empty_like(q)
        pkv.pkv_q8_decode_attention(desc, 0, q, kc, vc, ks, vs, tt, tl, 0.0625, out, pkv.alloc_q8_workspace(desc, n, 7))
        chunk = torch.empty_like(q)
        pkv.pkv_q8_prefill_attention(desc, 0, q, kc, vc, ks, vs, tt, tl, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), 1,
                                     0.0625, chunk, pkv.alloc_q8_prefill_workspace(desc))
        wide = torch.empty((137, n_kv * G, d), dtype=torch.bfloat16, device="cuda")
        pkv.pkv_q8_prefill_attention(desc, 0, x.contiguous(), kc, vc, ks, vs, tt, tl,
                                     torch.tensor([0, 100, 137], dtype=torch.int32, device="cuda"), 100, 0.0625, wide,
                                     pkv.alloc_q8_prefill_workspace(desc))
        assert pkv.pkv_get_device_status() == 0
        got.append((out, chunk, wide))
        del kc, vc
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def long_chunk(dtype, seed, spread=3, d=128, G=8, n_kv=2, length=600, tokens=500):
    """A chunk that is widened (two launches), its queries and the pools: (call(scale, n), case, qf). call
    attends to the last n tokens."""
    desc, t, _, kf, vf, tables, lens = q8_case(dtype, [length], G * n_kv, n_kv, d, seed=seed, spread=spread)
    q, qf = values(np.random.default_rng(seed), (tokens, G * n_kv, d), dtype)

    def call(scale, n=tokens):
        return prefill(desc, t, q[-n:], lens, [n], scale, dtype)
    return call, (desc, t, kf, vf, tables, lens), qf


def check_chunk(got, qf, k, v, tables, length, scale, dtype, step, factor=1, every=7, skip=None):
    """Every `every`-th token of a chunk at the end of one sequence against the restatement; elements of `skip`
    are not looked at."""
    n = len(got)
    for i in sorted({0, 1, n - 2, n - 1} | set(range(0, n, every))):
        want, tol, _, _ = R.decode(qf[i - n:i - n + 1 or None], k, v, tables, np.array([length - n + i + 1]), scale, dtype, step)
        assert np.all((np.abs(got[i] - want[0]) <= factor * tol[0]) | (False if skip is None else skip[i])), i


@pytest.mark.parametrize("scale", [-0.02, 0.0, -0.0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunks_of_any_scale(dtype, scale):
    """A softmax scale of zero (equal weights) or below, over a long chunk and a short one."""
    call, (desc, t, kf, vf, tables, lens), qf = long_chunk(dtype, seed=31)
    assert call(0.02)[1] == 2                              # with a positive scale the long chunk is widened
    for n in (500, 3):
        got, launches = call(scale, n)
        assert launches == 1 and pkv.pkv_get_device_status() == 0
        check_chunk(got, qf, np.nan_to_num(kf), np.nan_to_num(vf), tables, 600, scale, dtype, 2.0 ** -11)


@pytest.mark.parametrize("dtype,d,G,n_kv", [("f16", 64, 8, 1), ("f16", 128, 8, 1), ("f16", 256, 8, 1), ("bf16", 64, 8, 1)])
def test_chunks_of_many_small_weights(dtype, d, G, n_kv):
    """One key outweighs each of 40,000 others by 2^23.4 and only the others have values: a long chunk (widened)
    and a short one give their sum, each weight rounded by half a step of its own."""
    c, tokens = 40000, 600
    nb = c // BLOCK
    desc = pkv.make_desc(dtype, 1, nb, G * n_kv, n_kv, d)
    kc, vc = np.zeros((1, nb, n_kv, BLOCK, d), dtype=np.uint8), np.full((1, nb, n_kv, BLOCK, d), 0x50, dtype=np.uint8)
    kc[0, nb // 2, :, 3], vc[0, nb // 2, :, 3] = 0x41, 0                # 2.25 and 0; the other values are 8
    ks, vs = np.ones((2, 1, nb, n_kv), dtype=np.float32)
    scale = 16.25 / (2.25 * d)                                          # a logit of 16.25 = 23.44 ln 2
    t = dict(k=codes_to_torch(kc), v=codes_to_torch(vc), ks=torch.from_numpy(ks).cuda(), vs=torch.from_numpy(vs).cuda(),
             tables=torch.arange(nb, dtype=torch.int32, device="cuda")[None])
    ones = torch.ones((tokens, G * n_kv, d), dtype=pkv.torch_dtype(dtype))
    want, tol, _, _ = R.decode(np.ones((1, G * n_kv, d)), R.widen(kc[0], ks[0]), R.widen(vc[0], vs[0]),
                               np.arange(nb, dtype=np.int32)[None], np.array([c]), scale, dtype,
                               max(2.0 ** -11, R.HALF_STEP[dtype]))
    assert np.all(tol < 0.02 * want)
    for n, launches in ((tokens, 2), (1, 1)):
        got, count = prefill(desc, t, to_host(ones[:n], dtype), [c], [n], scale, dtype)
        assert count == launches
        assert np.all(np.abs(got[-1] - want[0]) <= 2 * tol[0])


def odd_scales(t, tables, names=("ks", "vs")):
    """Scales in (0, 1/32) that are no powers of two, in place; returns both pools widened in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in names:
        t[n].copy_((torch.rand(t[n].shape, device="cuda", generator=g) + 0.01) / 32.5)
    return [np.nan_to_num(R.widen(codes_to_host(t[a])[0], t[b][0].double().cpu().numpy())) for a, b in (("k", "ks"), ("v", "vs"))]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunks_of_any_block_scale(dtype):
    """Block scales that are no powers of two: exact in a short chunk; in a long one K and V are rounded to the
    activations' type first, by half a step h of each element. A logit is then off by at most dz = h |scale|
    sum|q||k|, a weight by a factor exp(+-2 dz), the output by that and h, relative to sum w|v|."""
    scale = 0.01
    call, (desc, t, _, _, tables, lens), qf = long_chunk(dtype, seed=33)
    k, v = odd_scales(t, tables)
    h = R.HALF_STEP[dtype]
    for n, launches in ((500, 2), (3, 1)):
        got, count = call(scale, n)
        assert count == launches and pkv.pkv_get_device_status() == 0
        for i in sorted({0, n - 1} | set(range(0, n, 31))):
            q, c = qf[i - n:i - n + 1 or None], 600 - n + i + 1
            want, tol, _, _ = R.decode(q, k, v, tables, np.array([c]), scale, dtype, 2.0 ** -11 if n == 3 else h)
            more = np.zeros_like(tol[0])
            for head in range(q.shape[1] if launches == 2 else 0):
                kg, vg = R.rows_of(k, tables[0], c, head // 8), R.rows_of(v, tables[0], c, head // 8)
                _, w = R.attend(q[0, head], kg, vg, scale)
                dz = h * scale * (np.abs(kg) @ np.abs(q[0, head])).max()
                more[head] = (np.expm1(2 * dz) + h * np.exp(2 * dz)) * (w @ np.abs(vg))
            assert np.all(np.abs(got[i] - want[0]) <= 2 * tol[0] + more), i


@pytest.mark.parametrize("dtype,size,top", [("f16", 200.0, 65504.0)])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_chunks_of_block_scales_out_of_range(dtype, size, top, which):
    """Codes times scale beyond the activations' type: a short chunk takes them as they are, a long one reads
    the type's largest number and says so. Rows and blocks that no sequence uses are not judged. (Rows near
    bf16's largest number overflow the fp32 sums of any order, so there is nothing to compare for bf16.)"""
    call, (desc, t, kf, vf, tables, lens), qf = long_chunk(dtype, seed=34, spread=0)
    name = which[0]
    codes = t[name].view(torch.uint8)
    codes[(codes & 127) >= 0x78] = 0x76                    # up to 224 (size * 224 < top), stale NaN rows too
    t[which].fill_(size)
    last, used = int(tables[0, 599 // 16]), 600 % 16
    codes[0, last, :, used:] = 0x7E                        # 448 behind the context
    spare = next(b for b in range(desc.num_blocks) if b not in tables[0])
    codes[0, spare] = 0x7E
    scale = 0.01 if which == "vs" else 0.01 / size / 64    # logits of some size
    pools = {"ks": np.nan_to_num(kf), "vs": np.nan_to_num(vf)}

    def true_pool():
        c = codes_to_host(t[name])[0].copy()
        c[last, :, used:] = 0
        return R.VALUES[c] * size
    pools[which] = true_pool()
    for n, launches in ((500, 2), (3, 1)):
        got, count = call(scale, n)
        assert count == launches and pkv.pkv_get_device_status() == 0
        check_chunk(got, qf, pools["ks"], pools["vs"], tables, 600, scale, dtype, max(2.0 ** -11, R.HALF_STEP[dtype]), 2, every=61)
    codes[0, int(tables[0, 3]), 0, 2, 7] = 0x7E            # one element of 448 * size
    codes[0, int(tables[0, 3]), 1, 2, 9] = 0xFE
    pools[which] = true_pool()
    got, count = call(scale, 3)
    assert count == 1 and pkv.pkv_get_device_status() == 0
    check_chunk(got, qf, pools["ks"], pools["vs"], tables, 600, scale, dtype, max(2.0 ** -11, R.HALF_STEP[dtype]), 2)
    got, count = call(scale)
    assert count == 2 and pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_SCALE
    pools[which] = np.clip(pools[which], -top, top)
    check_chunk(got, qf, pools["ks"], pools["vs"], tables, 600, scale, dtype, max(2.0 ** -11, R.HALF_STEP[dtype]), 2, every=61)


@pytest.mark.parametrize("dtype,d,G", [("f16", 64, 8), ("bf16", 64, 4), ("f16", 128, 8), ("bf16", 128, 2), ("f16", 256, 4),
                                       ("bf16", 256, 8)])
def test_long_chunks_are_causal_about_nan(dtype, d, G):
    """NaN codes of V in a long chunk: in a row of the cache before it, in rows of new tokens (the first, one in
    the middle, the last), in rows behind the context, and in a block that another sequence's chunk ends before.
    Each reaches the tokens that see its row, in its dim and head, and the next call over clean rows is clean."""
    n_kv, tokens, length = 2, 500, 620
    scale = 1 / np.sqrt(d) / 16
    rng = np.random.default_rng(d + G)
    desc, t, _, kf, vf, tables, lens = q8_case(dtype, [length, 560, 300], G * n_kv, n_kv, d, seed=35)
    tables[1] = tables[0]                                  # the second sequence holds the same rows, fewer of them
    t["tables"].copy_(torch.from_numpy(np.ascontiguousarray(tables)))
    counts = [tokens, tokens, 250]
    q, qf = values(rng, (sum(counts), G * n_kv, d), dtype)
    clean, launches = prefill(desc, t, q, lens, counts, scale, dtype)
    assert launches == 2 and pkv.pkv_get_device_status() == 0 and np.isfinite(clean).all()
    keep = t["v"].clone()
    bad = [(0, 0, 50, 3), (0, 1, 121, d - 1), (0, 0, 400, 17), (0, 1, 590, 20), (0, 0, 619, 40), (2, 1, 299, 1)]
    codes = t["v"].view(torch.uint8)
    for s, g, p, dim in bad:
        codes[0, int(tables[s, p // 16]), g, p % 16, dim] = 0xFF if p % 2 else 0x7F
    got, launches = prefill(desc, t, q, lens, counts, scale, dtype)
    assert launches == 2 and pkv.pkv_get_device_status() == 0
    want = np.zeros(got.shape, dtype=bool)
    row = 0
    v = R.widen(codes_to_host(t["v"])[0], t["vs"][0].double().cpu().numpy())
    for s, n in enumerate(counts):
        pos = int(lens[s]) - n + np.arange(n)
        for owner, g, p, dim in bad:
            if owner == s or (owner == 0 and s == 1 and p < lens[1]):
                want[row:row + n, g * G:(g + 1) * G, dim] |= (pos >= p)[:, None]
        check_chunk(np.where(want[row:row + n], 0.0, got[row:row + n]), qf[row:row + n],
                    *no_nan(kf, v), tables[s:s + 1], int(lens[s]), scale, dtype, R.HALF_STEP[dtype], 2,
                    skip=want[row:row + n], every=67)
        row += n
    assert np.array_equal(np.isnan(got), want) and want.any() and not want.all()
    t["v"].copy_(keep)
    again, _ = prefill(desc, t, q, lens, counts, scale, dtype)
    assert np.array_equal(again, clean)


def no_nan(*pools):
    return [np.nan_to_num(p) for p in pools]


def test_a_nan_does_not_outlive_its_call():
    """The words that tell of NaN codes are zero again behind the call: the same workspace serves a long chunk
    with one, a clean long chunk, decode and a graph of both kinds."""
    dtype, d, G, n_kv, tokens, length = "f16", 128, 8, 2, 500, 600
    desc, t, _, kf, vf, tables, lens = q8_case(dtype, [length], G * n_kv, n_kv, d, seed=36)
    q, _ = values(np.random.default_rng(36), (tokens, G * n_kv, d), dtype)
    tq, start = to_torch(q, dtype), torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    ws = pkv.alloc_q8_prefill_workspace(desc)
    dirty = t["v"].clone()
    dirty.view(torch.uint8)[0, int(tables[0, 20]), 1, 5, 7] = 0x7F

    def call(v, out):
        pkv.pkv_q8_prefill_attention(desc, 0, tq, t["k"], v, t["ks"], t["vs"], t["tables"], t["lens"], start, tokens, 0.01,
                                     out, ws)
    clean, first = torch.empty_like(tq), torch.empty_like(tq)
    call(t["v"], clean)
    call(dirty, first)
    assert not ws[:COUNTERS].view(torch.int32).any()
    nan = torch.isnan(first)
    assert nan[325 - 100:, G:, 7].all() and int(nan.sum()) == (tokens - 225) * G
    again = torch.empty_like(tq)
    call(t["v"], again)
    assert torch.equal(again, clean)
    outs = [torch.empty_like(tq) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(dirty, outs[0])
        call(t["v"], outs[1])
        call(dirty, outs[2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], clean)
    for o in (outs[0], outs[2]):
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))
    assert not ws[:COUNTERS].view(torch.int32).any() and pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("lens,max_blocks", [([301], 19), ([9000, 40, 2500], 700), ([700, 1300, 64, 2048] * 6, 128)])
@pytest.mark.parametrize("d,G", [(64, 8), (128, 1), (256, 4)])
def test_results_repeat_bit_for_bit(lens, max_blocks, d, G):
    """Outputs and sums of decode and of chunks do not depend on the order in which CTAs end: repeated beside
    another stream's work that takes SMs away at other times."""
    n_kv = 4
    desc, t, qf, kf, vf, tables, ln = q8_case("bf16", lens, G * n_kv, n_kv, d, seed=51, max_blocks=max_blocks)
    counts = [min(c, 3) for c in lens]
    q, _ = values(np.random.default_rng(51), (sum(counts), G * n_kv, d), "bf16")
    other, busy = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda")
    torch.cuda.synchronize()
    want = None
    for i in range(12):
        if i:
            with torch.cuda.stream(other):
                for _ in range(i % 4 * 8):
                    busy = busy @ busy * 1e-3
        scores = torch.zeros((len(lens), n_kv, max_blocks * BLOCK), device="cuda")
        got = [run_decode(desc, t, 0.02, scores), scores, torch.from_numpy(prefill(desc, t, q, ln, counts, 0.02, "bf16")[0])]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    assert pkv.pkv_get_device_status() == 0


def test_codes_and_workspaces_on_the_host_are_refused_before_launch():
    """Page-locked host memory in the place of codes (decode, short and long chunks) or of a long chunk's
    workspace: PKV_ERR_INVALID_ARG, nothing launched. Through the C entry points; the binding takes no such tensor."""
    import ctypes
    desc, t, _, kf, vf, tables, lens = q8_case("f16", [600], 16, 2, 128, seed=37)
    host = t["k"].view(torch.uint8).cpu().pin_memory()
    q = torch.zeros((500, 16, 128), dtype=torch.float16, device="cuda")
    out, ws = torch.full_like(q, 3.0), pkv.alloc_q8_prefill_workspace(desc)
    host_ws = torch.zeros(ws.numel(), dtype=torch.float32).pin_memory()
    dws = pkv.alloc_q8_workspace(desc, 1, tables.shape[1])
    codes = [t["k"].data_ptr(), t["v"].data_ptr()]
    scales = [t["ks"].data_ptr(), t["vs"].data_ptr()]
    L, d = pkv.lib(), ctypes.byref(desc)
    before = pkv.pkv_launch_count()

    def chunk(n, codes, w):
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        return L.pkv_q8_prefill_attention(d, 0, q.data_ptr(), *codes, *scales, t["tables"].data_ptr(), tables.shape[1],
                                          t["lens"].data_ptr(), starts.data_ptr(), 1, n, n, 0.1, out.data_ptr(), w.data_ptr(),
                                          ws.nbytes, None)
    for i in range(2):
        bad = list(codes)
        bad[i] = host.data_ptr()
        assert chunk(3, bad, ws) == chunk(500, bad, ws) == pkv.PKV_ERR_INVALID_ARG
        assert L.pkv_q8_decode_attention(d, 0, q.data_ptr(), *bad, *scales, t["tables"].data_ptr(), tables.shape[1],
                                         t["lens"].data_ptr(), 1, 0.1, out.data_ptr(), None, 0,
                                         None if dws is None else dws.data_ptr(), 0 if dws is None else dws.nbytes,
                                         None) == pkv.PKV_ERR_INVALID_ARG
    assert chunk(500, codes, host_ws) == pkv.PKV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert pkv.pkv_launch_count() == before and torch.all(out == 3.0)
    assert chunk(500, codes, ws) == pkv.PKV_OK and pkv.pkv_launch_count() == before + 2
    assert chunk(3, codes, ws) == pkv.PKV_OK and pkv.pkv_launch_count() == before + 3
    assert pkv.pkv_get_device_status() == 0


def test_calls_at_once_on_two_streams():
    """Appends, decode with summed weights, short and long chunks of two caches on two streams, each with its own
    workspaces, give what they give one after the other."""
    dtype, d, G, n_kv = "bf16", 128, 8, 2
    cases = []
    for i, lens in enumerate(([4000, 600, 33], [900, 5200])):
        desc, t, _, kf, vf, tables, ln = q8_case(dtype, lens, G * n_kv, n_kv, d, seed=60 + i, max_blocks=400)
        n = len(lens)
        long = min(lens[0], 500)
        starts = [torch.tensor([0, m] + [m] * (n - 1), dtype=torch.int32, device="cuda") for m in (3, long)]
        rows = torch.randn((4, n_kv, d), device="cuda").bfloat16()
        slots = torch.tensor([int(tables[1, 0]) * 16 + j for j in range(4)], device="cuda")
        qs = [torch.randn((m, G * n_kv, d), device="cuda").bfloat16() for m in (3, long)]
        cases.append((desc, t, n, starts, rows, slots, qs, pkv.alloc_q8_workspace(desc, n, 400, scored=True),
                      pkv.alloc_q8_prefill_workspace(desc)))
    torch.cuda.synchronize()

    def queue(case, times):
        desc, t, n, starts, rows, slots, qs, ws, pws = case
        out, scores = torch.empty_like(t["q"]), torch.zeros((n, n_kv, 6400), device="cuda")
        outs = [torch.empty_like(x) for x in qs]
        for _ in range(times):
            pkv.pkv_q8_append(desc, 0, rows, rows, slots, t["k"], t["v"], t["ks"], t["vs"])
            pkv.pkv_q8_decode_attention(desc, 0, t["q"], t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["lens"], 0.02, out, ws,
                                        scores=scores)
            for x, o, s in zip(qs, outs, starts):
                pkv.pkv_q8_prefill_attention(desc, 0, x, t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["lens"], s,
                                             x.shape[0], 0.02, o, pws)
        return [out, scores, *outs]
    want = [queue(c, 5) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(queue(c, 5))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    assert pkv.pkv_get_device_status() == 0
