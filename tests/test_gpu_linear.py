"""Linear attention over a pool of states, on the GPU against the recurrence in 64 bits (tests/linear_oracle.py)."""
import math

import numpy as np
import pytest
import torch

from linear_oracle import linear
from paged_kv_cache_258_gb300 import pkv

pytestmark = pytest.mark.gpu
SCALE = 0.125


def inputs(dtype, lens, n_qk, n_v, dk, dv, gates="token", seed=0, behind=3, size=1.0):
    """Packed rows (with `behind` NaN rows of no sequence), decays, states of len(lens) + 2 slots."""
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)
    t = pkv.torch_dtype(dtype)
    pad = lambda x: torch.cat([x, torch.full((behind, *x.shape[1:]), float("nan"))]).to(t).cuda()
    q, k = (pad(torch.randn((T, n_qk, dk), generator=g) * size) for _ in range(2))
    v = pad(torch.randn((T, n_v, dv), generator=g) * size)
    if gates == "token":
        d = -torch.exp(3 * torch.randn((T + behind, n_v), generator=g) - 3)
        if T > 5:
            d[T // 3, 0] = -math.inf          # forgets
            d[T // 2] = 0.0
        d[T:] = float("nan")
        d = d.cuda()
    elif gates == "head":
        d = -torch.exp(-8 * torch.rand(n_v, generator=g)).cuda()
    else:
        d = None
    state = torch.randn((2, n + 2, n_v, dk, dv), generator=g).cuda()
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return q, k, v, d, state, starts


def per_token(d, v):
    if d is None:
        return torch.zeros(v.shape[:2])
    return d.expand(v.shape[0], v.shape[1]) if d.dim() == 1 else d


def run(dtype, q, k, v, d, state, src, dst, starts, layer=1, decode=False, longest=None, n_tokens=None):
    desc = pkv.make_linear_desc(dtype, *state.shape[:2], q.shape[1], v.shape[1], q.shape[2], v.shape[2])
    out = torch.full_like(v, 7.0)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    if decode:
        pkv.pkv_linear_decode(desc, layer, q, k, v, d, state, i32(src), i32(dst), SCALE, out)
    else:
        longest = int(np.diff(starts).max(initial=0)) if longest is None else longest
        ws = pkv.alloc_linear_prefill_workspace(desc, len(src), q.shape[0], longest)
        if ws is not None:
            ws.fill_(float("nan"))
        pkv.pkv_linear_prefill(desc, layer, q, k, v, d, state, i32(src), i32(dst), i32(starts), longest, SCALE, out, ws)
    return out


def check(dtype, q, k, v, d, state, src, dst, starts, decode=False):
    was = state.clone()
    out = run(dtype, q, k, v, d, state, src, dst, starts, decode=decode)
    want, tol, after, after_tol = linear(q, k, v, per_token(d, v), was[1], src, dst, starts, SCALE, dtype)
    T = int(starts[-1])
    got = out.double().cpu()
    assert torch.all((got[:T] - want[:T]).abs() <= tol[:T])
    assert torch.all(out[T:] == 7.0)
    assert torch.all((state[1].double().cpu() - after).abs() <= after_tol)
    assert torch.equal(state[0], was[0])
    assert pkv.pkv_get_device_status() == 0
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("group,gates", [(1, "head"), (3, "token"), (2, "none")])
def test_decode_matches(dtype, dk, dv, group, gates):
    n = 6
    q, k, v, d, state, starts = inputs(dtype, [1] * n, 2, 2 * group, dk, dv, gates, seed=dk + dv + group, behind=0)
    check(dtype, q, k, v, d, state, [3, -1, 0, 0, 5, 1], [3, 7, 6, -1, 2, 1], starts, decode=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_decode_of_many(dtype):
    """More (sequence, head) pairs than two for each multiprocessor: whole rows of the state a CTA."""
    n = 40
    q, k, v, d, state, starts = inputs(dtype, [1] * n, 10, 10, 128, 128, seed=1, behind=0)
    src = list(np.random.default_rng(0).permutation(n + 2)[:n])
    check(dtype, q, k, v, d, state, src, src, starts, decode=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1], [5], [0, 3, 0, 9], [16, 17], [70, 2, 33], [127], [128], [129, 1], [300, 64, 0, 257]])
def test_prefill_matches(dtype, dk, dv, lens):
    q, k, v, d, state, starts = inputs(dtype, lens, 1, 3, dk, dv, "token", seed=sum(lens) + dk)
    n = len(lens)
    check(dtype, q, k, v, d, state, [i if i % 2 == 0 else -1 for i in range(n)], [n + 1 - i if i < 3 else 1 for i in range(n)], starts)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gates", ["head", "none"])
@pytest.mark.parametrize("group", [1, 2])
def test_prefill_decays_of_each_kind(dtype, gates, group):
    q, k, v, d, state, starts = inputs(dtype, [200, 140], 2, 2 * group, 64, 64, gates, seed=group)
    check(dtype, q, k, v, d, state, [0, 1], [0, 1], starts)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prefill_of_many(dtype):
    q, k, v, d, state, starts = inputs(dtype, [30 + i % 7 for i in range(80)], 4, 4, 64, 128, seed=2)
    check(dtype, q, k, v, d, state, list(range(80)), list(range(80)), starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv,n_v", [(128, 128, 2), (128, 64, 1), (64, 128, 1)])
def test_prefill_of_one_long_sequence(dtype, dk, dv, n_v):
    """Few heads and many tokens: the sequence is shared out along its length."""
    q, k, v, d, state, starts = inputs(dtype, [5000, 1, 3900], 1, n_v, dk, dv, "token", seed=4)
    d.clamp_(min=-0.05)
    check(dtype, q, k, v, d, state, [1, -1, 0], [1, 3, 0], starts)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -9, 20.0])
def test_small_and_large_values(dtype, size):
    """Weights and states far below 1, and pairs' weights and states past fp16's largest number."""
    q, k, v, d, state, starts = inputs(dtype, [333], 1, 2, 128, 64, "head", seed=6, size=size)
    state *= size ** 2
    q[:200] *= 1 / size / 8                       # (results within fp16; the last rows' are past it for size 20)
    out = check(dtype, q[:203], k[:203], v[:203], d, state, [0], [0], np.array([0, 200], dtype=np.int32))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_growing_decays(dtype):
    q, k, v, d, state, starts = inputs(dtype, [260], 1, 1, 64, 64, "token", seed=7)
    d[::3] = 0.04
    d[d == -math.inf] = -1.0
    check(dtype, q, k, v, d, state, [0], [0], starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("length", [40, 300])
def test_non_finite_values_reach_later_tokens_only(dtype, length):
    """NaN or infinity in v of a token: its column, from that token on; in q: that token; in k: from there on."""
    lens = [length, 20]
    q, k, v, d, state, starts = inputs(dtype, lens, 1, 2, 64, 64, "head", seed=8)
    base = run(dtype, q, k, v, d, state.clone(), [0, 1], [0, 1], starts)
    T = sum(lens)
    assert torch.isfinite(base[:T]).all()
    for value in (float("nan"), float("inf")):
        at = length - 9
        v2 = v.clone()
        v2[at, 1, 5] = value
        st = state.clone()
        got = run(dtype, q, k, v2, d, st, [0, 1], [0, 1], starts)
        touched = torch.zeros_like(got, dtype=torch.bool)
        touched[at:length, 1, 5] = True
        assert not torch.isfinite(got[touched]).any()
        assert torch.equal(got[~touched], base[~touched])
        assert not torch.isfinite(st[1, 0, 1, :, 5]).any() and torch.isfinite(st[1, 0, 1, :, :5]).all()
        k2 = k.clone()
        k2[at, 0, 3] = value
        got = run(dtype, q, k2, v, d, state.clone(), [0, 1], [0, 1], starts)
        assert torch.equal(got[:at], base[:at]) and torch.equal(got[length:T], base[length:T])
        assert not torch.isfinite(got[at:length]).any()
        q2 = q.clone()
        q2[at, 0, 3] = value
        got = run(dtype, q2, k, v, d, state.clone(), [0, 1], [0, 1], starts)
        assert torch.equal(got[:at], base[:at]) and torch.equal(got[at + 1:T], base[at + 1:T])
        assert not torch.isfinite(got[at]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_give_what_the_whole_gives(dtype):
    """A prompt in three chunks and then token by token: each piece within the tolerance of the whole recurrence."""
    T = 310
    q, k, v, d, state, starts = inputs(dtype, [T], 2, 4, 128, 64, "token", seed=9, behind=0)
    want, tol, after, after_tol = linear(q, k, v, d, state[1], [2], [2], starts, SCALE, dtype)
    outs = []
    for a, b in ((0, 130), (130, 137), (137, 300)):
        outs.append(run(dtype, q[a:b], k[a:b], v[a:b], d[a:b], state, [2], [2], np.array([0, b - a])))
    for a in range(300, T):
        outs.append(run(dtype, q[a:a + 1], k[a:a + 1], v[a:a + 1], d[a:a + 1], state, [2], [2], None, decode=True))
    assert torch.all((torch.cat(outs).double().cpu() - want).abs() <= tol)
    assert torch.all((state[1].double().cpu() - after).abs() <= after_tol)


def test_slow_decays_last():
    """A decay of 2^-14 a token over 3,000 tokens, token by token: exp(g) rounded to fp32 would be off by up to
    3,000 * 2^-25 = 9e-5 of what is left; (2 n + 16) 2^-24 would allow 3.6e-4. Here: every rounding counted, 3,000
    independent ones of at most half a step, sqrt(3,000) * 2^-24 * 6 = 2e-5."""
    n = 3000
    q, k, v, _, state, starts = inputs("f32", [n], 1, 1, 64, 64, "none", seed=10)
    k[:n] *= 0
    d = torch.full((1,), -(2.0 ** -14) * 1.0001, device="cuda")
    was = state.double()
    run("f32", q, k, v, d, state, [0], [0], starts)
    want = was[1, 0] * math.exp(float(d.double()) * n)
    assert ((state[1, 0].double() - want).norm() / want.norm()).item() < 2e-5


@pytest.mark.parametrize("decode", [False, True])
def test_bad_slots_and_ranges_are_skipped(decode):
    lens = [1, 1, 1, 1] if decode else [40, 150, 30, 200]
    q, k, v, d, state, starts = inputs("bf16", lens, 1, 2, 64, 64, "token", seed=11, behind=0)
    was = state.clone()
    src, dst = [0, 6, 2, 3], [0, 1, 60, 3]
    out = run("bf16", q, k, v, d, state, src, dst, starts, decode=decode)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_STATE_SLOT
    good = run("bf16", q, k, v, d, was2 := was.clone(), [0, 1, 2, 3], [0, -1, -1, 3], starts, decode=decode)
    for s in range(4):
        rows = slice(starts[s], starts[s + 1])
        assert torch.equal(out[rows], good[rows] if s in (0, 3) else torch.full_like(out[rows], 7.0))
    assert torch.equal(state, was2)
    if not decode:
        for bad in ([0, 40, 190, 220, 421], [0, 40, 190, 180, 420], [-1, 40, 190, 220, 420]):
            st = was.clone()
            out = run("bf16", q, k, v, d, st, [0, 1, 2, 3], [0, 1, 2, 3], np.array(bad), longest=200)
            assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_QUERY_RANGE
        st = was.clone()
        out = run("bf16", q, k, v, d, st, [0, 1, 2, 3], [0, 1, 2, 3], starts, longest=160)
        assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_QUERY_RANGE
        assert torch.all(out[220:] == 7.0) and torch.equal(st[:, 3], was[:, 3])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_repeats_bit_for_bit_on_another_stream(dtype):
    q, k, v, d, state, starts = inputs(dtype, [700, 20, 129], 2, 6, 128, 128, "token", seed=12)
    a, b = state.clone(), state.clone()
    first = run(dtype, q, k, v, d, a, [0, 1, 2], [0, 1, 2], starts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run(dtype, q, k, v, d, b, [0, 1, 2], [0, 1, 2], starts)
    side.synchronize()
    assert torch.equal(first[:849], second[:849]) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("length", [20, 200])
def test_rows_on_sixteen_byte_boundaries(dtype, length):
    """Every row array starts 16 bytes past a coarser boundary."""
    q, k, v, d, state, starts = inputs(dtype, [length, 3], 1, 2, 64, 128, "head", seed=13)
    want = run(dtype, q, k, v, d, state.clone(), [0, 1], [0, 1], starts)
    step = 16 // q.element_size()

    def shifted(x):
        flat = torch.zeros(x.numel() + step, dtype=x.dtype, device="cuda")
        y = flat[step:].view(x.shape)
        y.copy_(x)
        return y
    desc = pkv.make_linear_desc(dtype, *state.shape[:2], 1, 2, 64, 128)
    out = shifted(torch.full_like(v, 7.0))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    pkv.pkv_linear_prefill(desc, 1, shifted(q), shifted(k), shifted(v), d, state, i32([0, 1]), i32([0, 1]), i32(starts), length,
                           SCALE, out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_captured_and_replayed_with_other_inputs(dtype):
    """Long (shared out), short, and single-token calls in one graph, replayed on other contents of the same buffers."""
    lens = [2000, 40]
    sets = [inputs(dtype, lens, 1, 2, 128, 64, "token", seed=s) for s in (20, 21)]
    q, k, v, d, state, starts = [x.clone() if torch.is_tensor(x) else x for x in sets[0]]
    desc = pkv.make_linear_desc(dtype, *state.shape[:2], 1, 2, 128, 64)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    src, dst, st = i32([0, 1]), i32([2, 3]), i32(starts)
    ws = pkv.alloc_linear_prefill_workspace(desc, 2, q.shape[0], 2000)
    outs = [torch.zeros_like(v) for _ in range(3)]

    def calls():
        pkv.pkv_linear_prefill(desc, 1, q, k, v, d, state, src, dst, st, 2000, SCALE, outs[0], ws)
        pkv.pkv_linear_prefill(desc, 0, q[:6], k[:6], v[:6], d[:6], state, src, dst, i32_small, 3, SCALE, outs[1][:6])
        pkv.pkv_linear_decode(desc, 0, q[:2], k[:2], v[:2], d[:2], state, dst, src, SCALE, outs[2][:2])
    i32_small = i32([0, 3, 6])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    for x in (sets[1], sets[0]):
        for to, frm in zip((q, k, v, d, state), x):
            to.copy_(frm)
        graph.replay()
        got = [o.clone() for o in outs] + [state.clone()]
        for to, frm in zip((q, k, v, d, state), x):
            to.copy_(frm)
        calls()
        T = sum(lens)
        for a, b in zip(got, outs + [state]):
            assert torch.equal(a[:T], b[:T])
    assert pkv.pkv_get_device_status() == 0


def test_two_streams_at_once():
    a, b = (inputs("bf16", [3000], 1, 2, 128, 64, "head", seed=s) for s in (30, 31))
    want = [run("bf16", *x[:4], x[4].clone(), [0], [0], x[5]) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for st, x in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                got.append(run("bf16", *x[:4], x[4].clone(), [0], [0], x[5]))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[:3000], w[:3000])


def test_a_missing_workspace_is_refused():
    q, k, v, d, state, starts = inputs("bf16", [4000], 1, 1, 64, 64, "none", seed=14)
    desc = pkv.make_linear_desc("bf16", *state.shape[:2], 1, 1, 64, 64)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    need = pkv.pkv_linear_prefill_workspace_bytes(desc, 1, 4000, 4000)
    assert need > 0 and pkv.pkv_linear_prefill_workspace_bytes(desc, 1, 100, 100) == 0
    for ws in (None, torch.empty(need - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_linear_prefill(desc, 0, q, k, v, d, state, i32([0]), i32([0]), i32(starts), 4000, SCALE,
                                   torch.empty_like(v), ws)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def test_other_strides_and_types_are_refused():
    q, k, v, d, state, starts = inputs("bf16", [4], 2, 2, 64, 64, "token", seed=15, behind=0)
    desc = pkv.make_linear_desc("bf16", *state.shape[:2], 2, 2, 64, 64)
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = dict(q=q, k=k, v=v, g=d, state=state, src=slots, dst=slots, out=torch.empty_like(v))
    for name, bad in (("q", torch.cat([q, q], 2)[..., :64]), ("k", k.float()), ("v", v[:3]), ("g", d.double()), ("g", d[:, :1]),
                      ("state", state[:1]), ("src", slots.long()), ("dst", slots[:3]), ("out", torch.empty_like(v).transpose(0, 1))):
        a = dict(ok, **{name: bad})
        with pytest.raises(ValueError):
            pkv.pkv_linear_decode(desc, 0, a["q"], a["k"], a["v"], a["g"], a["state"], a["src"], a["dst"], SCALE, a["out"])


def test_offsets_past_32_bits():
    """A slot whose first element lies past 2^31, and a layer past it."""
    n_slots = 1030
    state = torch.zeros((2, n_slots, 64, 128, 128), device="cuda")   # 2^30 elements a layer and more
    q, k, v, d, small, starts = inputs("bf16", [150], 64, 64, 128, 128, "head", seed=16, behind=0)
    first = torch.randn((64, 128, 128), device="cuda")
    small[1, 0] = first
    want = run("bf16", q, k, v, d, small, [0], [1], starts)
    for layer, slot in ((1, n_slots - 1), (1, 1000), (0, n_slots - 1)):
        state[layer, slot] = first
        got = run("bf16", q, k, v, d, state, [slot], [slot], starts, layer=layer)
        assert torch.equal(got, want) and torch.equal(state[layer, slot], small[1, 1])
    one = run("bf16", q[:1], k[:1], v[:1], d, state, [n_slots - 1], [0], None, decode=True)
    two = run("bf16", q[:1], k[:1], v[:1], d, small, [1], [0], None, decode=True)
    assert torch.equal(one, two) and torch.equal(state[1, 0], small[1, 0])


RAGGED = [0, 1, 128, 129, 300, 7, 260, 64]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_more_units_than_the_gpu_holds(dtype, dk, dv):
    """CTAs go on with others' work: short, empty and long sequences one after the other in one CTA, none of which leaves
    anything to the next."""
    n = 24
    q, k, v, d, state, starts = inputs(dtype, [RAGGED[i % 8] for i in range(n)], 4, 8, dk, dv, seed=31)
    src, dst = [i if i % 3 else -1 for i in range(n)], [(i + 5) % n if i % 5 else -1 for i in range(n)]
    src = [x if x < 0 or dst.count(x) == 0 or dst[i] == x else -1 for i, x in enumerate(src)]  # none reads what another writes
    was = state.clone()
    first = check(dtype, q, k, v, d, state, src, dst, starts)
    for _ in range(3):
        again = was.clone()
        assert torch.equal(run(dtype, q, k, v, d, again, src, dst, starts), first) and torch.equal(again, state)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_more_units_than_the_gpu_holds_with_bad_ones_among_them(dtype):
    n = 24
    q, k, v, d, state, starts = inputs(dtype, [RAGGED[i % 8] for i in range(n)], 4, 8, 64, 64, "head", seed=32)
    was, own = state.clone(), list(range(n))
    base = run(dtype, q, k, v, d, state, own, own, starts)
    # sequences 3 and 12 have no such slot: skipped whole
    st, src, dst = was.clone(), list(own), list(own)
    src[3], dst[12] = n + 2, n + 9
    out = run(dtype, q, k, v, d, st, src, dst, starts)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_STATE_SLOT
    for s in range(n):
        rows = slice(int(starts[s]), int(starts[s + 1]))
        assert torch.equal(out[rows], torch.full_like(out[rows], 7.0) if s in (3, 12) else base[rows])
        assert torch.equal(st[1, s], was[1, s] if s in (3, 12) else state[1, s])
    # ranges that end before they start, and longer than said
    bad = starts.copy()
    bad[7] = bad[6] - 1
    out = run(dtype, q, k, v, d, was.clone(), own, own, bad, longest=300)
    assert pkv.pkv_get_device_status() == pkv.PKV_DEV_BAD_QUERY_RANGE
    rows = slice(int(starts[8]), int(starts[n]))
    assert torch.equal(out[rows], base[rows])
    # what is not finite stays in its sequence, and in v in its column
    v2, at = v.clone(), int(starts[12]) + 200
    v2[at, 2, 3] = float("nan")
    st = was.clone()
    out = run(dtype, q, k, v2, d, st, own, own, starts)
    touched = torch.zeros_like(out, dtype=torch.bool)
    touched[at:int(starts[13]), 2, 3] = True
    assert torch.isnan(out[touched]).all() and torch.equal(out[~touched], base[~touched])
    k2 = k.clone()
    k2[int(starts[4]):int(starts[5])] = float("inf")
    out = run(dtype, q, k2, v, d, was.clone(), own, own, starts)
    rest = torch.ones(int(starts[n]), dtype=torch.bool, device="cuda")
    rest[int(starts[4]):int(starts[5])] = False
    assert torch.equal(out[:int(starts[n])][rest], base[:int(starts[n])][rest])
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("dk,dv,n,n_v", [(64, 64, 30, 4), (64, 128, 30, 4), (128, 64, 20, 4), (128, 128, 30, 4), (64, 64, 4, 2),
                                         (128, 128, 8, 3)])
def test_token_after_token_of_some(dtype, dk, dv, n, n_v):
    """Short chunks of every length up to 33, from few (sequence, head) pairs to some for each multiprocessor."""
    lens = [(i * 13) % 34 for i in range(1, n + 1)]
    q, k, v, d, state, starts = inputs(dtype, lens, n_v, n_v, dk, dv, seed=33 + n)
    check(dtype, q, k, v, d, state, list(range(n)), list(range(n)), starts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_token_at_all(dtype):
    """Empty chunks alone: states go from slot to slot, or to zeros."""
    q, k, v, d, state, starts = inputs(dtype, [0, 0, 0], 1, 2, 64, 64, behind=0)
    was = state.clone()
    run(dtype, q, k, v, d, state, [0, -1, 2], [3, 1, -1], starts)
    want = was.clone()
    want[1, 3], want[1, 1] = was[1, 0], 0
    assert torch.equal(state, want) and pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1000, 20, 0, 129, 513], [1025], [1408, 1409]])
def test_segments_of_few_pieces(dtype, dk, dv, lens):
    """Shared out along the longest: others take fewer segments, one, or none; NaN in one stays in it."""
    q, k, v, d, state, starts = inputs(dtype, lens, 2, 2, dk, dv, seed=41 + len(lens))
    n, was = len(lens), state.clone()
    src = [i if i % 2 == 0 else -1 for i in range(n)]
    base = check(dtype, q, k, v, d, state, src, list(range(n)), starts)
    at = lens[0] - 300
    v2 = v.clone()
    v2[at, 1, 5] = float("nan")
    st = was.clone()
    out = run(dtype, q, k, v2, d, st, src, list(range(n)), starts)
    touched = torch.zeros_like(out, dtype=torch.bool)
    touched[at:lens[0], 1, 5] = True
    assert torch.isnan(out[touched]).all() and torch.equal(out[~touched], base[~touched])
    assert torch.isnan(st[1, 0, 1, :, 5]).all() and torch.equal(st[1, 1:], state[1, 1:])
    assert pkv.pkv_get_device_status() == 0


def test_more_units_than_the_gpu_holds_on_two_streams_and_from_graphs():
    """Two such calls at once, and two captured ones replayed in turns: each goes on with its own work only."""
    lens = [RAGGED[i % 8] for i in range(24)]
    own = list(range(24))
    a, b = (inputs("bf16", lens, 4, 8, 64, 128, seed=s) for s in (51, 52))
    T = sum(lens)
    want = []
    for x in (a, b):
        st = x[4].clone()
        want.append((run("bf16", *x[:4], st, own, own, x[5])[:T], st))
    streams = [torch.cuda.Stream() for _ in range(2)]
    states = [[x[4].clone() for x in (a, b)] for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for pair in states:
        for st, x, state in zip(streams, (a, b), pair):
            with torch.cuda.stream(st):
                got.append((run("bf16", *x[:4], state, own, own, x[5])[:T], state))
    torch.cuda.synchronize()
    for i, (out, state) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(state, want[i % 2][1])
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    desc = pkv.make_linear_desc("bf16", 2, 26, 4, 8, 64, 128)
    slots, start = i32(own), i32(a[5])
    graphs, outs, after = [], [], []
    for x in (a, b):
        outs.append(torch.zeros_like(x[2]))
        after.append(x[4].clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pkv.pkv_linear_prefill(desc, 1, *x[:4], after[-1], slots, slots, start, 300, SCALE, outs[-1])
    for _ in range(3):
        for x, state in zip((a, b), after):
            state.copy_(x[4])
        for graph in graphs:
            graph.replay()
        for out, state, w in zip(outs, after, want):
            assert torch.equal(out[:T], w[0]) and torch.equal(state, w[1])
    assert pkv.pkv_get_device_status() == 0
