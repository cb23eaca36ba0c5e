"""Linear attention where numbers leave the range of the rows' type, on the GPU against the recurrence in 64 bits: decays of
both signs, keys and queries that single a token out, states with columns of very different size, many tokens that forget."""
import math

import numpy as np
import pytest
import torch

from linear_oracle import HALF_STEP, linear
from paged_kv_cache_258_gb300 import pkv
from test_gpu_linear import RAGGED, SCALE, inputs, per_token, run

pytestmark = pytest.mark.gpu
LARGEST = {"f32": 3.4028234e38, "f16": 65504.0, "bf16": 3.3895e38}


def sums_error(g, starts):
    """Relative error of a weight exp(G_i - G_j) that comes from its sum in fp32. A log decay is turned to base 2 (half a
    step: 2^-24 |g|), then summed over a piece of 128 tokens: five additions of a scan, up to four of blocks and three
    differences, each off by half a step of a partial sum, which is at most M, the largest sum between two tokens of
    the piece: 12 * 2^-24 M. Both count once for each piece that a term passes. What passes a token that all but forgets
    (below -60) has no part in the bounds, nor have those. Returned for each sequence."""
    out = []
    for a, b in zip(starts[:-1], starts[1:]):
        x = g[a:b].double().cpu()
        x = torch.where(x < -60.0, 0.0, x)
        total = x.abs().sum(0)
        for p in range(0, b - a, 128):
            f = torch.cumsum(torch.cat([torch.zeros_like(x[:1]), x[p:p + 128]]), 0)
            total = total + 12 * (f.max(0).values - f.min(0).values)
        out.append(float(total.max()) * 2.0 ** -24 if b > a else 0.0)
    return out


def check(dtype, q, k, v, d, state, src, dst, starts):
    """As in test_gpu_linear, where the tolerance also holds the sums' errors, and a result past the type's largest number
    is infinite."""
    was = state.clone()
    out = run(dtype, q, k, v, d, state, src, dst, starts)
    g = per_token(d, v)
    want, tol, after, after_tol = linear(q, k, v, g, was[1], src, dst, starts, SCALE, dtype)
    reach, _, most, _ = linear(q.abs(), k.abs(), v.abs(), g, was[1].abs(), src, dst, starts, SCALE, dtype)
    got, state_got = out.double().cpu(), state[1].double().cpu()
    for s, e in enumerate(sums_error(g, starts)):
        rows = slice(int(starts[s]), int(starts[s + 1]))
        w, t = want[rows], tol[rows] + e * reach[rows]
        x = got[rows]  # infinite where a value within the tolerance is past the largest number
        past = (x == math.inf) & (w + t >= LARGEST[dtype]) | (x == -math.inf) & (w - t <= -LARGEST[dtype])
        assert bool(torch.all(((x - w).abs() <= t) | past)), s
        if dst[s] >= 0:
            assert torch.all((state_got[dst[s]] - after[dst[s]]).abs() <= after_tol[dst[s]] + e * most[dst[s]]), s
    T = int(starts[-1])
    assert torch.all(out[T:] == 7.0) and pkv.pkv_get_device_status() == 0
    return out


def gates_of(kind, T, n_v, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.arange(T)
    if kind == "alternating":
        d = torch.where(t % 2 == 0, 0.5, -0.5)[:, None].expand(T, n_v)
    elif kind == "normal":
        d = torch.randn((T, n_v), generator=g)
    elif kind == "growing":
        d = torch.full((T, n_v), 0.3)
    elif kind == "waves":
        d = torch.where(t // 40 % 2 == 0, 0.3, -0.3)[:, None] * torch.linspace(0.5, 1.5, n_v)
    else:                                      # strong decays with bursts between them
        d = torch.where(torch.rand((T, n_v), generator=g) < 0.1, 6.0, -1.0)
    return d.contiguous()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["alternating", "normal", "growing", "waves", "bursts"])
@pytest.mark.parametrize("dk,dv,lens", [(64, 64, [230, 64, 129]), (128, 128, [250]), (128, 64, [130, 0, 200])])
def test_decays_of_both_signs(dtype, kind, dk, dv, lens):
    q, k, v, _, state, starts = inputs(dtype, lens, 1, 2, dk, dv, "none", seed=60 + len(lens))
    d = torch.cat([gates_of(kind, sum(lens), 2, 61), torch.full((3, 2), math.nan)]).cuda()
    n = len(lens)
    check(dtype, q, k, v, d, state, [i if i % 2 == 0 else -1 for i in range(n)], list(range(n)), starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["alternating", "normal", "waves"])
def test_decays_of_both_signs_shared_out(dtype, kind):
    q, k, v, _, state, starts = inputs(dtype, [1100, 900], 1, 1, 64, 64, "none", seed=62)
    d = torch.cat([gates_of(kind, 2000, 1, 63), torch.full((3, 1), math.nan)]).cuda()
    check(dtype, q, k, v, d, state, [0, -1], [0, 1], starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["alternating", "normal"])
def test_decays_of_both_signs_of_more_units_than_the_gpu_holds(dtype, kind):
    lens = [RAGGED[i % 8] for i in range(24)]
    q, k, v, _, state, starts = inputs(dtype, lens, 4, 8, 64, 128, "none", seed=64)
    d = torch.cat([gates_of(kind, sum(lens), 8, 65), torch.full((3, 8), math.nan)]).cuda()
    check(dtype, q, k, v, d, state, list(range(24)), list(range(24)), starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("decay,far,key,value", [(-0.35, 100, 2.0 ** 13, 2.0 ** 13), (0.2, 0, 2.0 ** -6, 1.0)])
def test_a_query_that_meets_one_token(dtype, decay, far, key, value):
    """A row's only term: of a product of 2^26 that the decays leave 2^-50 of, or of a weight of 1 where the tokens before, which
    the query does not meet, have weights up to 2^36."""
    T, dk = 128, 128
    q, k, v, _, state, starts = inputs(dtype, [T], 1, 1, dk, 64, "none", seed=66, behind=0)
    k.zero_(), q.zero_()
    t = torch.arange(T)
    k[t, 0, t] = key
    q[t, 0, (t - far).clamp(min=0)] = key
    v.copy_(torch.randn(v.shape, generator=torch.Generator().manual_seed(67)) * value)
    check(dtype, q, k, v, torch.full((T, 1), decay, device="cuda"), state, [-1], [-1], starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -18, 2.0 ** 11])
def test_the_state_of_small_and_large_rows(dtype, size):
    """Values of a few bits above the type's smallest, and near its largest: the state has 22 bits of them all the same."""
    q, k, v, d, state, starts = inputs(dtype, [260], 1, 1, 64, 64, "head", seed=68)
    v *= size
    q *= 2.0 ** -6
    k *= 0.25
    check(dtype, q, k, v, d, state, [-1], [0], starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n_v", [1, 3])
def test_states_near_the_largest_number(dtype, n_v):
    """Elements of 2^125 and of 2^-125: a copy of the state for the queries is within the type either way."""
    q, k, v, d, state, starts = inputs(dtype, [200], 1, n_v, 64, 64, "head", seed=71)
    for scale in (2.0 ** 122, 2.0 ** -122):
        st = state * scale
        q2 = q * (2.0 ** -7)
        check(dtype, q2, k, v, d, st, [0], [0], starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_of_growing_decays(dtype):
    n = 5
    q, k, v, _, state, starts = inputs(dtype, [1] * n, 2, 4, 64, 64, "none", seed=78, behind=0)
    d = torch.randn((n, 4), generator=torch.Generator().manual_seed(79)).cuda() * 3
    was = state.clone()
    out = run(dtype, q, k, v, d, state, list(range(n)), list(range(n)), starts, decode=True)
    want, tol, after, after_tol = linear(q, k, v, d, was[1], list(range(n)), list(range(n)), starts, SCALE, dtype)
    assert torch.all((out.double().cpu() - want).abs() <= tol)
    assert torch.all((state[1].double().cpu() - after).abs() <= after_tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("n,length", [(1, 300), (1, 1100), (24, 200)])
def test_a_column_of_the_state_leaves_the_others_alone(dtype, dk, dv, n, length):
    """Infinite, NaN, or 2^30 larger than the others: their results are those of a state without it."""
    n_v = 1 if n == 1 else 8
    q, k, v, d, state, starts = inputs(dtype, [length] * n, 1, n_v, dk, dv, "head", seed=69)
    own, T = list(range(n)), n * length
    was = state.clone()
    base = run(dtype, q, k, v, d, state, own, own, starts)[:T]
    rest = torch.arange(dv, device="cuda") != 5
    for value in (math.inf, math.nan, None):
        st = was.clone()
        if value is None:
            st[1, :, 0, :, 5] *= 2.0 ** 30
        else:
            st[1, :, 0, 3, 5] = value
        out = run(dtype, q, k, v, d, st, own, own, starts)[:T]
        assert torch.equal(out[:, :, rest], base[:, :, rest]) and torch.equal(out[:, 1:], base[:, 1:])
        assert torch.equal(st[1, :n, 0][..., rest], state[1, :n, 0][..., rest]) and torch.equal(st[1, :n, 1:], state[1, :n, 1:])
        if value is not None:
            assert not torch.isfinite(out[:, 0, 5]).any() and not torch.isfinite(st[1, :n, 0, 3, 5]).any()
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_an_infinity_that_a_short_call_left(dtype):
    """A decode step's infinite v stays in its column of the state; the next long chunk's other columns are as without it."""
    q, k, v, d, state, starts = inputs(dtype, [300], 1, 2, 128, 64, "head", seed=70, behind=0)
    other = state.clone()
    v2 = v[:1].clone()
    v2[0, 1, 7] = math.inf
    run(dtype, q[:1], k[:1], v[:1], d, state, [0], [0], None, decode=True)
    run(dtype, q[:1], k[:1], v2, d, other, [0], [0], None, decode=True)
    assert torch.isinf(other[1, 0, 1, :, 7]).all()
    a, b = (run(dtype, q, k, v, d, st, [0], [0], starts) for st in (state, other))
    touched = torch.zeros_like(a, dtype=torch.bool)
    touched[:, 1, 7] = True
    assert torch.equal(a[~touched], b[~touched]) and not torch.isfinite(b[touched]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_many_tokens_that_forget(dtype):
    lens = [320, 150]
    q, k, v, _, state, starts = inputs(dtype, lens, 2, 4, 64, 64, "none", seed=72)
    g = torch.Generator().manual_seed(73)
    T = sum(lens)
    d = -0.01 * torch.rand((T + 3, 4), generator=g)
    t = torch.arange(T + 3)
    d[t % 32 < 20] = -math.inf
    d[(t % 32 > 22) & (t % 5 == 0), 1] = -90.0
    check(dtype, q, k, v, d.cuda(), state, [0, -1], [0, 1], starts)


def test_weights_behind_tokens_that_forget():
    """Each result is one term: exp(g_i) v_(i-1), v = 1 and products of 1, so that the weight's rounding to fp16 is the only one
    (its result is then a number of the type already): half a step, and 2^-20 for the sums, exponential and products in
    fp32. Twenty tokens of each 32 forget."""
    T, dk = 320, 64
    q, k, v, _, state, starts = inputs("f16", [T], 1, 4, dk, 64, "none", seed=74)
    k.zero_(), q.zero_(), v.fill_(1.0)
    t = torch.arange(T)
    k[t, 0, t % dk] = 1.0
    q[t, 0, (t - 1) % dk] = 1.0
    d = -0.7 * torch.rand((T, 4), generator=torch.Generator().manual_seed(75))
    d[t % 32 < 20] = -math.inf
    gates = torch.cat([d, torch.zeros(3, 4)]).cuda()
    out = run("f16", q, k, v, gates, state, [-1], [-1], starts)[:T].double().cpu()
    want = SCALE * torch.exp(d.double())[:, :, None].expand(-1, -1, 64)
    rows = (t % 32 >= 20) & (t > 0)
    assert torch.all((out[rows] - want[rows]).abs() <= (HALF_STEP["f16"] + 2.0 ** -20) * want[rows])
    assert pkv.pkv_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_what_is_not_finite_stays_behind_a_token_that_forgets(dtype, value):
    """0 times it is NaN: a key's infinity or NaN, in the forgetting token's own block of 32, an earlier one, or an earlier piece."""
    q, k, v, d, state, starts = inputs(dtype, [200], 1, 2, 64, 64, "token", seed=80, behind=0)
    d.clamp_(min=-0.1)
    d[[40, 60, 100, 101, 190]] = -math.inf
    base = run(dtype, q, k, v, d, state.clone(), [0], [0], starts)
    for at in (33, 58, 99, 10):
        k2 = k.clone()
        k2[at, 0, 3] = value
        st = state.clone()
        out = run(dtype, q, k2, v, d, st, [0], [0], starts)
        assert torch.equal(out[:at], base[:at]) and not torch.isfinite(out[at:]).any()
        assert not torch.isfinite(st[1, 0, :, 3]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n_qk,group", [(1, 16), (2, 40), (1, 64), (33, 1)])
@pytest.mark.parametrize("lens", [[1, 30], [200, 130]])
def test_many_heads_and_large_groups(dtype, n_qk, group, lens):
    q, k, v, d, state, starts = inputs(dtype, lens, n_qk, n_qk * group, 64, 64, "token", seed=76)
    check(dtype, q, k, v, d, state, [0, -1], [1, 2], starts)


@pytest.mark.parametrize("dk,dv,n,n_v", [(64, 64, 30, 4), (64, 128, 30, 4), (128, 64, 20, 4), (128, 128, 30, 4), (64, 64, 4, 2),
                                         (128, 128, 8, 3)])
def test_short_chunks_of_bf16(dk, dv, n, n_v):
    lens = [(i * 13) % 34 for i in range(1, n + 1)]
    q, k, v, d, state, starts = inputs("bf16", lens, n_v, n_v, dk, dv, seed=77 + n)
    check("bf16", q, k, v, d, state, list(range(n)), list(range(n)), starts)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[900, 333], [2000], [RAGGED[i % 8] for i in range(24)]])
def test_repeats_beside_other_work(dtype, lens):
    """Bit for bit, on two streams at once and from a graph: far-apart columns, forgetting tokens, decays of both signs."""
    n, n_v = len(lens), 8 if len(lens) > 2 else 2
    own, T = list(range(n)), sum(lens)
    sets = []
    for seed in (81, 82):
        q, k, v, _, state, starts = inputs(dtype, lens, 2, n_v, 64, 128, "none", seed=seed)
        d = torch.cat([gates_of("normal", T, n_v, seed) * 0.3, torch.full((3, n_v), math.nan)]).cuda()
        d[:T][torch.arange(T) % 37 == 5] = -math.inf
        state[1, ::2, 0, :, 3] *= 2.0 ** 30
        state[1, ::3, 1, 4, 60] = math.inf
        sets.append((q, k, v, d, state))
    want = []
    for x in sets:
        st = x[4].clone()
        want.append((run(dtype, *x[:4], st, own, own, starts)[:T], st))
    same = lambda a, b: torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32), b.view(torch.int16 if b.element_size() == 2 else torch.int32))
    streams = [torch.cuda.Stream() for _ in sets]
    states = [[x[4].clone() for x in sets] for _ in range(6)]
    torch.cuda.synchronize()
    got = []
    for pair in states:
        for st, x, state in zip(streams, sets, pair):
            with torch.cuda.stream(st):
                got.append((run(dtype, *x[:4], state, own, own, starts)[:T], state))
    torch.cuda.synchronize()
    for i, (out, state) in enumerate(got):
        assert same(out, want[i % 2][0]) and same(state, want[i % 2][1])
    desc = pkv.make_linear_desc(dtype, 2, n + 2, 2, n_v, 64, 128)
    slots, start = (torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (own, starts))
    ws = pkv.alloc_linear_prefill_workspace(desc, n, T + 3, max(lens))
    buf = [x.clone() for x in sets[0]]
    out, graph = torch.zeros_like(buf[2]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_linear_prefill(desc, 1, *buf, slots, slots, start, max(lens), SCALE, out, ws)
    for i in (1, 0, 1):
        for to, frm in zip(buf, sets[i]):
            to.copy_(frm)
        graph.replay()
        assert same(out[:T], want[i][0]) and same(buf[4], want[i][1])
    assert pkv.pkv_get_device_status() == 0
