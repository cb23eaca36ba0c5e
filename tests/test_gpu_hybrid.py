"""A hybrid model's steps on the GPU: tables grown on the device, paged attention on some layers, linear attention over
states on the others; replayed from a graph, against the host-planned steps."""
import numpy as np
import pytest
import torch

from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300.engine import DecodeBatch, DeviceTables, LinearStates, PagedKVCache, PrefillStep

pytestmark = pytest.mark.gpu
L, SCALE = 2, 0.125


def rows(g, t, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(t)


def model(dtype, n, nb):
    desc = pkv.make_desc(dtype, L, nb, 8, 2, 128)
    ldesc = pkv.make_linear_desc(dtype, L, n + 1, 2, 6, 128, 64)
    cache = PagedKVCache(desc, free_order=np.random.default_rng(3).permutation(nb).astype(np.int32))
    return desc, ldesc, cache, LinearStates(ldesc)


def inputs(g, t, n):
    """One step's rows of n tokens: attention layers' q, k, v and linear layers' q, k, v, log decay."""
    return (rows(g, t, L, n, 8, 128), rows(g, t, L, n, 2, 128), rows(g, t, L, n, 2, 128), rows(g, t, L, n, 2, 128),
            rows(g, t, L, n, 2, 128), rows(g, t, L, n, 6, 64), -torch.rand((L, n, 6), generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_steps_on_the_device_equal_host_planned_steps(dtype):
    t = pkv.torch_dtype(dtype)
    prompts, steps, mb, nb = [37, 5, 64, 230, 1], 40, 20, 120
    n, total = len(prompts), sum(prompts)
    ids = list(range(10, 10 + n))
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    data = [inputs(g, t, total)] + [inputs(g, t, n) for _ in range(steps)]

    # the host plans
    desc, ldesc, cache, states = model(dtype, n, nb)
    want = []
    pre = PrefillStep(cache, total, n, mb)
    for x in ids:
        states.add(x)
    q, k, v, lq, lk, lv, d = data[0]
    out, lout = torch.empty_like(q), torch.empty_like(lv)
    pre.step([(x, c, True) for x, c in zip(ids, prompts)], q, k, v, out, SCALE)
    start = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    src, dst = states.slots(ids)
    for layer in range(L):
        pkv.pkv_linear_prefill(ldesc, layer, lq[layer], lk[layer], lv[layer], d[layer], states.state, src, dst, start,
                               max(prompts), SCALE, lout[layer])
    want.append((out, lout))
    batch = DecodeBatch(cache, ids, mb)
    src, dst = states.slots(ids)
    for q, k, v, lq, lk, lv, d in data[1:]:
        out, lout = torch.empty_like(q), torch.empty_like(lv)
        batch.step(q, k, v, out, SCALE)
        for layer in range(L):
            pkv.pkv_linear_decode(ldesc, layer, lq[layer], lk[layer], lv[layer], d[layer], states.state, src, dst, SCALE,
                                  lout[layer])
        want.append((out, lout))
    torch.cuda.synchronize()
    end = cache.mgr.pack_tables(ids, mb)

    # the device plans, its decode steps from one captured graph
    desc, ldesc, cache, other = model(dtype, n, nb)
    for x in ids:
        other.add(x)
        cache.add_sequence(x, 0)
    tables = DeviceTables(cache, ids, mb, max_tokens=total + 3)
    counts = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    tables.extend(counts)
    q, k, v, lq, lk, lv, d = (torch.cat([x, torch.full_like(x[:, :3], float("nan"))], 1) for x in data[0])
    out, lout = torch.empty_like(q), torch.empty_like(lv)
    src, dst = other.slots(ids)
    linear = pkv.linear_prefill_launcher(ldesc, lq, lk, lv, d, other.state, src, dst, tables.query_start, max(prompts), SCALE,
                                         lout)
    for layer in range(L):
        cache.append(layer, k[layer], v[layer], tables.slots)
        pkv.pkv_paged_prefill_attention(desc, layer, q[layer], cache.k_pool, cache.v_pool, tables.tables, tables.lens,
                                        tables.query_start, max(prompts), SCALE, out[layer])
        linear(layer)
    assert torch.equal(out[:, :total], want[0][0]) and torch.equal(lout[:, :total], want[0][1])
    assert tables.follow(prompts) == n
    tables = DeviceTables(cache, ids, mb)
    assert torch.equal(tables.lens.cpu(), torch.tensor(prompts, dtype=torch.int32))
    buf = inputs(g, t, n)
    q, k, v, lq, lk, lv, d = buf
    out, lout = torch.empty_like(q), torch.empty_like(lv)
    ws = pkv.alloc_workspace(desc, n, mb)
    src, dst = other.slots(ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tables.extend(stream=side)
        attend = pkv.decode_append_launcher(desc, q, k, v, cache.k_pool, cache.v_pool, tables.tables, tables.lens, SCALE, out, ws,
                                            stream=side)
        linear = pkv.linear_decode_launcher(ldesc, lq, lk, lv, d, other.state, src, dst, SCALE, lout, stream=side)
        for layer in range(L):
            attend(layer)
            linear(layer)
    for step in range(steps):
        for to, frm in zip(buf, data[1 + step]):
            to.copy_(frm)
        graph.replay()
        assert torch.equal(out, want[1 + step][0]) and torch.equal(lout, want[1 + step][1]), step
    for _ in range(steps):
        assert tables.follow() == n
    rc, host, lens = cache.mgr.pack_tables(ids, mb)
    assert np.array_equal(host, end[1]) and np.array_equal(tables.tables.cpu().numpy(), host)
    assert np.array_equal(tables.lens.cpu().numpy(), lens)
    assert torch.equal(other.state[:, dst.long()], states.state[:, dst.long()])
    assert pkv.pkv_get_device_status() == 0


def test_a_pool_that_runs_out():
    """The device serves the rows that fit, and the manager that follows serves the same."""
    desc, _, cache, _ = model("bf16", 4, 9)
    ids = [0, 1, 2, 3]
    for x, c in zip(ids, (16, 30, 32, 5)):
        cache.add_sequence(x, c)                       # 1 + 2 + 2 + 1 blocks of 9
    tables = DeviceTables(cache, ids, 6, max_tokens=200)
    for counts in ([1, 1, 1, 1], [20, 20, 1, 3], [0, 0, 40, 1]):
        tables.extend(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        served = tables.follow(counts)
        assert tables.totals[1].item() == served
        rc, host, lens = cache.mgr.pack_tables(ids, 6)
        assert np.array_equal(tables.tables.cpu().numpy(), host) and np.array_equal(tables.lens.cpu().numpy(), lens)
    assert served == 2


def test_tables_that_cannot_grow_on_the_device_are_refused():
    _, _, cache, _ = model("bf16", 4, 20)
    cache.add_sequence(0, 20)
    cache.add_sequence(1, 32)
    cache.fork(0, 2)
    cache.fork(1, 3)
    with pytest.raises(ValueError, match="shared"):
        DeviceTables(cache, [0, 1], 5)
    with pytest.raises(ValueError, match="twice"):
        DeviceTables(cache, [1, 1], 5)
    with pytest.raises(pkv.PkvError):
        DeviceTables(cache, [1, 7], 5)
    DeviceTables(cache, [1, 3], 5).extend()             # whole blocks may be shared


def test_states_of_sequences():
    _, ldesc, _, states = model("f16", 3, 4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v, d = (x[0] for x in inputs(g, torch.float16, 2)[3:])
    one = lambda ids: pkv.pkv_linear_decode(ldesc, 0, q[:len(ids)], k[:len(ids)], v[:len(ids)], d[:len(ids)], states.state,
                                            *states.slots(ids), SCALE, torch.empty_like(v[:len(ids)]))
    states.add(5)
    states.add(6)
    states.fork(5, 7)                                   # before 5 has any state: 7 starts from zeros too
    one([5, 6])
    states.fork(5, 8)
    a, b, c, e = (states._slot[x] for x in (5, 6, 7, 8))
    assert torch.equal(states.state[0, e], states.state[0, a]) and states.state[0, a].abs().max() > 0
    assert states.state[0, c].abs().max() == 0
    first = states.state[0, a].clone()
    with pytest.raises(pkv.PkvError):
        states.add(9)                                   # all four slots are taken
    for bad in (lambda: states.add(5), lambda: states.fork(11, 12), lambda: states.free(11), lambda: states.slots([5, 5]),
                lambda: states.slots([11])):
        with pytest.raises(pkv.PkvError):
            bad()
    one([5])
    states.free(5)
    states.add(9)                                       # 5's slot, from zeros
    assert states._slot[9] == a
    one([9])
    assert torch.equal(states.state[0, a], first)


def test_a_step_that_was_not_run_can_be_taken_back():
    _, ldesc, _, states = model("f16", 3, 4)
    states.state.fill_(3.0)                             # what earlier sequences left
    states.add(1)
    states.slots([1])                                   # the step that was to begin it is not run
    states.restart(1)
    src, dst = states.slots([1])
    assert src.tolist() == [-1] and dst.tolist() == [states._slot[1]]
    assert states.slots([1])[0].tolist() == dst.tolist()
    with pytest.raises(pkv.PkvError):
        states.restart(2)


def test_a_step_is_captured_on_the_current_stream():
    _, _, cache, _ = model("f16", 2, 40)
    for x in (1, 2):
        cache.add_sequence(x, 0)
    tables = DeviceTables(cache, [1, 2], 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tables.extend()
    assert tables.lens.tolist() == [0, 0]               # captured, not run
    for _ in range(40):
        graph.replay()
    assert tables.lens.tolist() == [40, 40] and tables.totals.tolist() == [6, 2, 2]
    for _ in range(40):
        assert tables.follow() == 2
    rc, host, lens = cache.mgr.pack_tables([1, 2], 8)
    assert np.array_equal(tables.tables.cpu().numpy(), host) and list(lens) == [40, 40]
