"""States of sequences with steps on another stream than the one they were made on, which is busy."""
import pytest
import torch

from paged_kv_cache_258_gb300 import pkv
from paged_kv_cache_258_gb300.engine import LinearStates

pytestmark = pytest.mark.gpu
BUSY = 200_000_000                                     # cycles: about a tenth of a second


def step(states, ids, seed, **on):
    """One token of each of ids on the current stream (or as `on` says); returns its results."""
    g = torch.Generator().manual_seed(seed)
    rows = lambda *s: torch.randn(s, generator=g).half().cuda()
    d = states.desc
    with torch.cuda.stream(on.get("stream", torch.cuda.current_stream())):
        q, k, v = rows(len(ids), d.n_qk_heads, d.dim_k), rows(len(ids), d.n_qk_heads, d.dim_k), rows(len(ids), d.n_v_heads, d.dim_v)
        out = torch.zeros_like(v)
    src, dst = states.slots(ids, **on)
    pkv.pkv_linear_decode(d, 0, q, k, v, None, states.state, src, dst, 1.0, out, **on)
    return out


def made(stream):
    states = LinearStates(pkv.make_linear_desc("f16", 1, 6, 1, 2, 64, 64), stream=stream)
    for x in range(4):
        states.add(x)
    return states


@pytest.fixture
def want():
    """Results of two steps of sequences 2 and 3, a fork of 3 behind them, and a step of 3 and the fork."""
    states = made(torch.cuda.current_stream())
    a = [step(states, [2, 3], 0), step(states, [2, 3], 1)]
    states.fork(3, 9)
    return [*a, step(states, [3, 9], 2)], states.state.clone()


@pytest.mark.parametrize("given", [False, True])
def test_steps_on_another_stream(want, given):
    """With `stream` given to each call, or by the current stream."""
    home, side = torch.cuda.Stream(), torch.cuda.Stream()
    states = made(home)
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        torch.cuda._sleep(BUSY)                        # the stream they were made on is busy all along
    on = dict(stream=side) if given else {}
    with torch.cuda.stream(torch.cuda.current_stream() if given else side):
        got = [step(states, [2, 3], 0, **on)]
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY // 4)               # what the fork copies is not there yet when it is called
        got.append(step(states, [2, 3], 1, **on))
        states.fork(3, 9, **on)
        got.append(step(states, [3, 9], 2, **on))
    side.synchronize()
    torch.cuda.synchronize()
    for g, w in zip(got, want[0]):
        assert torch.equal(g, w)
    assert torch.equal(states.state, want[1]) and pkv.pkv_get_device_status() == 0


def test_made_on_a_busy_stream(want):
    """The states are zeros when the constructor returns: no step on another stream is overwritten by them."""
    home = torch.cuda.Stream()
    with torch.cuda.stream(home):
        torch.cuda._sleep(BUSY // 4)
    states = made(home)
    got = [step(states, [2, 3], 0), step(states, [2, 3], 1)]
    states.fork(3, 9)
    got.append(step(states, [3, 9], 2))
    torch.cuda.synchronize()
    for g, w in zip(got, want[0]):
        assert torch.equal(g, w)
    assert torch.equal(states.state, want[1])
