"""Linear attention and tables from request lengths without a GPU: sizes and refusals before any launch."""
import ctypes

import pytest
import torch

from paged_kv_cache_258_gb300 import pkv

PTR, MIS, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), ctypes.c_void_p(0)
ODD = ctypes.c_void_p(0x10002)


def desc_of(dtype="bf16", layers=2, slots=5, n_qk=2, n_v=6, dk=128, dv=64):
    return pkv.make_linear_desc(dtype, layers, slots, n_qk, n_v, dk, dv)


def test_sizes():
    assert pkv.pkv_linear_state_bytes(desc_of()) == 2 * 5 * 6 * 128 * 64 * 4
    # one sequence of the hybrid model the pages count: 144 MiB of states
    assert pkv.pkv_linear_state_bytes(pkv.make_linear_desc("bf16", 48, 1, 16, 48, 128, 128)) == 144 << 20
    assert pkv.linear_state_shape(desc_of()) == (2, 5, 6, 128, 64)
    assert pkv.pkv_linear_state_bytes(desc_of(dk=256)) == 0
    for bad in ((0, 5, 5), (1, 0, 5), (1, 5, 0)):
        assert pkv.pkv_linear_prefill_workspace_bytes(desc_of(), *bad) == 0
    assert pkv.pkv_linear_prefill_workspace_bytes(desc_of(dv=32), 1, 5, 5) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(), pkv.PKV_OK), (dict(dtype="f32"), pkv.PKV_OK), (dict(n_qk=6), pkv.PKV_OK), (dict(dk=64, dv=128), pkv.PKV_OK),
    (dict(dk=256), pkv.PKV_ERR_UNSUPPORTED), (dict(dv=96), pkv.PKV_ERR_UNSUPPORTED), (dict(n_qk=4), pkv.PKV_ERR_UNSUPPORTED),
    (dict(n_v=65536), pkv.PKV_ERR_UNSUPPORTED), (dict(layers=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(slots=-1), pkv.PKV_ERR_INVALID_ARG), (dict(n_qk=0), pkv.PKV_ERR_INVALID_ARG), (dict(dk=0), pkv.PKV_ERR_INVALID_ARG),
])
def test_descriptors(kw, want):
    assert pkv.pkv_linear_validate_desc(desc_of(**kw)) == want
    if want:
        assert decode(desc_of(**kw)) == prefill(desc_of(**kw)) == want


def test_an_unknown_type_is_refused():
    d = desc_of()
    d.dtype = 7
    assert pkv.pkv_linear_validate_desc(d) == decode(d) == prefill(d) == pkv.PKV_ERR_UNSUPPORTED


def decode(d, layer=0, n=3, q=PTR, k=PTR, v=PTR, g=NULL, stride=0, state=PTR, src=PTR, dst=PTR, out=PTR):
    return pkv.lib().pkv_linear_decode(ctypes.byref(d), layer, q, k, v, g, stride, state, src, dst, n, 0.1, out, NULL)


def prefill(d, layer=0, n=3, tok=900, mq=700, q=PTR, k=PTR, v=PTR, g=NULL, stride=0, state=PTR, src=PTR, dst=PTR, start=PTR,
            out=PTR, ws=NULL, ws_bytes=0):
    return pkv.lib().pkv_linear_prefill(ctypes.byref(d), layer, q, k, v, g, stride, state, src, dst, start, n, tok, mq, 0.1,
                                        out, ws, ws_bytes, NULL)


def extend(nb=9, free=PTR, n_free=4, used=PTR, tables=PTR, mb=4, lens=PTR, new=NULL, n=3, slots=PTR, most=8, start=PTR,
           new_lens=PTR, totals=PTR):
    return pkv.lib().pkv_extend_tables(nb, free, n_free, used, tables, mb, lens, new, n, slots, most, start, new_lens, totals,
                                       NULL)


@pytest.mark.parametrize("call,kw", [
    *[(c, kw) for c in (decode, prefill) for kw in (
        dict(layer=2), dict(layer=-1), dict(n=-1), dict(q=NULL), dict(q=MIS), dict(k=MIS), dict(v=NULL), dict(v=MIS),
        dict(out=NULL), dict(out=MIS), dict(state=NULL), dict(state=MIS), dict(src=NULL), dict(src=ODD), dict(dst=NULL),
        dict(dst=ODD), dict(g=ODD), dict(g=PTR, stride=5), dict(g=PTR, stride=-6))],
    (prefill, dict(tok=-1)), (prefill, dict(mq=-1)), (prefill, dict(mq=901)), (prefill, dict(start=NULL)),
    (prefill, dict(start=ODD)),
    (extend, dict(nb=0)), (extend, dict(n_free=-1)), (extend, dict(n=-1)), (extend, dict(most=-1)), (extend, dict(mb=0)),
    (extend, dict(mb=(1 << 24) + 1)), (extend, dict(free=NULL)), (extend, dict(used=NULL)), (extend, dict(tables=NULL)),
    (extend, dict(lens=NULL)), (extend, dict(slots=NULL)), (extend, dict(slots=MIS)), (extend, dict(start=NULL)),
    (extend, dict(new_lens=NULL)), (extend, dict(totals=NULL)), (extend, dict(totals=ODD)), (extend, dict(new=ODD)),
])
def test_bad_arguments_are_refused(call, kw):
    got = call(**kw) if call is extend else call(desc_of(), **kw)
    assert got == pkv.PKV_ERR_INVALID_ARG


def test_sizes_past_the_limits_are_refused():
    assert decode(desc_of(), n=65536) == prefill(desc_of(), n=65536, tok=70000) == pkv.PKV_ERR_UNSUPPORTED
    wide = desc_of(n_qk=65535, n_v=65535, dv=128)
    assert decode(wide, n=65535) == prefill(wide, n=65535, tok=70000) == pkv.PKV_ERR_UNSUPPORTED
    assert extend(n=65536) == pkv.PKV_ERR_UNSUPPORTED


def test_no_sequences_is_no_call():
    assert decode(desc_of(), n=0, q=NULL, state=NULL) == prefill(desc_of(), n=0, q=NULL, start=NULL) == pkv.PKV_OK


def test_host_tensors_are_refused():
    d = desc_of("f32", n_qk=1, n_v=1, dk=64)
    q, v, st = torch.zeros(2, 1, 64), torch.zeros(2, 1, 64), torch.zeros(pkv.linear_state_shape(d))
    slots, start = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_linear_decode(d, 0, q, q, v, None, st, slots, slots, 1.0, v)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_linear_prefill(d, 0, q, q, v, None, st, slots, slots, start, 2, 1.0, v)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.linear_decode_launcher(d, q[None], q[None], v[None], None, st, slots, slots, 1.0, v[None])
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_extend_tables(9, slots, slots[:1], t, slots, None, torch.zeros(4, dtype=torch.int64), start, slots, start)


def test_overlapping_lengths_are_refused():
    t, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="overlap"):
        pkv.pkv_extend_tables(9, lens, lens[:1], t, lens[:2], None, torch.zeros(4, dtype=torch.int64), lens, lens[1:], lens)


def test_rows_may_be_null_without_tokens_only():
    for bad in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(out=NULL)):
        assert prefill(desc_of(), tok=1, mq=1, **bad) == pkv.PKV_ERR_INVALID_ARG
    assert prefill(desc_of(), tok=0, mq=0, q=NULL, k=NULL, v=NULL, out=NULL, state=NULL) == pkv.PKV_ERR_INVALID_ARG


def test_token_counts_that_32_bits_cannot_round_up_are_refused():
    assert prefill(desc_of(), tok=2 ** 31 - 1, mq=2 ** 31 - 1) == pkv.PKV_ERR_UNSUPPORTED
