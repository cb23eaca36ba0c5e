"""The cache-shrinking operators of the paged KV cache, measured: 8-bit pools (append, decode, prefill) and
eviction by accumulated attention weight (decode that sums its weights, and the eviction itself).

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the library's entry points. ``exact`` restates each operator in 64 bits.

Layouts: pools [layers, blocks, n_kv, 16, d]; scales [layers, blocks, n_kv]; tables int32 [n_seqs, max_blocks];
scores [layers, n_seqs, n_kv, max_blocks * 16]; query head h reads KV head h // (n_q // n_kv). An 8-bit pool
holds e4m3 codes; a code stands for code * scale, the scale a power of two for each (block, KV head).
"""
import math

import torch

own = False

BLOCK = 16
E4M3_MAX = 448.0
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
MIN_EXP = {"f16": -15, "bf16": -117}      # least exponent of a block's scale, by the rows' type
LOG2E = 1.4426950408889634
NEG = float("-inf")


# ---- cases ----------------------------------------------------------------------------------------

def _case(name, op, dtype, n_kv, group, d, n_seqs, lo, hi, **more):
    return dict(name=name, op=op, dtype=dtype, n_kv=n_kv, group=group, d=d, n_seqs=n_seqs, lo=lo, hi=hi, **more)


def listed():
    return [
        # one decode step of the GPT-style batch: 64 new rows, each into the middle of its sequence's last block
        _case("append8 step", "append8", "f16", 32, 1, 128, 64, 64, 2048, chunk=1),
        # one prompt chunk of the long-document model, starting inside a block
        _case("append8 chunk", "append8", "bf16", 4, 4, 256, 1, 9005, 9005, chunk=2432),
        # a single short session: latency
        _case("decode8 one", "decode8", "bf16", 8, 4, 128, 1, 301, 301, scored=False),
        # the GPT-style batch (multi-head, lengths 64..2,048)
        _case("decode8 batch", "decode8", "f16", 32, 1, 128, 64, 64, 2048, scored=False),
        # long documents, grouped queries
        _case("decode8 long", "decode8", "bf16", 4, 4, 256, 10, 30000, 32768, scored=False),
        # the same cache while weights are summed for a later eviction, ragged, one empty row
        _case("decode8 scored", "decode8", "bf16", 8, 8, 128, 32, 0, 8192, scored=True),
        # a few short follow-up prompts in one step
        _case("prefill8 turns", "prefill8", "f16", 8, 4, 64, 4, 700, 1900, chunk=70),
        # one chunk of a long document late in its prompt
        _case("prefill8 long", "prefill8", "bf16", 4, 4, 256, 1, 30000, 30000, chunk=2432),
        # 16-bit pools: the GPT-style batch with its weights summed
        _case("scored batch", "scored", "f16", 32, 1, 128, 64, 64, 2048),
        # 16-bit pools: long documents with their weights summed
        _case("scored long", "scored", "bf16", 4, 4, 256, 10, 30000, 32768),
        # half of each session's tokens leave a 16-bit cache
        _case("evict half", "evict", "f16", 8, 4, 128, 16, 500, 4096, layers=4, keep=0.5, recent=64, bits8=False),
        # long sessions cut to a fixed share in an 8-bit cache
        _case("evict8 long", "evict", "bf16", 4, 4, 256, 8, 9000, 16384, layers=4, keep=0.25, recent=200, bits8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "decode8", "decode8", "prefill8", "scored", "evict"])
    while True:
        d = rng.choice([64, 128, 256])
        group = rng.choice([1, 2, 4, 8])
        n_kv = _log(rng, 1, 32)
        n_seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768)
        lo = hi if n_seqs == 1 else _log(rng, 1, hi) - rng.choice([0, 1])
        dtype = rng.choice(["f16", "bf16"])
        c = _case("", op, dtype, n_kv, group, d, n_seqs, lo, hi)
        del c["name"]
        if op in ("append8", "prefill8"):
            c["chunk"] = _log(rng, 1, 2500)
        if op == "decode8":
            c["scored"] = rng.random() < 0.4
        if op == "evict":
            c.update(layers=_log(rng, 1, 8), keep=round(rng.uniform(0.05, 0.95), 3), recent=_log(rng, 1, 300),
                     bits8=rng.random() < 0.5)
        elems = sum(_lens(c)) * n_kv * d * c.get("layers", 1)
        queries = sum(_chunks(c)) * n_kv * group * max(_lens(c)) if op == "prefill8" else 0
        if max(_lens(c)) > 0 and n_kv * group <= 64 and elems <= 200e6 and queries <= 1.0e9:
            return c


def _lens(case):
    """Context lengths, spread over [lo, hi] by a fixed irrational step: they follow from the case alone."""
    n, lo, hi = case["n_seqs"], case["lo"], case["hi"]
    out = [lo + int(((i * 0.6180339887498949 + 0.37) % 1.0) * (hi - lo + 1)) for i in range(n)]
    out[0] = hi
    if n > 1:
        out[-1] = lo
    return out


def _chunks(case):
    """New tokens of each sequence in an append or prefill: the case's chunk, less where the context is shorter."""
    return [min(case["chunk"], c) for c in _lens(case)]


def _keeps(case):
    return [int(c * case["keep"]) for c in _lens(case)]


# ---- inputs ---------------------------------------------------------------------------------------

def _pow2_scale(amax, min_exp):
    """The least power of two S with amax <= 448 S, no less than 2^min_exp (448 = 1.75 * 2^8)."""
    mant, exp = torch.frexp(amax)                        # amax = mant * 2^exp, mant in [1/2, 1)
    e = torch.where(mant > 0.875, exp - 8, exp - 9)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, min_exp)).clamp(min=min_exp))


def _quantise(x, dtype):
    """Blocks x [..., 16, d] (float32) -> e4m3 codes and their scales [...]."""
    s = _pow2_scale(x.abs().amax(dim=(-1, -2)), MIN_EXP[dtype])
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _values(g, shape, dev, spread):
    """N(0, 1) times a factor for each channel (keys have channels of their own size)."""
    f = torch.exp(spread * torch.randn((*(1,) * (len(shape) - 1), shape[-1]), device=dev, generator=g))
    return torch.randn(shape, device=dev, generator=g).mul_(f)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], TORCH[case["dtype"]]
    n_kv, d, n = case["n_kv"], case["d"], case["n_seqs"]
    n_q, layers = n_kv * case["group"], case.get("layers", 1)
    lens = _lens(case)
    blocks = [-(-c // BLOCK) for c in lens]
    mb = max(max(blocks), 1)
    keeps = _keeps(case) if op == "evict" else []
    fresh = sum(-(-k // BLOCK) for k in keeps)           # an eviction moves the kept rows into blocks of their own
    nb = sum(blocks) + fresh + 3
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    s = dict(case=dict(case), scale=1.0 / math.sqrt(d), nb=nb, layers=layers, n_q=n_q, max_query=0)
    tables, at = torch.full((n, mb), -1, dtype=torch.int32), 0
    for i, b in enumerate(blocks):
        tables[i, :b] = perm[at:at + b]
        at += b
    s["tables"] = tables.to(dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    bits8 = op in ("append8", "decode8", "prefill8") or case.get("bits8", False)
    for name, spread in (("k", 0.4), ("v", 0.1)):
        pools, scales = [], []
        for _ in range(layers):
            x = _values(g, (nb, n_kv, BLOCK, d), dev, spread)
            if bits8:
                x, sc = _quantise(x, case["dtype"])
                scales.append(sc)
            pools.append(x if bits8 else x.to(dt))
        s[name + "_pool"] = torch.stack(pools)
        if bits8:
            s[name + "_scales"] = torch.stack(scales)
    if op in ("append8", "prefill8"):
        new = _chunks(case)
        starts = [0]
        for c in new:
            starts.append(starts[-1] + c)
        s["query_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["max_query"] = max(new)
        if op == "append8":
            pos = torch.cat([torch.arange(c - m, c) for c, m in zip(lens, new)])
            row = torch.cat([torch.full((m,), i) for i, m in enumerate(new)]).long()
            block = tables[row, pos // BLOCK].long()
            s["slots"] = (block * BLOCK + pos % BLOCK).to(dev)
            touched, index = torch.unique(block, return_inverse=True)
            s["touched"], s["index"] = touched.to(dev), index.to(dev)
            s["k_new"] = _values(g, (starts[-1], n_kv, d), dev, 0.4).to(dt)
            s["v_new"] = _values(g, (starts[-1], n_kv, d), dev, 0.1).to(dt)
        else:
            s["q"] = torch.randn((starts[-1], n_q, d), device=dev, generator=g).to(dt)
            s["out"] = torch.empty_like(s["q"])
    if op in ("decode8", "scored"):
        s["q"] = torch.randn((n, n_q, d), device=dev, generator=g).to(dt)
        s["out"] = torch.empty_like(s["q"])
        if op == "scored" or case["scored"]:
            s["scores"] = torch.rand((n, n_kv, mb * BLOCK), device=dev, generator=g)
    if op == "evict":
        dst, at = torch.full((n, mb), -1, dtype=torch.int32), sum(blocks)
        for i, k in enumerate(keeps):
            b = -(-k // BLOCK)
            dst[i, :b] = perm[at:at + b]
            at += b
        s["dst"] = dst.to(dev)
        s["keep"] = torch.tensor(keeps, dtype=torch.int32, device=dev)
        s["max_keep"] = max(max(keeps), 1)
        # sums of softmax weights: most positions hold little, a few hold much
        s["scores"] = torch.exp(2.0 * torch.randn((layers, n, n_kv, mb * BLOCK), device=dev, generator=g)) / mb
        s["new_scores"] = torch.zeros_like(s["scores"])
        s["kept"] = torch.full((layers, n, n_kv, s["max_keep"]), -1, dtype=torch.int32, device=dev)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"append8": _append8, "decode8": _decode, "prefill8": _prefill8, "scored": _decode,
            "evict": _evict}[s["case"]["op"]](s)


def _own(s):
    """The library's calls. The descriptor and the workspace are made at a state's first pass and kept, as a
    program that serves keeps them."""
    from paged_kv_cache_258_gb300 import pkv
    c = s["case"]
    op = c["op"]
    if "desc" not in s:
        s["desc"] = pkv.make_desc(c["dtype"], s["layers"], s["nb"], s["n_q"], c["n_kv"], c["d"])
        n, mb = s["tables"].shape
        s["ws"] = None
        if op == "decode8":
            s["ws"] = pkv.alloc_q8_workspace(s["desc"], n, mb, scored=c["scored"])
        elif op == "prefill8":
            s["ws"] = pkv.alloc_q8_prefill_workspace(s["desc"])
        elif op == "scored":
            s["ws"] = pkv.alloc_scored_workspace(s["desc"], n, mb)
        elif op == "evict" and c["bits8"]:
            s["ws"] = pkv.alloc_evict_workspace(s["desc"], n, mb)
    desc = s["desc"]
    if op == "append8":
        pkv.pkv_q8_append(desc, 0, s["k_new"], s["v_new"], s["slots"], s["k_pool"], s["v_pool"], s["k_scales"],
                          s["v_scales"])
        return {"k": s["k_pool"], "v": s["v_pool"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if op == "decode8":
        pkv.pkv_q8_decode_attention(desc, 0, s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                                    s["tables"], s["lens"], s["scale"], s["out"], s["ws"], scores=s.get("scores"))
        return {"out": s["out"], "scores": s["scores"]} if c["scored"] else {"out": s["out"]}
    if op == "prefill8":
        pkv.pkv_q8_prefill_attention(desc, 0, s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                                     s["tables"], s["lens"], s["query_start"], s["max_query"], s["scale"], s["out"],
                                     s["ws"])
        return {"out": s["out"]}
    if op == "scored":
        pkv.pkv_paged_decode_attention_scored(desc, 0, s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"],
                                              s["scale"], s["out"], s["scores"], s["ws"])
        return {"out": s["out"], "scores": s["scores"]}
    pkv.pkv_evict_tokens(desc, s["k_pool"], s["v_pool"], s["tables"], s["dst"], s["lens"], s["keep"], c["recent"],
                         s["scores"], s["new_scores"], s["kept"], k_scales=s.get("k_scales"),
                         v_scales=s.get("v_scales"), workspace=s["ws"])
    return _evicted(s)


def _evicted(s):
    got = {"k": s["k_pool"], "v": s["v_pool"], "new_scores": s["new_scores"], "kept": s["kept"]}
    if s["case"]["bits8"]:
        got.update(k_scales=s["k_scales"], v_scales=s["v_scales"])
    return got


def _append8(s):
    touched, index, slots = s["touched"], s["index"], s["slots"]
    off = slots % BLOCK
    n_b, n_kv = touched.numel(), s["case"]["n_kv"]
    started = torch.zeros(n_b, dtype=torch.int32, device=slots.device).index_add_(0, index, (off == 0).int()) > 0
    written = torch.zeros((n_b, BLOCK), dtype=torch.bool, device=slots.device)
    written[index, off] = True
    got = {}
    for name in ("k", "v"):
        pool, scales, x = s[name + "_pool"][0], s[name + "_scales"][0], s[name + "_new"].float()
        amax = torch.zeros((n_b, n_kv), device=x.device).index_reduce_(0, index, x.abs().amax(-1), "amax")
        need = _pow2_scale(amax, MIN_EXP[s["case"]["dtype"]])
        old = scales[touched]
        new = torch.where(started[:, None], need, torch.maximum(old, need))
        codes = pool[touched].float()
        keep = (started[:, None] | (old == new))[:, :, None, None] | written[:, None, :, None]
        codes = torch.where(keep, codes, codes * (old / new)[:, :, None, None])
        codes[index, :, off] = x / new[index][:, :, None]
        pool[touched] = codes.to(torch.float8_e4m3fn)
        scales[touched] = new
        got[name], got[name + "_scales"] = s[name + "_pool"], s[name + "_scales"]
    return got


def _gather(s, name):
    """Rows of every sequence by position, float32 [n_seqs, n_kv, max_blocks * 16, d]."""
    t = s["tables"].clamp(min=0).long()
    x = s[name + "_pool"][0][t].float()                               # [n, mb, n_kv, 16, d]
    if name + "_scales" in s:
        x = x * s[name + "_scales"][0][t][:, :, :, None, None]
    n, mb, h, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, mb * BLOCK, d)


def _softmax(z, live):
    """Weights along the last axis over the positions that `live` admits; a row with none gives zeros."""
    z = torch.where(live, z, torch.full_like(z, NEG))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == NEG, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _decode(s):
    c = s["case"]
    k, v = _gather(s, "k"), _gather(s, "v")
    n, h, length, d = k.shape
    live = (torch.arange(length, device=k.device) < s["lens"][:, None])[:, None, None]
    q = s["q"].float().view(n, h, c["group"], d) * s["scale"]
    w = _softmax(q @ k.transpose(-1, -2), live)                       # [n, n_kv, group, length]
    v = torch.where(live.transpose(-1, -2), v, torch.zeros_like(v))
    s["out"].copy_((w @ v).view(n, s["n_q"], d))
    if "scores" not in s:
        return {"out": s["out"]}
    s["scores"] += w.sum(2)
    return {"out": s["out"], "scores": s["scores"]}


def _prefill8(s):
    c = s["case"]
    k, v = _gather(s, "k"), _gather(s, "v")
    n, h, length, d = k.shape
    start, count = s["query_start"][:-1].long(), s["query_start"].diff().long()
    i = torch.arange(s["max_query"], device=k.device)
    inside = i < count[:, None]                                       # [n, max_query]
    rows = torch.where(inside, start[:, None] + i, start[:, None])
    pos = (s["lens"].long() - count)[:, None] + i
    q = s["q"].float()[rows.clamp(max=s["q"].shape[0] - 1)] * s["scale"]
    q = q.view(n, -1, h, c["group"], d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)
    live = (torch.arange(length, device=k.device) <= pos[:, :, None]).repeat(1, c["group"], 1)[:, None]
    w = _softmax(q @ k.transpose(-1, -2), live)
    past = (torch.arange(length, device=k.device) >= s["lens"][:, None])[:, None, :, None]
    o = w @ torch.where(past, torch.zeros_like(v), v)
    o = o.view(n, h, c["group"], -1, d).permute(0, 3, 1, 2, 4).reshape(n, -1, s["n_q"], d)
    s["out"][rows[inside]] = o[inside].to(s["out"].dtype)
    return {"out": s["out"]}


def _evict(s):
    c, scores, lens = s["case"], s["scores"], s["lens"].long()
    layers, n, h, length = scores.shape
    dev = scores.device
    k = torch.minimum(s["keep"].long(), lens)
    recent = k.clamp(max=c["recent"])
    j = torch.arange(length, device=dev)
    older = j < (lens - recent)[:, None]                              # [n, length]
    newest = ~older & (j < lens[:, None])
    z = torch.where(older[None, :, None], scores, torch.full_like(scores, NEG))
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    kept = ((rank < (k - recent)[None, :, None, None]) & older[None, :, None]) | newest[None, :, None]
    pos = torch.sort(torch.where(kept, j, torch.full_like(j, length)), dim=-1).values[..., :s["max_keep"]]
    i = torch.arange(pos.shape[-1], device=dev)
    live = (i < k[:, None])[None, :, None].expand_as(pos)
    pos = torch.where(live, pos, torch.zeros_like(pos))
    s["kept"].copy_(torch.where(live, pos.int(), s["kept"]))
    moved = torch.zeros((layers, n, h, length), device=dev)
    moved[..., :pos.shape[-1]] = torch.where(live, scores.gather(-1, pos), torch.zeros_like(pos, dtype=scores.dtype))
    inside = (j < lens[:, None])[None, :, None]
    s["new_scores"].copy_(torch.where(inside, moved, s["new_scores"]))
    at = torch.nonzero(live, as_tuple=True)                           # (layer, sequence, head, row) of every kept row
    src = s["tables"].long()[at[1], pos[at] // BLOCK], pos[at] % BLOCK
    dst = s["dst"].long()[at[1], at[3] // BLOCK], at[3] % BLOCK
    for name in ("k", "v"):
        pool = s[name + "_pool"]
        rows = pool[at[0], src[0], at[2], src[1]]
        if c["bits8"]:
            scales = s[name + "_scales"]
            old = scales[at[0], src[0], at[2]]
            flat = scales.clone().view(-1)
            cell = (at[0] * s["nb"] + dst[0]) * h + at[2]
            flat[cell] = 0.0
            flat.scatter_reduce_(0, cell, old, "amax")
            rows = (rows.float() * (old / flat[cell])[:, None]).to(pool.dtype)
            scales.copy_(flat.view_as(scales))
        pool[at[0], dst[0], at[2], dst[1]] = rows
    return _evicted(s)


# ---- the work of one pass -------------------------------------------------------------------------

def work(case):
    op, n_kv, d, group = case["op"], case["n_kv"], case["d"], case["group"]
    lens = _lens(case)
    total, n, n_q = sum(lens), case["n_seqs"], n_kv * group
    tables = 4 * sum(-(-c // BLOCK) for c in lens) + 4 * n
    scales = 8 * n_kv * sum(-(-c // BLOCK) for c in lens)            # K and V, float32 for each (block, head)
    if op == "append8":
        tok = sum(_chunks(case))
        blocks = sum(-(-c // BLOCK) - (c - m) // BLOCK for c, m in zip(lens, _chunks(case)) if m)
        return {"bytes": tok * n_kv * 2 * d * 3 + 8 * tok + 16 * n_kv * blocks, "flops": 2 * tok * n_kv * 2 * d}
    if op in ("decode8", "scored"):
        row = 2 * d * (1 if op == "decode8" else 2)
        add = 8 * total * n_kv if op == "scored" or case["scored"] else 0
        return {"bytes": total * n_kv * row + (scales if op == "decode8" else 0) + add + 4 * n * n_q * d + tables,
                "flops": 4 * total * n_q * d}
    if op == "prefill8":
        pairs = sum(m * (c - m) + m * (m + 1) // 2 for c, m in zip(lens, _chunks(case)))
        tok = sum(_chunks(case))
        return {"bytes": total * n_kv * 2 * d + scales + 4 * tok * n_q * d + tables, "flops": 4 * d * n_q * pairs}
    k = sum(min(a, b) for a, b in zip(_keeps(case), lens))
    row = 2 * d * (1 if case["bits8"] else 2)
    return {"bytes": case["layers"] * n_kv * (8 * total + 4 * k + 2 * k * row) + tables,
            "flops": case["layers"] * n_kv * total}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append8": _exact_append, "decode8": _exact_attention, "scored": _exact_attention,
            "prefill8": _exact_attention, "evict": _exact_evict}[case["op"]](s)


def _grid(dev):
    """The non-negative e4m3 values in order: m/8 * 2^-6 below 2^-6, then (1 + m/8) * 2^e up to 448."""
    g = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(g[:-1], dtype=torch.float64, device=dev)


def _to_grid(x):
    """The nearest e4m3 value of each x, halfway cases to the even code."""
    g = _grid(x.device)
    up = torch.searchsorted(g, x.abs().contiguous()).clamp(max=g.numel() - 1)
    down = (up - 1).clamp(min=0)
    a = x.abs()
    near_up = (g[up] - a < a - g[down]) | ((g[up] - a == a - g[down]) & (up % 2 == 0)) | (up == down)
    return torch.where(near_up, g[up], g[down]) * torch.sign(x)


def _least_scale(amax, dtype):
    """For each amax the least 2^e, e >= the type's least, with amax <= 448 * 2^e, found by trying."""
    e = torch.arange(MIN_EXP[dtype], 128, dtype=torch.float64, device=amax.device)
    return torch.exp2(e[torch.searchsorted(E4M3_MAX * torch.exp2(e), amax.contiguous())])


def _exact_append(s):
    dtype, got = s["case"]["dtype"], {}
    slots = s["slots"].tolist()
    blocks = {}
    for t, slot in enumerate(slots):
        blocks.setdefault(slot // BLOCK, []).append((t, slot % BLOCK))
    full = [b for b, rows in blocks.items() if len(rows) == BLOCK]
    part = [b for b in blocks if len(blocks[b]) < BLOCK]
    for name in ("k", "v"):
        pool, scales = s[name + "_pool"][0].double(), s[name + "_scales"][0].double()
        x = s[name + "_new"].double()
        if full:                                                      # blocks that the call writes whole
            t = torch.tensor([[a for a, _ in sorted(blocks[b], key=lambda r: r[1])] for b in full], device=x.device)
            rows = x[t].transpose(1, 2)
            sc = _least_scale(rows.abs().amax((-1, -2)), dtype)
            pool[full], scales[full] = _to_grid(rows / sc[..., None, None]), sc
        for b in part:
            t, o = [a for a, _ in blocks[b]], [a for _, a in blocks[b]]
            rows = x[t].transpose(0, 1)                               # [n_kv, rows, d]
            sc = _least_scale(rows.abs().amax((-1, -2)), dtype)
            if 0 not in o:
                sc = torch.maximum(sc, scales[b])
                pool[b] = _to_grid(pool[b] * (scales[b] / sc)[:, None, None])
            pool[b][:, o] = _to_grid(rows / sc[:, None, None])
            scales[b] = sc
        got[name], got[name + "_scales"] = pool[None], scales[None]
    return got


def _exact_attention(s):
    """One sequence and KV head at a time, straight from the formula."""
    c = s["case"]
    lens, d, G = _lens(c), c["d"], c["group"]
    chunk = _chunks(c) if c["op"] == "prefill8" else [1] * c["n_seqs"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if "scores" in s else None
    row = 0
    for i, (length, m) in enumerate(zip(lens, chunk)):
        if length:
            t = s["tables"][i, :-(-length // BLOCK)].long()
            for h in range(c["n_kv"]):
                kv = []
                for name in ("k", "v"):
                    x = s[name + "_pool"][0, t, h].double()
                    if name + "_scales" in s:
                        x = x * s[name + "_scales"][0, t, h].double()[:, None, None]
                    kv.append(x.reshape(-1, d)[:length])
                for a in range(0, m, 512):                            # rows of a long chunk in pieces
                    b = min(m, a + 512)
                    q = s["q"][row + a:row + b, h * G:(h + 1) * G].double().transpose(0, 1)
                    z = q @ kv[0].T / math.sqrt(d)                    # [G, b - a, length]
                    last = length - m + torch.arange(a, b, device="cuda")
                    z = z.masked_fill(torch.arange(length, device="cuda") > last[:, None], NEG)
                    w = torch.softmax(z, -1)
                    out[row + a:row + b, h * G:(h + 1) * G] = (w @ kv[1]).transpose(0, 1)
                    if scores is not None:
                        scores[i, h, :length] += w[:, 0].sum(0)
        row += m
    return {"out": out} if scores is None else {"out": out, "scores": scores}


def _exact_evict(s):
    c = s["case"]
    G8 = c["bits8"]
    pools = {n: s[n + "_pool"].double() for n in ("k", "v")}
    scales = {n: s[n + "_scales"].double() for n in ("k", "v")} if G8 else {}
    new, kept = s["new_scores"].double(), s["kept"].clone()
    scores = s["scores"].double()
    tables, dst = s["tables"].tolist(), s["dst"].tolist()
    for i, (length, keep) in enumerate(zip(_lens(c), _keeps(c))):
        k = min(keep, length)
        if not length:
            continue
        r = min(c["recent"], k)
        old = scores[:, i, :, :length - r]
        order = torch.argsort(-old, dim=-1, stable=True)[..., :k - r]
        newest = torch.arange(length - r, length, device="cuda").expand(*order.shape[:2], r)
        pos = torch.cat([order.sort(-1).values, newest], -1)          # [layers, n_kv, k]
        kept[:, i, :, :k] = pos.int()
        new[:, i, :, :length] = 0
        new[:, i, :, :k] = scores[:, i].gather(-1, pos)
        t = torch.tensor(tables[i], device="cuda")
        u = torch.tensor(dst[i], device="cuda")
        la = torch.arange(c.get("layers", 1), device="cuda")[:, None, None]
        he = torch.arange(c["n_kv"], device="cuda")[None, :, None]
        for n in ("k", "v"):
            rows = pools[n][la, t[pos // BLOCK], he, pos % BLOCK]     # [layers, n_kv, k, d]
            to = torch.arange(k, device="cuda")
            if G8:
                sc = scales[n][la, t[pos // BLOCK], he]
                pad = torch.nn.functional.pad(sc, (0, -k % BLOCK)).view(*sc.shape[:2], -1, BLOCK).amax(-1)
                scales[n][la, u[:pad.shape[-1]], he] = pad
                rows = _to_grid(rows * (sc / pad[..., to // BLOCK])[..., None])
            pools[n][la, u[to // BLOCK], he, to % BLOCK] = rows
    got = {"k": pools["k"], "v": pools["v"], "new_scores": new, "kept": None}
    if G8:
        got.update(k_scales=scales["k"], v_scales=scales["v"])
    return got
