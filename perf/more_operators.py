"""The operators of a hybrid model's serving step, measured: linear attention with a decay for each head (packed
prompts in chunks, and one token a sequence) over a pool of fixed-size states, and a step's block tables, slot map
and query starts built on the GPU from request lengths.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the library's entry points. ``exact`` restates each operator in 64 bits.

Linear attention, head h of v reading head h // (n_v / n_qk) of q and k, g the log of the decay:
    S_t = exp(g_t) S_{t-1} + k_t^T v_t,   o_t = scale * q_t S_t,   S [dim_k, dim_v] in float32.
Layouts: q, k [tokens, n_qk, dim_k]; v, out [tokens, n_v, dim_v]; state [layers, slots, n_v, dim_k, dim_v]; log decay
[tokens, n_v], [n_v] or none. Sequence s reads its state from slot src[s] (negative: zeros) and leaves it in dst[s].

Tables: a row of length len gets new tokens; blocks of 16 come from a list of free ones, in row order, each row whole or
not at all; the first row that does not fit, and those behind it, get nothing. slot = block * 16 + position % 16.
"""
import math

import torch

own = False

BLOCK = 16
CHUNK = 128                                   # tokens that the plain prompt form takes at once
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ----------------------------------------------------------------------------------------

def _linear(name, op, dtype, n_qk, group, dk, dv, n_seqs, lo, hi, gates, fresh):
    return dict(name=name, op=op, dtype=dtype, n_qk=n_qk, group=group, dk=dk, dv=dv, n_seqs=n_seqs, lo=lo, hi=hi,
                gates=gates, fresh=fresh)


def _tables(name, n_seqs, lo, hi, new_lo, new_hi, share):
    return dict(name=name, op="tables", n_seqs=n_seqs, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, share=share)


def listed():
    return [
        # one decode step of the GPT-style batch: a token each, a new block for one row in 16
        _tables("tables step", 64, 64, 2048, 1, 1, 1.0),
        # shared-prefix churn: 200 sequences, some decoding, some a chunk into their prompts, not quite enough blocks
        _tables("tables mixed", 200, 0, 1535, 1, 512, 0.9),
        # a queue of prompts (64..512 tokens) admitted at once from nothing
        _tables("tables prompts", 1000, 0, 0, 64, 512, 1.0),
        # a single session of the hybrid model: latency
        _linear("decode one", "decode", "bf16", 16, 3, 128, 128, 1, 1, 1, "token", False),
        # the GPT-style batch's heads, a constant decay for each head
        _linear("decode batch", "decode", "f16", 32, 1, 128, 128, 64, 1, 1, "head", False),
        # a small state (128 x 64) for many sequences
        _linear("decode many", "decode", "bf16", 8, 4, 128, 64, 250, 1, 1, "token", False),
        # a few short follow-up prompts in one step
        _linear("prefill turns", "prefill", "f16", 8, 4, 64, 64, 4, 25, 70, "head", False),
        # one chunk of a long document late in its prompt
        _linear("prefill chunk", "prefill", "bf16", 16, 3, 128, 128, 1, 2432, 2432, "token", False),
        # prompts of the GPT-style batch packed together, from nothing
        _linear("prefill packed", "prefill", "f16", 32, 1, 128, 128, 16, 64, 2048, "head", True),
        # few heads, one document
        _linear("prefill few heads", "prefill", "bf16", 2, 4, 128, 64, 1, 9005, 9005, "token", True),
        # the precision mode
        _linear("prefill f32", "prefill", "f32", 8, 1, 64, 64, 3, 61, 500, "token", False),
        # a whole long document of the hybrid model
        _linear("prefill long", "prefill", "bf16", 16, 3, 128, 128, 1, 32768, 32768, "token", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "decode", "decode", "prefill", "prefill", "prefill"])
    while True:
        n_seqs = _log(rng, 1, 1000 if op == "tables" else 250 if op == "decode" else 64)
        hi = _log(rng, 1, 32768)
        lo = hi if n_seqs == 1 else _log(rng, 1, hi) - rng.choice([0, 1])
        if op == "tables":
            new_hi = rng.choice([1, _log(rng, 1, 2500)])
            c = _tables("", n_seqs, lo, hi, rng.choice([0, 1]), new_hi, rng.choice([1.0, round(rng.uniform(0.3, 1.2), 2)]))
            cost_ok = n_seqs * new_hi <= 600_000 and n_seqs * hi <= 4_000_000
        else:
            dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
            if op == "decode":
                lo = hi = 1
            elif dtype == "f32":
                hi = min(hi, 600)
                lo = min(lo, hi)
            c = _linear("", op, dtype, _log(rng, 1, 32), rng.choice([1, 2, 3, 4]), rng.choice([64, 128]),
                        rng.choice([64, 128]), n_seqs, lo, hi, rng.choice(["token", "head", "none"]), rng.random() < 0.4)
            n_v, tokens = c["n_qk"] * c["group"], sum(_lens(c))
            state = n_seqs * n_v * c["dk"] * c["dv"]
            cost_ok = (0 < tokens and n_v <= 64 and state <= 50e6 and tokens * n_v * c["dk"] * c["dv"] <= 25e9
                       and state * -(-hi // CHUNK) <= 200e6)
        del c["name"]
        if cost_ok:
            return c


def _spread(n, lo, hi, at=0.37):
    """n numbers over [lo, hi] by a fixed irrational step: they follow from the case alone."""
    out = [lo + int(((i * 0.6180339887498949 + at) % 1.0) * (hi - lo + 1)) for i in range(n)]
    out[0] = hi
    if n > 1:
        out[-1] = lo
    return out


def _lens(case):
    """Tokens of each sequence (linear attention), or cached tokens of each row (tables)."""
    return _spread(case["n_seqs"], case["lo"], case["hi"])


def _news(case):
    """New tokens of each row; every third row decodes one where the others bring chunks."""
    new = _spread(case["n_seqs"], case["new_lo"], case["new_hi"], 0.71)
    return [1 if case["lo"] < case["hi"] and i % 3 == 2 else m for i, m in enumerate(new)]


def _blocks(n):
    return -(-n // BLOCK)


def _needs(case):
    return [_blocks(c + m) - _blocks(c) for c, m in zip(_lens(case), _news(case))]


# ---- inputs ---------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = case["n_seqs"]
    s = dict(case=dict(case))
    if case["op"] == "tables":
        lens, new = _lens(case), _news(case)
        held, need = sum(_blocks(c) for c in lens), sum(_needs(case))
        free = int(math.ceil(need * case["share"]))              # a share under 1: the last rows do not fit
        used = 5                                                 # taken by earlier steps
        s["nb"] = nb = held + free + used + 3
        perm = torch.randperm(nb, device=dev, generator=g).to(torch.int32)
        s["mb"] = mb = max(max(_blocks(c + m) for c, m in zip(lens, new)), 1) + 2
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        count = (s["lens"] + BLOCK - 1) // BLOCK
        first = torch.cumsum(count, 0) - count
        j = torch.arange(mb, device=dev)
        s["tables"] = torch.where(j < count[:, None], perm[(first[:, None] + j).clamp(max=nb - 1)], -1).to(torch.int32)
        s["free"] = perm[held:held + used + free].contiguous()
        s["used"] = torch.tensor([used], dtype=torch.int32, device=dev)
        s["max_tokens"] = sum(new)
        s["slots"] = torch.empty(max(s["max_tokens"], 1), dtype=torch.int64, device=dev)
        s["start"] = torch.empty(n + 1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty_like(s["lens"])
        s["totals"] = torch.empty(3, dtype=torch.int32, device=dev)
        return s
    lens, dt = _lens(case), TORCH[case["dtype"]]
    n_qk, n_v, dk, dv = case["n_qk"], case["n_qk"] * case["group"], case["dk"], case["dv"]
    tokens = sum(lens)
    # keys and queries of length one, as such layers normalise them; values about 1
    q, k = (torch.randn((tokens, n_qk, dk), device=dev, generator=g) for _ in range(2))
    s["q"], s["k"] = (x.div_(x.norm(dim=-1, keepdim=True)).to(dt) for x in (q, k))
    s["v"] = torch.randn((tokens, n_v, dv), device=dev, generator=g).to(dt)
    s["out"] = torch.empty_like(s["v"])
    # decays: half lives of a few to a few thousand tokens, the heads' own, and the tokens' own about them
    rate = torch.exp(-7.5 * torch.rand(n_v, device=dev, generator=g))
    s["g"] = None
    if case["gates"] == "head":
        s["g"] = -0.7 * rate
    elif case["gates"] == "token":
        s["g"] = -0.7 * rate * torch.exp(torch.randn((tokens, n_v), device=dev, generator=g))
    slots = n + 2
    s["state"] = torch.randn((1, slots, n_v, dk, dv), device=dev, generator=g)
    s["dst"] = torch.randperm(slots, device=dev, generator=g)[:n].to(torch.int32)
    s["src"] = torch.full_like(s["dst"], -1) if case["fresh"] else s["dst"].clone()
    starts = torch.tensor([0] + lens).cumsum(0)
    s["start"] = starts.to(torch.int32).to(dev)
    s["longest"] = max(lens)
    s["scale"] = 1.0 / math.sqrt(dk)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"tables": _plain_tables, "decode": _plain_decode, "prefill": _plain_prefill}[op](s)


def _own(s, op):
    """The library's calls. What a program that serves keeps from step to step (descriptor, workspace, the launcher
    of its step buffers) is made at a state's first pass."""
    from paged_kv_cache_258_gb300 import pkv
    c = s["case"]
    if op == "tables":
        if "launch" not in s:
            s["launch"] = pkv.extend_tables_launcher(s["nb"], s["free"], s["used"], s["tables"], s["lens"], s["new"],
                                                     s["slots"][:s["max_tokens"]], s["start"], s["new_lens"], s["totals"])
        s["launch"]()
        return _tables_out(s)
    if "desc" not in s:
        n_v = c["n_qk"] * c["group"]
        s["desc"] = pkv.make_linear_desc(c["dtype"], 1, s["state"].shape[1], c["n_qk"], n_v, c["dk"], c["dv"])
        if op == "decode":
            g = s["g"] if s["g"] is None else s["g"][None]
            s["launch"] = pkv.linear_decode_launcher(s["desc"], s["q"][None], s["k"][None], s["v"][None], g, s["state"],
                                                     s["src"], s["dst"], s["scale"], s["out"][None])
        else:
            s["ws"] = pkv.alloc_linear_prefill_workspace(s["desc"], c["n_seqs"], s["q"].shape[0], s["longest"])
    if op == "decode":
        s["launch"](0)
    else:
        pkv.pkv_linear_prefill(s["desc"], 0, s["q"], s["k"], s["v"], s["g"], s["state"], s["src"], s["dst"], s["start"],
                               s["longest"], s["scale"], s["out"], s["ws"])
    return {"out": s["out"], "state": s["state"]}


def _tables_out(s):
    return {"tables": s["tables"], "slots": s["slots"][:s["max_tokens"]], "start": s["start"],
            "lens": s["new_lens"], "totals": s["totals"]}


def _plain_tables(s):
    lens, new, tables, free = s["lens"].long(), s["new"].long(), s["tables"], s["free"]
    n, mb = tables.shape
    dev = lens.device
    old, want = (lens + BLOCK - 1) // BLOCK, (lens + new + BLOCK - 1) // BLOCK
    used = s["used"].long()
    fits = (torch.cumsum(want - old, 0) <= free.numel() - used) & (torch.cumsum(new, 0) <= s["max_tokens"]) & (want <= mb)
    served = torch.cumsum((~fits).long(), 0) == 0
    new, want = torch.where(served, new, 0), torch.where(served, want, old)
    end, taken = torch.cumsum(new, 0), torch.cumsum(want - old, 0)
    s["start"][0] = 0
    s["start"][1:] = end
    s["new_lens"].copy_(lens + new)
    s["totals"].copy_(torch.stack([(used + taken[-1:])[0], served.sum(), end[-1]]))
    j = torch.arange(mb, device=dev)
    fresh = (j >= old[:, None]) & (j < want[:, None])
    if free.numel():
        at = (used + (taken - (want - old))[:, None] + j - old[:, None]).clamp(0, free.numel() - 1)
        tables.copy_(torch.where(fresh, free[at], tables))
    t = torch.arange(s["max_tokens"], device=dev)
    row = torch.searchsorted(end, t, right=True).clamp(max=n - 1)
    pos = (lens[row] + t - (end - new)[row]).clamp(min=0)
    block = tables[row, (pos // BLOCK).clamp(max=mb - 1)].long()
    s["slots"][:s["max_tokens"]] = torch.where(t < end[-1], block * BLOCK + pos % BLOCK, -1)
    return _tables_out(s)


def _before(s):
    """The states that the sequences start from [n, n_v, dk, dv]."""
    src = s["src"].long()
    x = s["state"][0][src.clamp(min=0)]
    return torch.where((src >= 0)[:, None, None, None], x, torch.zeros_like(x))


def _plain_decode(s):
    group = s["case"]["group"]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    x = _before(s)
    if s["g"] is not None:
        x = x * torch.exp(s["g"])[..., None, None]
    x = x + k[..., None] * s["v"].float()[:, :, None]
    s["out"].copy_(((q * s["scale"])[:, :, None] @ x)[:, :, 0])
    s["state"][0, s["dst"].long()] = x
    return {"out": s["out"], "state": s["state"]}


def _plain_prefill(s):
    c = s["case"]
    n, n_v, dk, dv, group = c["n_seqs"], c["n_qk"] * c["group"], c["dk"], c["dv"], c["group"]
    dev, C = s["q"].device, min(CHUNK, s["longest"])
    nc = -(-s["longest"] // C)
    start, count = s["start"][:-1].long(), s["start"].diff().long()
    i = torch.arange(nc * C, device=dev)
    inside = i < count[:, None]
    rows = torch.where(inside, start[:, None] + i, 0)

    def take(x):                                                      # [n, heads, nc, C, ...], zero behind a sequence
        y = x.float()[rows] * inside.view(n, -1, *(1,) * (x.dim() - 1))
        return y.view(n, nc, C, *x.shape[1:]).transpose(2, 3).transpose(1, 2)

    q, k = (take(s[x]).repeat_interleave(group, 1) for x in ("q", "k"))
    v = take(s["v"])
    g = s["g"]
    if g is None:
        g = torch.zeros(n_v, device=dev)
    if g.dim() == 1:
        g = g.expand(s["q"].shape[0], n_v)
    g = take(g).double()                                              # [n, n_v, nc, C]
    G = torch.cumsum(g, -1)
    last = G[..., -1:]
    below = torch.ones((C, C), dtype=torch.bool, device=dev).tril()
    D = torch.exp(torch.where(below, G[..., :, None] - G[..., None, :], -math.inf).float())
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    u = (k * torch.exp((last - G).float())[..., None]).transpose(-1, -2) @ v      # what each chunk adds
    E = torch.nn.functional.pad(torch.cumsum(last[..., 0], -1), (1, 0))           # [n, n_v, nc + 1]
    earlier = torch.ones((nc + 1, nc), dtype=torch.bool, device=dev).tril(-1)
    M = torch.exp(torch.where(earlier, E[..., :, None] - E[..., None, 1:], -math.inf).float())
    x = (M @ u.reshape(n, n_v, nc, dk * dv)).view(n, n_v, nc + 1, dk, dv)
    x += torch.exp(E.float())[..., None, None] * _before(s)[:, :, None]
    o += torch.exp(G.float())[..., None] * (q @ x[:, :, :-1])
    o = (o * s["scale"]).transpose(1, 2).transpose(2, 3).reshape(n, nc * C, n_v, dv)
    s["out"][rows[inside]] = o[inside].to(s["out"].dtype)
    s["state"][0, s["dst"].long()] = x[:, :, -1]
    return {"out": s["out"], "state": s["state"]}


# ---- the work of one pass -------------------------------------------------------------------------

def work(case):
    if case["op"] == "tables":
        n, need, new = case["n_seqs"], sum(_needs(case)), sum(_news(case))
        return {"bytes": 16 * n + 8 * int(need * min(case["share"], 1.0)) + 8 * new, "flops": new}
    n, n_qk, n_v, dk, dv = case["n_seqs"], case["n_qk"], case["n_qk"] * case["group"], case["dk"], case["dv"]
    tokens, e = sum(_lens(case)), 4 if case["dtype"] == "f32" else 2
    rows = tokens * (2 * n_qk * dk + 2 * n_v * dv) * e
    gates = {"none": 0, "head": 4 * n_v, "token": 4 * n_v * tokens}[case["gates"]]
    states = n * n_v * dk * dv * 4 * (1 if case["fresh"] else 2)
    return {"bytes": rows + gates + states + 12 * n, "flops": 4 * tokens * n_v * dk * dv}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_tables(s) if case["op"] == "tables" else _exact_linear(s)


def _exact_tables(s):
    """Row after row and token after token, as a block manager appends them."""
    free, used, tables = s["free"].tolist(), s["used"].item(), s["tables"].tolist()
    lens, start, slots, served, open_ = s["lens"].tolist(), [0], [], 0, True
    for i, m in enumerate(s["new"].tolist()):
        need = _blocks(lens[i] + m) - _blocks(lens[i])
        open_ = open_ and used + need <= len(free) and len(slots) + m <= s["max_tokens"] and _blocks(lens[i] + m) <= s["mb"]
        if open_:
            served += 1
            for _ in range(m):
                if lens[i] % BLOCK == 0:
                    tables[i][lens[i] // BLOCK] = free[used]
                    used += 1
                slots.append(tables[i][lens[i] // BLOCK] * BLOCK + lens[i] % BLOCK)
                lens[i] += 1
        start.append(len(slots))
    pad = [-1] * (s["max_tokens"] - len(slots))
    return {"tables": torch.tensor(tables, dtype=torch.int32), "slots": torch.tensor(slots + pad, dtype=torch.int64),
            "start": torch.tensor(start, dtype=torch.int32), "lens": torch.tensor(lens, dtype=torch.int32),
            "totals": torch.tensor([used, served, len(slots)], dtype=torch.int32)}


def _exact_linear(s):
    """The recurrence, 32 tokens at a time: with a = exp of the summed log decays from the piece's front to a token,
    the state and outputs follow from the state before the piece and the pairs inside it."""
    c = s["case"]
    group, n_v = c["group"], c["n_qk"] * c["group"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    state = s["state"].double()
    at = s["start"].tolist()
    head = torch.arange(n_v, device="cuda") // group
    for i, (src, dst) in enumerate(zip(s["src"].tolist(), s["dst"].tolist())):
        x = state[0, src].clone() if src >= 0 else torch.zeros_like(state[0, 0])
        for a in range(at[i], at[i + 1], 32):
            b = min(a + 32, at[i + 1])
            q, k = s["q"][a:b].double().transpose(0, 1)[head], s["k"][a:b].double().transpose(0, 1)[head]
            v = s["v"][a:b].double().transpose(0, 1)
            if s["g"] is None:
                g = torch.zeros((n_v, b - a), dtype=torch.float64, device="cuda")
            else:
                g = s["g"].double().expand(s["q"].shape[0], n_v)[a:b].T
            run_ = torch.cumsum(g, 1)
            pair = run_[:, :, None] - run_[:, None, :]
            pair = torch.exp(pair.masked_fill(torch.arange(b - a, device="cuda")[:, None] < torch.arange(b - a, device="cuda"), -math.inf))
            inter = torch.einsum("htk,hkv->htv", q, x) * torch.exp(run_)[..., None]
            inner = ((q @ k.mT) * pair) @ v
            out[a:b] = ((inter + inner) / math.sqrt(c["dk"])).transpose(0, 1)
            x = torch.exp(run_[:, -1])[:, None, None] * x + torch.einsum("hjk,hj,hjv->hkv", k, pair[:, -1], v)
        state[0, dst] = x
    return {"out": out, "state": state}
