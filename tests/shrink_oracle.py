"""Plain 64-bit restatements of the cache-shrinking calls for the tests: 8-bit pools, decode with summed
weights, eviction. numpy only; shares no code with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 16
MIN_EXP = {"f16": -15, "bf16": -117}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # of a rounding, relative to the value


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        out[c] = np.nan if c & 0x7F == 0x7F else sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return out


VALUES = e4m3_values()
_POS = VALUES[:127]


def to_codes(x: np.ndarray) -> np.ndarray:
    """Nearest code of each x (|x| <= 448), halfway to the even one; NaN to the NaN code of its sign bit."""
    a = np.abs(x)
    up = np.clip(np.searchsorted(_POS, a), 0, 126)
    down = np.maximum(up - 1, 0)
    du, dd = _POS[up] - a, a - _POS[down]
    code = np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)
    code = np.where(np.isnan(x), 127, code)
    return (code | (np.signbit(x) * 128)).astype(np.uint8)


def least_scale(amax: float, dtype: str) -> float:
    e = MIN_EXP[dtype]
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, slots, codes, scales, dtype) -> None:
    """Rows x [n_tok, n_kv, d] (float64) into codes uint8 [nb, n_kv, 16, d], scales [nb, n_kv], in place."""
    nb = codes.shape[0]
    blocks: dict[int, dict[int, int]] = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < nb * BLOCK:
            blocks.setdefault(int(slot) // BLOCK, {})[int(slot) % BLOCK] = t
    for b, rows in blocks.items():
        for g in range(codes.shape[1]):
            new = np.stack([x[t, g] for t in rows.values()])
            fin = np.abs(new[np.isfinite(new)])
            need = least_scale(fin.max() if fin.size else 0.0, dtype)
            old = scales[b, g]
            s = need if 0 in rows else max(old, need)
            if 0 not in rows and s != old:
                for r in range(BLOCK):
                    if r not in rows:
                        codes[b, g, r] = to_codes(VALUES[codes[b, g, r]] * (old / s))
            for r, t in rows.items():
                codes[b, g, r] = to_codes(np.where(np.isfinite(x[t, g]), x[t, g] / s, np.nan))
            scales[b, g] = s


def widen(codes, scales) -> np.ndarray:
    return VALUES[codes] * scales[..., None, None].astype(np.float64)


def rows_of(pool, table, length, g) -> np.ndarray:
    """The first `length` rows of KV head g, in order (float64)."""
    n = -(-length // BLOCK)
    return pool[np.asarray(table[:n], dtype=np.int64), g].reshape(-1, pool.shape[-1])[:length].astype(np.float64)


def attend(q, k, v, scale):
    """One query row over rows k, v: (out, weights, bound data). q [d], k, v [n, d] in float64."""
    z = (k @ q) * scale
    w = np.exp(z - z.max())
    w /= w.sum()
    return w @ v, w


def decode(q, k_pool, v_pool, tables, lens, scale, dtype, p_step):
    """(out, out tolerance, weights [n, n_kv, S], their tolerance) of decode over float64 pools
    [nb, n_kv, 16, d]. p_step: half a step of the type the kernel rounds its weights to.

    Tolerances, worst case: a logit is a dot product of d terms in fp32, then two more roundings and an
    exp2 within 2 ulp, so it is off by dz = 2^-24 (d + 8) (scale sum|q||k| + |z|) and a weight by a factor
    1 +- (2 dz + 2^-21) (its own and the sum's). The output adds the weights' rounding p_step and, for
    the sums of n terms in fp32, n 2^-24, all relative to sum w|v|, then its own rounding.
    """
    n, n_q, d = q.shape
    n_kv = k_pool.shape[1]
    G = n_q // n_kv
    S = tables.shape[1] * BLOCK
    out, tol = np.zeros((n, n_q, d)), np.zeros((n, n_q, d))
    w_sum, w_tol = np.zeros((n, n_kv, S)), np.zeros((n, n_kv, S))
    for s in range(n):
        c = int(lens[s])
        if c == 0:
            continue
        for h in range(n_q):
            g = h // G
            k, v = rows_of(k_pool, tables[s], c, g), rows_of(v_pool, tables[s], c, g)
            o, w = attend(q[s, h], k, v, scale)
            z = np.abs(k) @ np.abs(q[s, h]) * abs(scale)
            dz = 2.0 ** -24 * (d + 8) * 2 * z.max()
            rel = 2 * dz + 2.0 ** -21
            size = w @ np.abs(v)
            out[s, h] = o
            err = (rel + p_step + c * 2.0 ** -24) * size
            tol[s, h] = err + HALF_STEP[dtype] * (np.abs(o) + err) + {"f16": 2.0 ** -25, "bf16": 0.0}[dtype]
            w_sum[s, g, :c] += w
            w_tol[s, g, :c] += rel * w + 2.0 ** -30
    return out, tol, w_sum, w_tol


def evict(pools, scales, src, dst, lens, keep, recent, scores, new_scores, kept) -> None:
    """In place on pools (list of [L, nb, n_kv, 16, d] arrays, or codes with scales [L, nb, n_kv])."""
    L, n, n_kv, _ = scores.shape
    before = [p.copy() for p in pools]
    before_s = [s.copy() for s in scales] if scales else None
    old_scores = scores.copy()
    for layer in range(L):
        for s in range(n):
            c = int(lens[s])
            k = min(int(keep[s]), c)
            r = min(recent, k)
            for g in range(n_kv):
                x = old_scores[layer, s, g, :c - r].astype(np.float64)
                key = np.where(np.isnan(x), np.inf, x)
                nan = np.isnan(x)
                order = sorted(range(c - r), key=lambda j: (not nan[j], -key[j], j))[:k - r]
                pos = sorted(order) + list(range(c - r, c))
                kept[layer, s, g, :k] = pos
                new_scores[layer, s, g, :c] = 0
                new_scores[layer, s, g, :k] = old_scores[layer, s, g, pos]
                for i in range(len(pools)):
                    for b in range(-(-k // BLOCK)):
                        rows = pos[b * BLOCK:(b + 1) * BLOCK]
                        if scales:
                            top = max(before_s[i][layer, src[s, j // BLOCK], g] for j in rows)
                            scales[i][layer, dst[s, b], g] = top
                        for a, j in enumerate(rows):
                            row = before[i][layer, src[s, j // BLOCK], g, j % BLOCK]
                            if scales:
                                f = before_s[i][layer, src[s, j // BLOCK], g]
                                row = row if f == top else to_codes(VALUES[row] * (f / top))
                            pools[i][layer, dst[s, b], g, a] = row
