"""Linear attention in 64 bits, token after token, with bounds on what the kernels' roundings may move.

For every sum of products the bound carries the sum of the products' absolute values: with
    A_t = exp(g_t) A_{t-1} + |k_t|^T |v_t|        (A_0 = |S_0|)
a relative error e of each term moves S_t by at most e A_t and out_t by at most e scale |q_t| A_t.
"""
import torch

LEAST = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}   # fp16 below 2^-14 holds multiples of 2^-24: off by up to half of that
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # half of the distance to the next number


def linear(q, k, v, g, state, src, dst, start, scale, dtype):
    """(out, its tolerance, state after, its tolerance), float64 on the CPU. q, k [T, n_qk, dk]; v [T, n_v, dv]; g
    [T, n_v]; state [slots, n_v, dk, dv]; rows of no sequence stay NaN, with a tolerance of NaN.

    The roundings counted, relative to each term:
      fp32 arithmetic: a term passes through its product, one addition a token behind it (a sum in any order has no
        more), the decays' exponentials (each exact to 2 units, their arguments summed in fp32: an error of
        2^-24 |G| (n + 2) for a sum of n terms of which the whole is G, and exp(G) |G| <= 1) and dk additions over q:
        (2 n + dk + 16) 2^-24 for the n-th token
      16-bit types: the weight q.k of a pair inside a chunk, or the element of the state through which a token sees an
        earlier one, is rounded to the type (half a step, one of the two for each term), and the result once more. The
        state gains values split into numbers of the type, two of fp16 or three of bf16: 2^-22 or less is left out.
    """
    h = HALF_STEP[dtype]
    n_v, group = v.shape[1], v.shape[1] // q.shape[1]
    q, k, v, g = (x.double().cpu() for x in (q, k, v, g))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    out = torch.full(v.shape, float("nan"), dtype=torch.float64)
    tol = out.clone()
    after = state.double().cpu().clone()
    after_tol = torch.zeros_like(after)
    before = after.clone()
    for s, (a, b) in enumerate(zip(start[:-1], start[1:])):
        x = before[src[s]].clone() if src[s] >= 0 else torch.zeros_like(before[0])
        y = x.abs()
        n = 0
        for t in range(a, b):
            e = torch.exp(g[t])[:, None, None]
            e = torch.where(e == 0, 0.0, e)
            x = torch.where(e == 0, torch.zeros_like(x), e * x) + k[t][:, :, None] * v[t][:, None, :]
            y = torch.where(e == 0, torch.zeros_like(y), e * y) + (k[t][:, :, None] * v[t][:, None, :]).abs()
            n += 1
            fp32 = (2 * n + q.shape[2] + 16) * 2.0 ** -24
            out[t] = scale * torch.einsum("hk,hkv->hv", q[t], x)
            reach = scale * torch.einsum("hk,hkv->hv", q[t].abs(), y)
            tol[t] = (fp32 + (h * (1 + h) if dtype != "f32" else 0.0)) * reach + h * out[t].abs() + LEAST[dtype]
        if dst[s] >= 0:
            after[dst[s]] = x
            if b > a:
                after_tol[dst[s]] = ((2 * n + 16) * 2.0 ** -24 + (2.0 ** -22 if dtype != "f32" else 0.0)) * y
    return out, tol, after, after_tol
