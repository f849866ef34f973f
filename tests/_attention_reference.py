"""The attention operators in 64 bits on the CPU, token by token, and the error
bounds that the tests hold the kernels to.

Bounds.  u = 2^-8 is the relative error of one rounding to bf16.
 * A transformed head element a cos - b sin is rounded to bf16 once (u |y|);
   its fp32 value is off by at most (D + 16) 2^-24 (|a| + |b|): D + O(10)
   operations go into the norm, a handful into the rotation.
 * A softmax weight is rounded to 16 bits (u at most) for the product with v,
   and the score it comes from is off by ds <= (D + 8) 2^-23 * scale *
   sum_i |q_i k_i| (a dot product of D terms in fp32 that may cut instead of
   rounding).  With E|v| the weighted mean of |v|:
   |out - exact| <= (u + 2 ds + 2^-18) E|v| + u |exact|, and
   |lse - exact| <= ds + 2^-18 (1 + |exact|), where 2^-18 covers the sums of
   fp32 weights and the exponential's approximation.
"""
import math

import torch

U = 2.0 ** -8


def transform(x, weight, pos, rope, interleaved, eps):
    """x [T, H, D] double -> (y, |a| + |b| of each element)."""
    x = x.double()
    D = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if rope is None:
        return x, x.abs()
    half = rope.shape[1] // 2
    y, mag = x.clone(), x.abs()
    cs, sn = rope[pos.long(), :half].double(), rope[pos.long(), half:].double()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cs[:, i, None], sn[:, i, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def transform_bound(y, mag):
    return U * y.abs() + (y.shape[-1] + 16) * 2.0 ** -24 * mag


def key_rows(cache, table_row, page, length, head, heads_first, scale):
    """Keys (or values) 0 .. length-1 of one head, [length, D] double."""
    rows = []
    for j in range(length):
        p = int(table_row[j // page])
        rows.append(cache[p, head, j % page] if heads_first else cache[p, j % page, head])
    if not rows:
        return torch.zeros(0, cache.shape[-1], dtype=torch.float64)
    x = torch.stack(rows).double()
    return x if scale is None else x * float(scale[head])


def attention(q, k_cache, v_cache, q_start, kv_len, table, heads_first=False, k_scale=None,
              v_scale=None, scale=None, window=0):
    """(out, lse, bound of out, bound of lse), double; rows of no request are NaN."""
    T, hq, D = q.shape
    hk, page = (k_cache.shape[1], k_cache.shape[2]) if heads_first else (k_cache.shape[2],
                                                                        k_cache.shape[1])
    g = hq // hk
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, hq), math.nan, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(kv_len)):
        a, e, length = int(q_start[r]), int(q_start[r + 1]), int(kv_len[r])
        n = e - a
        if n == 0:
            continue
        pos = torch.arange(length - n, length)[:, None]
        j = torch.arange(length)
        see = j <= pos
        if window:
            see = see & (j > pos - window)
        for kv in range(hk):
            k = key_rows(k_cache, table[r], page, length, kv, heads_first, k_scale)
            v = key_rows(v_cache, table[r], page, length, kv, heads_first, v_scale)
            for h in range(kv * g, (kv + 1) * g):
                x = q[a:e, h].double()
                s = (x @ k.T * scale).masked_fill(~see, -math.inf)
                ds = (x.abs() @ k.abs().T * scale).masked_fill(~see, 0.0)
                ds = (D + 8) * 2.0 ** -23 * (ds.amax(1) if length else torch.zeros(n).double())
                none = ~see.any(1) if length else torch.ones(n, dtype=torch.bool)
                p = torch.softmax(s, 1) if length else s
                p = torch.where(none[:, None], torch.zeros_like(p), p)
                # hidden values take no part, whatever they are; elementwise, since a
                # matrix product may skip a weight of zero whose value is infinite
                w = [(p[i][see[i]][:, None], v[see[i]]) for i in range(n)]
                o = torch.stack([(a * b).sum(0) for a, b in w])
                ev = torch.stack([(a * b.abs()).sum(0) for a, b in w])
                ls = torch.logsumexp(s, 1) if length else torch.full((n,), -math.inf).double()
                out[a:e, h], lse[a:e, h] = o, ls
                b_out[a:e, h] = (U + 2 * ds[:, None] + 2.0 ** -18) * ev + U * o.abs()
                b_lse[a:e, h] = ds + 2.0 ** -18 * (1 + torch.where(none, 0.0, ls).abs())
    return out, lse, b_out, b_lse
