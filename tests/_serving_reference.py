"""The operators of a serving step in 64 bits on the CPU, and the error bounds that the
tests hold the kernels to.

Attention over pages with scales of their own.  The bounds of _attention_reference (one
rounding u = 2^-8 of weights and of the output, scores off by ds, fp32 sums) hold for the
keys and values with their scales multiplied in, and two terms come in:
 * a query element below 2^-9 of its row's largest counts to within 2^-17 of that
   largest: ds grows by 2^-17 max|q| scale sum |k_i| over those elements;
 * a weight times its value's scale, p vs, is held to within u of itself down to a floor
   below which it is off by 2^-34 of the row's largest at most (16-bit weights: fp16
   relative to a reference at which the largest is 2^10 or more, off by 2^-25 below 2^-14;
   sums of E4M3 numbers: the last of them, 2^24 times what the others leave, off by 2^-10,
   where the largest is 1 or more), for each of n keys, times a value of 448 at most.
"""
import math

import torch

from _attention_reference import U

LOW, HIGH = 2.0 ** -40, 2.0 ** 40


def e4m3(x):
    """float64 to E4M3, saturating, ties to even: the nearest of all 253 finite numbers."""
    m, e = torch.frexp(x.abs())                            # m in [0.5, 1)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)   # 8 steps to a binade
    y = torch.round(x.abs() / step) * step                 # (torch.round: ties to even)
    return torch.sign(x) * y.clamp(max=448.0)


def scale_of(top):
    """The smallest power of two s within LOW .. HIGH with top <= 448 s."""
    s = LOW
    while s < HIGH and top > 448.0 * s:
        s *= 2
    return s


def request_attention(q, k, v, vs, pos0, scale, window):
    """One request and key head: q [n, g, D], k and v [L, D] with their scales in, vs [L]
    the values' scales, all double.  (out, lse, bounds), [n, g, ...]."""
    n, g, D = q.shape
    L = k.shape[0]
    pos = pos0 + torch.arange(n)[:, None]
    j = torch.arange(L)
    see = j <= pos
    if window:
        see = see & (j > pos - window)
    see = see[:, None, :].expand(n, g, L)
    s = (q @ k.T * scale).masked_fill(~see, -math.inf)
    small = torch.where(q.abs() < 2.0 ** -9 * q.abs().amax(-1, keepdim=True), 1.0, 0.0)
    ds = (D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * scale
    ds = ds + 2.0 ** -17 * q.abs().amax(-1, keepdim=True) * (small.double() @ k.abs().T) * scale
    none = ~see.any(-1)
    ds = ds.masked_fill(~see, 0.0).amax(-1) if L else torch.zeros(n, g, dtype=torch.float64)
    if L:
        p = torch.where(none[..., None], 0.0, torch.softmax(s, -1))
        lse = torch.logsumexp(s, -1)
        tiny = L * 448 * 2.0 ** -34 * (p * vs).amax(-1)
    else:
        p, lse = s, torch.full((n, g), -math.inf, dtype=torch.float64)
        tiny = torch.zeros(n, g, dtype=torch.float64)
    seen = see.any(0).any(0)
    v = torch.where(seen[:, None], v, 0.0)                # hidden values take no part
    o, ev = p @ v, p @ v.abs()
    b_out = (U + 2 * ds[..., None] + 2.0 ** -18) * ev + U * o.abs() + tiny[..., None]
    b_lse = ds + 2.0 ** -18 * (1 + torch.where(none, 0.0, lse).abs())
    return o, lse, b_out, b_lse


def plan(ring, state, before, cached, new, table, page, rows):
    """attn_plan_pages with lists, request by request: (kv_len, q_start, table, positions,
    slots, ring, state, faults)."""
    table, ring = [list(t) for t in table], list(ring)
    cap = len(table[0]) * page if table else 0
    first, free = state
    faults = set()
    if not (0 <= first < len(ring) and 0 <= free <= len(ring)):
        faults.add(7)
        first = free = 0
    taken, want_pages, want_rows = 0, 0, 0
    kv_len, q_start, positions, slots, back = [], [0], [], [], []
    for r, n in enumerate(new):
        old, stand = before[r], before[r] if cached is None else cached[r]
        if old < 0 or old > cap or (n >= 0 and (stand < 0 or stand > old or stand + n > cap)):
            faults.add(7)
            kv_len.append(old)
            q_start.append(q_start[-1])
            continue
        if n < 0:
            stand = n = 0
        have = -(-old // page)
        take = max(0, -(-(stand + n) // page) - have)
        want_pages += take
        want_rows += n
        if (take and want_pages > free) or (n and want_rows > rows):
            faults.add(8)
            take = n = 0
        need = -(-(stand + n) // page)
        for j in range(have, need):
            table[r][j] = ring[(first + taken) % len(ring)]
            taken += 1
        back += table[r][need:have]
        for p in range(stand, stand + n):
            positions.append(p)
            slots.append(table[r][p // page] * page + p % page)
        kv_len.append(stand + n)
        q_start.append(q_start[-1] + n)
    room = len(ring) - free
    if len(back) > room:
        faults.add(7)
        back = back[:room]
    for j, p in enumerate(back):
        ring[(first + free + j) % len(ring)] = p
    state = [(first + taken) % len(ring), free - taken + len(back)]
    return kv_len, q_start, table, positions, slots, ring, state, faults


def verify(target, draft, tokens, q_start, accept_u, sample_u):
    """draft_verify request by request, in 64 bits: (accepted, next)."""
    def probability(x):
        return torch.nan_to_num(x.double(), nan=0.0).clamp(0, 1)
    accepted, following = [], []
    for r in range(len(q_start) - 1):
        s, n = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r]) - 1
        if n < 0:
            accepted.append(0)
            following.append(-1)
            continue
        k = 0
        while k < n:
            x = int(tokens[s + k + 1])
            if not 0 <= x < target.shape[1]:
                break
            p = float(probability(target[s + k, x]))
            q = 1.0 if draft is None else float(probability(draft[s + k, x]))
            if not float(accept_u[s + k]) * q < p:
                break
            k += 1
        p = probability(target[s + k])
        w = p
        if k < n and draft is None:
            x = int(tokens[s + k + 1])
            if 0 <= x < target.shape[1]:
                w = p.clone()
                w[x] = 0
        elif k < n:
            w = (p - probability(draft[s + k])).clamp(min=0)
        if not (w > 0).any():
            w = p
        accepted.append(k)
        if not (w > 0).any():
            following.append(-1)
            continue
        total = w.cumsum(0)
        u = float(sample_u[r])
        u = max(0.0, u) if u == u else 0.0
        past = torch.nonzero((total > u * total[-1]) & (w > 0))
        following.append(int(past[0]) if len(past) else int(torch.nonzero(w > 0)[-1]))
    return accepted, following
