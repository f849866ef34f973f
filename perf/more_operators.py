"""Operators of a serving step with drafted tokens on an 8-bit paged cache: cases, inputs, plain forms and exact values.

Four operators, in the order in which a step calls them:

  plan     lengths, page tables, row offsets, positions and cache slots of a step, from the tokens that each request
           brings, with pages taken from and given back to a pool
  append   norm and rotation of new keys, quantised with the new values to E4M3 pages that have one scale, a power of
           two, for each page and head; the queries' transform in the same call
  attend   causal attention of each request's new tokens over such a cache
  verify   drafted tokens held against the target's probabilities with given random numbers: how many of each request
           stand, and the token that follows them

With `own` false, run() computes them in elementary torch operations; with `own` true it makes the calls of
nvfp4_block_scaled_route_gb300.binding.  The head layout of most cases is that of the repository's hidden size,
7168 = 56 heads of 128, with 8 heads of keys; batches of 64 and prompts of up to 16384 tokens are its workloads'.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 10000.0
TOP = 448.0                       # the largest E4M3 number
LOW, HIGH = -40, 40               # exponents of page scales


# ------------------------------------------------------------------ cases --
def listed():
    wide = {"hq": 56, "hkv": 8, "d": 128}
    full = {"rot": 128, "norm": True, "pairs": False, **wide}
    return [
        # a decode step of a full batch, a drafted token or two in some, a few requests that end: latency
        {"name": "plan-64x3", "op": "plan", "batch": 64, "new": 3, "ctx": 4096, "page": 64, "ends": 0.05},
        # a step that takes up many prompts at once, 16-token pages
        {"name": "plan-300x100", "op": "plan", "batch": 300, "new": 100, "ctx": 300, "page": 16, "ends": 0.1},
        # one token for each of 64 requests of uneven length: a decode step
        {"name": "append-64x1", "op": "append", "batch": 64, "new": 1, "ctx": 4096, "page": 16, "heads_first": True,
         **full},
        # up to five drafted tokens for each of 16 requests
        {"name": "append-16x5", "op": "append", "batch": 16, "new": 5, "ctx": 6000, "page": 64, "heads_first": False,
         **full},
        # three uneven prompts of up to 8192 tokens
        {"name": "append-3x8192", "op": "append", "batch": 3, "new": 8192, "ctx": 8192, "page": 64,
         "heads_first": False, **full},
        # one token of one request with a short history: latency
        {"name": "decode-1x1000", "op": "attend", "batch": 1, "new": 1, "ctx": 1000, "page": 16, "heads_first": False,
         "window": 0, **wide},
        # the full decode batch, uneven histories of up to 16384 tokens, small pages
        {"name": "decode-64x16384", "op": "attend", "batch": 64, "new": 1, "ctx": 16384, "page": 16,
         "heads_first": False, "window": 0, **wide},
        # up to five drafted tokens checked for each of 16 requests
        {"name": "drafts-16x5", "op": "attend", "batch": 16, "new": 5, "ctx": 6000, "page": 32, "heads_first": True,
         "window": 0, **wide},
        # the last chunk of a long prompt: 2048 tokens over the 14336 that the cache holds already
        {"name": "chunk-2048-of-16384", "op": "attend", "batch": 1, "new": 2048, "ctx": 16384, "page": 64,
         "heads_first": False, "window": 0, **wide},
        # uneven prompts with 64-wide heads, as many heads of keys as of queries, attention within a window
        {"name": "prompts-6x1500-window", "op": "attend", "batch": 6, "new": 1500, "ctx": 2500, "page": 128,
         "heads_first": True, "window": 700, "hq": 24, "hkv": 24, "d": 64},
        # two requests with four drafted tokens each, a small odd vocabulary, tokens guessed without probabilities
        {"name": "verify-2x4", "op": "verify", "batch": 2, "drafts": 4, "vocab": 32003, "half": False, "given": False,
         "off": 0.2},
        # a full batch with up to five drafted tokens each
        {"name": "verify-64x5", "op": "verify", "batch": 64, "drafts": 5, "vocab": 129280, "half": False,
         "given": True, "off": 0.2},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["plan", "append", "attend", "attend", "verify"])
        if op == "verify":
            c = {"op": op, "batch": _spread(rng, 1, 256), "drafts": rng.randint(1, 8),
                 "vocab": _spread(rng, 1000, 262144), "half": rng.random() < 0.3, "given": rng.random() < 0.7,
                 "off": rng.choice([0.05, 0.2, 0.5])}
            if c["batch"] * (c["drafts"] + 1) * c["vocab"] > 1 << 28:
                continue
        elif op == "plan":
            batch = _spread(rng, 1, 1024)
            new = _spread(rng, 1, max(1, 32768 // batch))
            c = {"op": op, "batch": batch, "new": new, "ctx": new + _spread(rng, 1, 16384) - 1,
                 "page": rng.choice([16, 32, 64, 128]), "ends": rng.choice([0.0, 0.1])}
            if batch * c["ctx"] > 1 << 21:
                continue
        else:
            d = rng.choice([64, 128, 128])
            hkv = rng.choice([1, 2, 3, 4, 8, 8])
            batch = _spread(rng, 1, 64)
            new = _spread(rng, 1, max(1, 16384 // batch)) if rng.random() < 0.6 else rng.randint(1, 6)
            c = {"op": op, "batch": batch, "new": new, "ctx": new + _spread(rng, 1, 65536) - 1,
                 "page": rng.choice([16, 32, 64, 128, 256]), "heads_first": rng.random() < 0.5, "d": d, "hkv": hkv,
                 "hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])}
            if c["hq"] > 64 or batch * c["ctx"] > 1 << 20:
                continue
            if op == "append":
                c.update(rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.7, pairs=rng.random() < 0.3)
            else:
                c.update(window=0 if rng.random() < 0.7 else _spread(rng, 16, 8192))
                # what the plain form holds of scores at once
                if batch * new * c["ctx"] * c["hq"] > 2 << 30:
                    continue
        if _cost(c) <= top:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(case):
    """New tokens and cache length (new ones counted) of each request: they go by the case alone."""
    b, new, ctx = case["batch"], case["new"], case["ctx"]
    rng = random.Random(1000003 * b + 10007 * new + ctx)
    ns = [new] + [rng.randint((new + 1) // 2, new) for _ in range(b - 1)]
    lens = [ctx] + [n + _spread(rng, max(1, (ctx - new + 1) // 16), max(1, ctx - new + 1)) - 1 for n in ns[1:]]
    return ns, lens


def _steps(case):
    """For a plan: each request's length after the step before, how many of those tokens stand, and its new tokens
    (-1: it ends).  They go by the case alone."""
    ns, lens = _lengths(case)
    rng = random.Random(77 * case["batch"] + case["ctx"])
    before = [length - n for n, length in zip(ns, lens)]
    stand = [max(0, p - (rng.randint(0, 4) if rng.random() < 0.5 else 0)) for p in before]
    new = [-1 if r > 0 and rng.random() < case["ends"] else n for r, n in enumerate(ns)]
    return before, stand, new


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rope_table(positions, rot):
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _scale_of(top):
    """The smallest power of two s with top <= 448 s, within 2^LOW .. 2^HIGH."""
    m, e = torch.frexp(top)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(top > 0, k, LOW).clamp(LOW, HIGH).double()).float()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "plan":
        _prepare_plan(s, g)
    elif case["op"] == "verify":
        _prepare_verify(s, g)
    else:
        _prepare_cache(s, g)
    if own:
        s["own"] = _handles(s)
    return s


def _prepare_plan(s, g):
    case, page = s["case"], s["case"]["page"]
    before, stand, new = _steps(case)
    held = [-(-n // page) for n in before]
    need = [0 if n < 0 else -(-(c + n) // page) for c, n in zip(stand, new)]
    pages = sum(held) + sum(need) + 8
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros(len(before), max(max(held), max(need), 1), dtype=torch.int32, device=DEV)
    held_t = torch.tensor(held, device=DEV)
    mine = torch.arange(table.shape[1], device=DEV) < held_t[:, None]
    table[mine] = order[:sum(held)]
    # the pool: a ring of free pages, somewhere along which the next one stands
    free = pages - sum(held)
    first = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
    ring = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ring[(first + torch.arange(free, device=DEV)) % pages] = order[sum(held):]
    rows = sum(max(n, 0) for n in new)
    s.update(ring=ring, state=_ints([first, free]), state_out=_ints([0, 0]), before=_ints(before), stand=_ints(stand),
             new=_ints(new), table=table, kv_len=_ints([0] * len(before)), q_start=_ints([0] * (len(before) + 1)),
             positions=_ints([0] * rows), slots=torch.zeros(rows, dtype=torch.int64, device=DEV), rows=rows)


def _prepare_verify(s, g):
    case = s["case"]
    b, vocab = case["batch"], case["vocab"]
    rng = random.Random(31 * b + vocab + case["drafts"])
    n = [case["drafts"]] + [rng.randint((case["drafts"] + 1) // 2, case["drafts"]) for _ in range(b - 1)]
    rows = sum(n) + b
    kind = torch.bfloat16 if case["half"] else torch.float32
    q_start = torch.tensor([0] + [x + 1 for x in n], device=DEV).cumsum(0)
    target = torch.empty(rows, vocab, dtype=kind, device=DEV)
    draft = torch.empty(rows, vocab, dtype=kind, device=DEV)
    tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    for at in range(0, rows, 64):
        here = slice(at, min(at + 64, rows))
        count = here.stop - at
        p = torch.softmax(torch.randn(count, vocab, generator=g, device=DEV).mul_(3), dim=1)
        other = torch.softmax(torch.randn(count, vocab, generator=g, device=DEV).mul_(3), dim=1)
        q = p * (1 - case["off"]) + other * case["off"]
        target[here], draft[here] = p, q
        # row i of both is the distribution of token i + 1
        tokens[at + 1:here.stop + 1] = torch.multinomial(q, 1, generator=g)[:rows - at - 1, 0].int()
    s.update(target=target, draft=draft if case["given"] else None, tokens=tokens, q_start=q_start.int(),
             kv_len=torch.randint(9, 5000, (b,), generator=g, device=DEV).int(),
             accept_u=torch.rand(rows, generator=g, device=DEV), sample_u=torch.rand(b, generator=g, device=DEV))


def _prepare_cache(s, g):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    ns, lens = _lengths(case)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 8
    order = torch.randperm(pages, generator=g, device=DEV).int()       # pages as a free list hands them out
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    s["page_table"], s["kv_len"] = table, _ints(lens)
    s["q_start"] = torch.tensor([0] + ns, device=DEV).cumsum(0).int()
    shape = (pages, hkv, page, d) if case["heads_first"] else (pages, page, hkv, d)

    def cache():
        """Values whose size changes from page to page and head to head, and the scales that they call for."""
        size = torch.randn(pages, hkv, generator=g, device=DEV).mul_(0.5).exp_()
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        wide = (lambda t: t[:, :, None, None]) if case["heads_first"] else (lambda t: t[:, None, :, None])
        x.mul_(wide(size))
        scale = _scale_of(x.abs().amax(dim=(2, 3) if case["heads_first"] else (1, 3)).float())
        return x.div_(wide(scale)).to(torch.float8_e4m3fn), scale

    s["k_cache"], s["k_scale"] = cache()
    s["v_cache"], s["v_scale"] = cache()
    tokens = sum(ns)
    if case["op"] == "append":
        s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        # the packed output of a q/k/v projection and its three views
        qkv = torch.randn(tokens, (hq + 2 * hkv) * d, generator=g, device=DEV).mul_(1.5).bfloat16()
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
        s["rope"] = _rope_table(max(lens), case["rot"])
    else:
        s["q"] = torch.randn(tokens, hq, d, generator=g, device=DEV).mul_(1.5).bfloat16()


def _handles(s):
    """What a program that serves with the framework keeps: pool, cache and batch handles, workspaces, output buffers."""
    from nvfp4_block_scaled_route_gb300 import binding as nb
    case = s["case"]
    h = {"nb": nb}
    if case["op"] == "plan":
        h["pool"] = nb.PagePool(s["ring"], s["state"])
        h["batch"] = nb.AttnBatch(s["q_start"], s["kv_len"], s["table"], max_new=case["new"])
        h["ws"] = nb.attn_workspace()
        return h
    if case["op"] == "verify":
        b = case["batch"]
        h["batch"] = nb.AttnBatch(s["q_start"], s["kv_len"], torch.zeros(b, 1, dtype=torch.int32, device=DEV),
                                  max_new=case["drafts"] + 1)
        h["accepted"], h["next"], h["stand"] = _ints([0] * b), _ints([0] * b), _ints([0] * b)
        h["ws"] = nb.attn_workspace()
        return h
    h["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    h["cache"] = nb.PagedKVCache(s["k_cache"], s["v_cache"], heads_first=case["heads_first"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
    h["batch"] = nb.AttnBatch(s["q_start"], s["kv_len"], s["page_table"], max_new=case["new"])
    if case["op"] == "append":
        h["ws"] = nb.attn_workspace()
    else:
        h["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        h["ws"] = nb.paged_attention_workspace(h["cache"], h["batch"], s["q"].shape[1])
    return h


# -------------------------------------------------------------------- run --
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        h = s["own"]
        nb = h["nb"]
        if op == "plan":
            nb.plan_pages(h["pool"], h["batch"], case["page"], s["new"], cached=s["stand"], kv_before=s["before"],
                          state_out=s["state_out"], positions=s["positions"], slots=s["slots"], ws=h["ws"])
            return s["kv_len"], s["q_start"], s["table"], s["positions"], s["slots"], s["ring"], s["state_out"]
        if op == "verify":
            nb.draft_verify(s["target"], s["draft"], s["tokens"], h["batch"], s["accept_u"], s["sample_u"],
                            accepted=h["accepted"], next_token=h["next"], cached=h["stand"], ws=h["ws"])
            return h["accepted"], h["next"], h["stand"]
        if op == "append":
            q = nb.kv_append(h["cache"], h["batch"], s["k"], s["v"], rope=s["rope"], k_weight=s["k_weight"], q=s["q"],
                             q_weight=s["q_weight"], q_out=h["q_out"], eps=EPS, interleaved=case["pairs"], ws=h["ws"])
            return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        o = nb.paged_attention(s["q"], h["cache"], h["batch"], window=case["window"], out=h["q_out"], lse=h["lse"],
                               ws=h["ws"])
        return o, h["lse"]
    return {"plan": _plan, "verify": _verify, "append": _append, "attend": _attend}[op](s)


def _plan(s):
    page, ring, table = s["case"]["page"], s["ring"], s["table"]
    before, new = s["before"].long(), s["new"].long()
    ended = new < 0
    kv_len = torch.where(ended, 0, s["stand"].long() + new)
    held, need = (before + page - 1) // page, (kv_len + page - 1) // page
    take, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    first, free = s["state"].long()
    n = new.clamp(min=0)
    q_start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    # pages from the front of the ring, in the order of the requests
    i = torch.arange(table.shape[1], device=DEV)
    fresh = (i >= held[:, None]) & (i < need[:, None])
    which = (take.cumsum(0) - take)[:, None] + i - held[:, None]
    table.copy_(torch.where(fresh, ring[(first + which.clamp(min=0)) % ring.numel()], table))
    # those given back behind its end
    left = (i >= need[:, None]) & (i < held[:, None])
    which = (give.cumsum(0) - give)[:, None] + i - need[:, None]
    ring[(first + free + which[left]) % ring.numel()] = table[left]
    state = torch.stack([(first + take.sum()) % ring.numel(), free - take.sum() + give.sum()])
    # the rows
    t = torch.arange(s["rows"], device=DEV)
    r = torch.searchsorted(q_start, t, right=True) - 1
    pos = kv_len[r] - q_start[r + 1] + t
    slots = table[r, pos // page].long() * page + pos % page
    return kv_len.int(), q_start.int(), table, pos.int(), slots, ring, state.int()


def _verify(s):
    target, draft, tokens = s["target"], s["draft"], s["tokens"].long()
    start = s["q_start"].long()
    n = start[1:] - start[:-1] - 1                                                       # drafted tokens
    i = torch.arange(s["case"]["drafts"], device=DEV)
    real = i < n[:, None]
    row = torch.where(real, start[:-1, None] + i, 0)                                     # [B, drafts]
    token = tokens[row + 1]
    p = target[row, token].double()
    q = torch.ones_like(p) if draft is None else draft[row, token].double()
    stands = real & (s["accept_u"][row].double() * q < p)
    accepted = stands.long().cumprod(dim=1).sum(dim=1)
    # the next token: from the target's row behind the last drafted one, else from what it has over the draft's
    at = start[:-1] + accepted
    weight = target[at].double()
    cut = accepted < n
    if draft is None:
        guessed = tokens[torch.where(cut, at + 1, 0)]
        here = torch.arange(weight.shape[1], device=DEV) == guessed[:, None]
        weight = torch.where(here & cut[:, None], 0, weight)
    else:
        weight = torch.where(cut[:, None], (weight - draft[at].double()).clamp(min=0), weight)
    total = weight.cumsum(dim=1)
    # the first token whose running sum passes u times the whole
    nxt = (total > s["sample_u"].double()[:, None] * total[:, -1:]).int().argmax(dim=1)
    return accepted.int(), nxt.int(), (s["kv_len"].long() - (n - accepted)).int()


def _rotate(x, weight, positions, rope, pairs):
    """Norm and rotation of [T, H, D], in x's type."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * weight.to(x.dtype)
    half = rope.shape[1] // 2
    row = rope[positions].to(x.dtype)
    cos, sin = row[:, None, :half], row[:, None, half:]
    if pairs:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    return torch.cat([turned, x[..., 2 * half:]], dim=2)


def _append(s):
    case, page = s["case"], s["case"]["page"]
    start, length = s["q_start"].long(), s["kv_len"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(start, t, right=True) - 1
    pos = length[r] - start[r + 1] + t
    q = _rotate(s["q"].float(), s["q_weight"], pos, s["rope"], case["pairs"]).bfloat16()
    # (64 bits for the keys: they stand next to borders of E4M3 numbers)
    k = _rotate(s["k"].double(), s["k_weight"], pos, s["rope"], case["pairs"]).float()
    # the pages that get new tokens, and where their offsets come from
    first = length - (start[1:] - start[:-1])
    index = first[:, None] // page + torch.arange((case["new"] + page - 2) // page + 1, device=DEV)
    real = index * page < length[:, None]
    request = torch.arange(len(length), device=DEV)[:, None].expand_as(index)[real]
    index = index[real]
    pages = s["page_table"][request, index].long()
    at = index[:, None] * page + torch.arange(page, device=DEV)                          # positions [U, page]
    is_new = (at >= first[request, None]) & (at < length[request, None])
    is_old = at < first[request, None]
    row = torch.where(is_new, at - first[request, None] + start[request, None], 0)
    grown = index * page < first[request]                                                # holds tokens already

    def fill(cache, scale, x):
        raw = cache.view(torch.uint8)[pages]
        if case["heads_first"]:
            raw = raw.transpose(1, 2)                                                    # [U, page, H, D]
        fresh = x[row]
        size = torch.where(is_new[..., None, None] & fresh.isfinite(), fresh.abs(), 0).amax(dim=(1, 3))
        want, had = _scale_of(size), scale[pages]
        want = torch.where(grown[:, None], torch.maximum(want, had), want)
        old = raw.view(torch.float8_e4m3fn).float() * (had / want)[:, None, :, None]
        fresh = (fresh / want[:, None, :, None]).clamp(-TOP, TOP)
        fresh, old = (y.to(torch.float8_e4m3fn).view(torch.uint8) for y in (fresh, old))
        out = torch.where(is_new[..., None, None], fresh, torch.where(is_old[..., None, None], old, raw))
        cache.view(torch.uint8)[pages] = out.transpose(1, 2) if case["heads_first"] else out
        scale[pages] = want

    fill(s["k_cache"], s["k_scale"], k)
    fill(s["v_cache"], s["v_scale"], s["v"].float())
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _gather(s, cache, scale):
    """A cache's pages as [B, Hkv, L, D] in 32 bits."""
    p = s["page_table"].long()
    x = cache.view(torch.uint8)[p].view(torch.float8_e4m3fn).float()
    if not s["case"]["heads_first"]:
        x = x.transpose(2, 3)
    x = x * scale[p][..., None, None]                                                    # [B, pages, Hkv, page, D]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s):
    case = s["case"]
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["new"]
    start, length = s["q_start"].long(), s["kv_len"].long()
    k, v = _gather(s, s["k_cache"], s["k_scale"]), _gather(s, s["v_cache"], s["v_scale"])
    i = torch.arange(n, device=DEV)
    real = i < (start[1:] - start[:-1])[:, None]                                         # [B, n]
    row = torch.where(real, start[:-1, None] + i, 0)
    q = s["q"][row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)        # [B, Hkv, g, n, D]
    scores = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).mul_(d ** -0.5)            # [B, Hkv, g*n, L]
    scores = scores.unflatten(2, (hq // hkv, n))
    j = torch.arange(k.shape[2], device=DEV)
    pos = (length - start[1:])[:, None] + row                                            # [B, n]
    see = j <= pos[..., None]
    if case["window"]:
        see &= j > pos[..., None] - case["window"]
    scores.masked_fill_(~see[:, None, None], -math.inf)
    top = scores.amax(dim=4, keepdim=True)
    p = scores.sub_(torch.where(top.isfinite(), top, 0)).exp_()
    total = p.sum(dim=4, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.mul_((j < length[:, None])[:, None, :, None])).unflatten(2, (hq // hkv, n))
    o = torch.where(total > 0, o / total, 0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                                           # [B, n, Hq, D]
    lse = (top + total.log()).squeeze(4).permute(0, 3, 1, 2).flatten(2, 3)
    return o[real].bfloat16(), lse[real]


# ------------------------------------------------------------------- work --
def work(case):
    if case["op"] == "plan":
        before, stand, new = _steps(case)
        page = case["page"]
        held = [-(-n // page) for n in before]
        need = [0 if n < 0 else -(-(c + n) // page) for c, n in zip(stand, new)]
        moved = sum(abs(a - b) for a, b in zip(held, need))
        rows = sum(max(n, 0) for n in new)
        used = sum((c + n - 1) // page - c // page + 1 for c, n in zip(stand, new) if n > 0)      # pages of the rows
        return {"bytes": 20 * case["batch"] + 8 * moved + 12 * rows + 4 * used, "flops": 4 * rows}
    if case["op"] == "verify":
        # the target's row behind the last accepted token; where one was turned down, the draft's too
        down = 1 - (1 - case["off"]) ** (0.75 * case["drafts"])
        el = 2 if case["half"] else 4
        rows = 1 + (down if case["given"] else 0)
        b = case["batch"]
        return {"bytes": int(b * (rows * case["vocab"] * el + case["drafts"] * 16)), "flops": 2 * b * case["vocab"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ns, lens = _lengths(case)
    t, page = sum(ns), case["page"]
    if case["op"] == "append":
        touched = sum((length - 1) // page - (length - n) // page + 1 for n, length in zip(ns, lens))
        return {"bytes": t * (hq * d * 4 + 2 * hkv * d * 3 + case["rot"] * 4) + touched * hkv * 16,
                "flops": t * (hq + 2 * hkv) * d * 8}
    w = case["window"]
    keys = seen = 0
    for n, length in zip(ns, lens):
        first = length - n
        keys += length - max(0, first - w + 1) if w else length
        full = first + 1 + length                       # twice the mean number of keys that a row sees without a window
        if not w:
            seen += n * full / 2
        else:
            short = max(0, min(n, w - first))           # rows that see fewer than w keys
            seen += short * (2 * first + short + 1) / 2 + (n - short) * w
    return {"bytes": int(t * hq * (4 * d + 4) + 2 * keys * hkv * (d + 4 / page)), "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "verify": _exact_verify, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_plan(s):
    """Request by request, with lists on the host."""
    page = s["case"]["page"]
    before, stand, new = (s[x].tolist() for x in ("before", "stand", "new"))
    ring, table = s["ring"].tolist(), s["table"].tolist()
    first, free = s["state"].tolist()
    end = first + free
    kv_len, q_start, positions, slots, back = [], [0], [], [], []
    for r, n in enumerate(new):
        have = -(-before[r] // page)
        kv_len.append(0 if n < 0 else stand[r] + n)
        need = -(-kv_len[r] // page)
        for j in range(have, need):
            table[r][j] = ring[first % len(ring)]
            first += 1
        back += table[r][need:have]
        q_start.append(q_start[-1] + max(n, 0))
        for p in range(kv_len[r] - max(n, 0), kv_len[r]):
            positions.append(p)
            slots.append(table[r][p // page] * page + p % page)
    for j, p in enumerate(back):
        ring[(end + j) % len(ring)] = p
    return tuple(torch.tensor(x, device=DEV) for x in (kv_len, q_start, table, positions, slots, ring,
                                                       [first % len(ring), end + len(back) - first]))


def _exact_verify(s):
    """Token by token, as the method is stated."""
    start, tokens = s["q_start"].tolist(), s["tokens"].tolist()
    u, last = s["accept_u"].tolist(), s["sample_u"].tolist()
    kv_len = s["kv_len"].tolist()
    accepted, following, stand = [], [], []
    for r in range(len(kv_len)):
        a, n = start[r], start[r + 1] - start[r] - 1
        k = 0
        while k < n:
            y = tokens[a + k + 1]
            q = 1.0 if s["draft"] is None else float(s["draft"][a + k, y])
            if u[a + k] * q >= float(s["target"][a + k, y]):
                break
            k += 1
        w = s["target"][a + k].double()
        if k < n:
            if s["draft"] is None:
                w[tokens[a + k + 1]] = 0
            else:
                w = torch.relu(w - s["draft"][a + k].double())
        run_sum = torch.cumsum(w, 0)
        accepted.append(k)
        following.append(int(torch.searchsorted(run_sum, last[r] * run_sum[-1], right=True)))
        stand.append(kv_len[r] - n + k)
    return _ints(accepted), _ints(following), _ints(stand)


def _exact_append(s):
    case, page = s["case"], s["case"]["page"]
    ns, lens = _lengths(case)

    def turn(x, weight, pos):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
        half = case["rot"] // 2
        c, sn = s["rope"][pos].double()[:, None].split(half, dim=-1)
        out = x.clone()
        one = slice(0, 2 * half, 2) if case["pairs"] else slice(0, half)
        two = slice(1, 2 * half, 2) if case["pairs"] else slice(half, 2 * half)
        out[..., one] = x[..., one] * c - x[..., two] * sn
        out[..., two] = x[..., two] * c + x[..., one] * sn
        return out

    pos = torch.cat([torch.arange(length - n, length, device=DEV) for n, length in zip(ns, lens)])
    k, v = turn(s["k"], s["k_weight"], pos), s["v"].double()
    found = [turn(s["q"], s["q_weight"], pos)]
    powers = torch.exp2(torch.arange(LOW, HIGH + 1, dtype=torch.float64, device=DEV))
    scales = []
    for cache, scale, x in ((s["k_cache"], s["k_scale"], k), (s["v_cache"], s["v_scale"], v)):
        out, scale = cache.double(), scale.double()
        rows = out.transpose(1, 2) if case["heads_first"] else out                       # [pages, page, H, D]
        at = 0
        for r, (n, length) in enumerate(zip(ns, lens)):
            p = length - n
            while p < length:
                take = min(length - p, page - p % page)
                id_, off = int(s["page_table"][r, p // page]), p % page
                here = x[at:at + take]
                # the first power of two whose 448-fold reaches the largest value
                want = powers[torch.searchsorted(powers * TOP, here.abs().amax(dim=(0, 2))).clamp(max=HIGH - LOW)]
                if off:
                    want = torch.maximum(want, scale[id_])
                    rows[id_, :off] *= (scale[id_] / want)[:, None]
                rows[id_, off:off + take] = here / want[:, None]
                scale[id_] = want
                p, at = p + take, at + take
        found.append(out)
        scales.append(scale)
    return (*found, *scales)


def _exact_attend(s):
    case = s["case"]
    if work(case)["flops"] > 3e12:
        return None
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    ns, lens = _lengths(case)
    o = torch.zeros(sum(ns), hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((sum(ns), hq), -math.inf, dtype=torch.float64, device=DEV)
    begin = 0
    for r, (n, length) in enumerate(zip(ns, lens)):
        pages = s["page_table"][r, :-(-length // page)].long()
        here = slice(begin, begin + n)
        begin += n
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        j = torch.arange(length, device=DEV)
        hide = (j > pos) | ((j <= pos - case["window"]) if case["window"] else False)
        for kv in range(hkv):
            def rows(cache, scale):
                x = cache.view(torch.uint8)[pages]
                x = (x[:, kv] if case["heads_first"] else x[:, :, kv]).contiguous().view(torch.float8_e4m3fn).double()
                return (x * scale[pages, kv].double()[:, None, None]).flatten(0, 1)[:length]
            k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
            for h in range(kv * (hq // hkv), (kv + 1) * (hq // hkv)):
                a = (s["q"][here, h].double() @ k.T / math.sqrt(d)).masked_fill_(hide, -math.inf)
                lse[here, h] = torch.logsumexp(a, dim=1)
                o[here, h] = torch.softmax(a, dim=1) @ v
    return o, lse
