"""Attention operators of the decoder layer around the expert FFN: cases, inputs, plain forms and exact values.

Three operators, which a serving step calls one after the other:

  rotate   per-head RMS norm of queries and keys with the rotary embedding, dense outputs
  append   the same transform with keys and values going into a paged cache (bf16 or E4M3 with a scale per head),
           the queries transformed in the same call
  attend   attention of each request's new tokens over its paged cache, causal, optionally within a window

With `own` false, run() computes them in elementary torch operations in 32 bits; with `own` true it makes the calls of
nvfp4_block_scaled_route_gb300.binding.  The head layout of most cases is that of the repository's hidden size,
7168 = 56 heads of 128, with 8 heads of keys; the token counts 1, 64, 4096 and 16384 are its workloads'.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases --
def listed():
    wide = {"hq": 56, "hkv": 8, "d": 128}
    return [
        # one decode step of one request: the smallest call, all latency
        {"name": "rotate-1", "op": "rotate", "tokens": 1, "rot": 128, "norm": True, "pairs": False, **wide},
        # a prompt of the 4096-token prefill workload, read from a packed projection output
        {"name": "rotate-4096", "op": "rotate", "tokens": 4096, "rot": 128, "norm": True, "pairs": False, **wide},
        # 64-wide heads, half of each head rotated in neighbouring pairs, no norm, an odd token count
        {"name": "rotate-pairs-1031", "op": "rotate", "tokens": 1031, "rot": 32, "norm": False, "pairs": True, "hq": 20,
         "hkv": 4, "d": 64},
        # one token for each of 64 requests of uneven length: a decode step of a full batch
        {"name": "append-64x1", "op": "append", "batch": 64, "new": 1, "ctx": 4096, "ragged": True, "page": 16,
         "heads_first": True, "fp8": False, "rot": 128, "norm": True, "pairs": False, **wide},
        # three uneven prompts of up to 8192 tokens, into an 8-bit cache
        {"name": "append-3x8192-fp8", "op": "append", "batch": 3, "new": 8192, "ctx": 8192, "ragged": True, "page": 64,
         "heads_first": False, "fp8": True, "rot": 128, "norm": True, "pairs": False, **wide},
        # one token of one request with a short history: latency
        {"name": "decode-1x1000", "op": "attend", "batch": 1, "new": 1, "ctx": 1000, "ragged": False, "page": 16,
         "heads_first": False, "fp8": False, "window": 0, **wide},
        # the full decode batch, uneven histories of up to 16384 tokens
        {"name": "decode-64x16384", "op": "attend", "batch": 64, "new": 1, "ctx": 16384, "ragged": True, "page": 16,
         "heads_first": False, "fp8": False, "window": 0, **wide},
        # two long conversations on an 8-bit cache: few rows, a long axis
        {"name": "decode-2x131072-fp8", "op": "attend", "batch": 2, "new": 1, "ctx": 131072, "ragged": True, "page": 64,
         "heads_first": True, "fp8": True, "window": 0, **wide},
        # up to five drafted tokens checked for each of 16 requests
        {"name": "verify-16x5", "op": "attend", "batch": 16, "new": 5, "ctx": 6000, "ragged": True, "page": 32,
         "heads_first": True, "fp8": False, "window": 0, **wide},
        # the last chunk of a long prompt: 2048 tokens over the 14336 that the cache holds already
        {"name": "chunk-2048-of-16384", "op": "attend", "batch": 1, "new": 2048, "ctx": 16384, "ragged": False,
         "page": 64, "heads_first": False, "fp8": False, "window": 0, **wide},
        # uneven prompts with 64-wide heads, as many heads of keys as of queries, attention within a window
        {"name": "prompts-6x1500-window", "op": "attend", "batch": 6, "new": 1500, "ctx": 2500, "ragged": True,
         "page": 16, "heads_first": True, "fp8": False, "window": 700, "hq": 24, "hkv": 24, "d": 64},
        # a chunk on an 8-bit cache, several requests at once
        {"name": "chunk-4x512-fp8", "op": "attend", "batch": 4, "new": 512, "ctx": 9000, "ragged": True, "page": 128,
         "heads_first": False, "fp8": True, "window": 0, **wide},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 3, 4, 8, 8])
        c = {"op": rng.choice(["rotate", "append", "attend", "attend", "attend"]), "d": d, "hkv": hkv,
             "hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])}
        if c["hq"] > 64:
            continue
        if c["op"] != "attend":
            c.update(rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.7, pairs=rng.random() < 0.3)
        if c["op"] == "rotate":
            c.update(tokens=_spread(rng, 1, 16384))
        else:
            batch = _spread(rng, 1, 64)
            new = _spread(rng, 1, max(1, 16384 // batch)) if rng.random() < 0.6 else rng.randint(1, 6)
            c.update(batch=batch, new=new, ctx=new + _spread(rng, 1, 65536) - 1, ragged=rng.random() < 0.7,
                     page=rng.choice([16, 32, 64, 128]), heads_first=rng.random() < 0.5, fp8=rng.random() < 0.4)
            if c["batch"] * c["ctx"] > 1 << 20:
                continue
        if c["op"] == "attend":
            c.update(window=0 if rng.random() < 0.7 else _spread(rng, 16, 8192))
            # what the plain form holds of scores at once
            if c["batch"] * c["new"] * c["ctx"] * c["hq"] > 2 << 30:
                continue
        if _cost(c) <= top:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(case):
    """New tokens and cache length (new ones counted) of each request: they go by the case alone."""
    b, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * b, [ctx] * b
    rng = random.Random(1000003 * b + 10007 * new + ctx)
    ns = [new] + [rng.randint((new + 1) // 2, new) for _ in range(b - 1)]
    lens = [ctx] + [n + _spread(rng, max(1, (ctx - new + 1) // 16), max(1, ctx - new + 1)) - 1 for n in ns[1:]]
    return ns, lens


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rope_table(positions, rot):
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _projection(g, tokens, hq, hkv, d):
    """The packed output of a q/k/v projection and its three views."""
    qkv = torch.randn(tokens, (hq + 2 * hkv) * d, generator=g, device=DEV).mul_(1.5).bfloat16()
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
    return q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))


def prepare(case, seed):
    g = _gen(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case}
    if case["op"] != "attend":
        s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
    if case["op"] == "rotate":
        t = case["tokens"]
        s["q"], s["k"], _ = _projection(g, t, hq, hkv, d)
        first = int(torch.randint(0, 1000, (1,), generator=g, device=DEV))
        s["positions"] = torch.arange(first, first + t, dtype=torch.int32, device=DEV)
        s["rope"] = _rope_table(t + 1000, case["rot"])
        if own:
            s["own"] = _handles(s)
        return s

    ns, lens = _lengths(case)
    page = case["page"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 8
    order = torch.randperm(pages, generator=g, device=DEV).int()       # pages as a free list hands them out
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    s["page_table"] = table
    s["q_start"] = torch.tensor([0] + ns, device=DEV).cumsum(0).int()
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape = (pages, hkv, page, d) if case["heads_first"] else (pages, page, hkv, d)
    scales = torch.rand(2, hkv, generator=g, device=DEV) * 0.01 + 0.01
    s["k_scale"], s["v_scale"] = (scales[0], scales[1]) if case["fp8"] else (None, None)

    def cache(scale):
        if not case["fp8"]:
            return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        x.div_(scale[:, None, None] if case["heads_first"] else scale[:, None])
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn)

    s["k_cache"], s["v_cache"] = cache(scales[0]), cache(scales[1])
    tokens = sum(ns)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _projection(g, tokens, hq, hkv, d)
        s["rope"] = _rope_table(max(lens), case["rot"])
    else:
        s["q"] = torch.randn(tokens, hq, d, generator=g, device=DEV).mul_(1.5).bfloat16()
    if own:
        s["own"] = _handles(s)
    return s


def _handles(s):
    """What a program that serves with the framework keeps: the cache's and the batch's handles, workspace, output buffers."""
    from nvfp4_block_scaled_route_gb300 import binding as nb
    h = {"nb": nb, "q_out": torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)}
    if s["case"]["op"] == "rotate":
        h["k_out"] = torch.empty(s["k"].shape, dtype=torch.bfloat16, device=DEV)
        h["ws"] = nb.attn_workspace()
        return h
    h["cache"] = nb.PagedKVCache(s["k_cache"], s["v_cache"], heads_first=s["case"]["heads_first"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
    h["batch"] = nb.AttnBatch(s["q_start"], s["kv_len"], s["page_table"], max_new=s["case"]["new"])
    if s["case"]["op"] == "append":
        h["ws"] = nb.attn_workspace()
    else:
        h["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        h["ws"] = nb.paged_attention_workspace(h["cache"], h["batch"], s["q"].shape[1])
    return h


# -------------------------------------------------------------------- run --
def run(s):
    case = s["case"]
    if own:
        h = s["own"]
        nb = h["nb"]
        if case["op"] == "rotate":
            return nb.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=EPS, interleaved=case["pairs"], q_out=h["q_out"],
                                   k_out=h["k_out"], ws=h["ws"])
        if case["op"] == "append":
            q = nb.kv_append(h["cache"], h["batch"], s["k"], s["v"], rope=s["rope"], k_weight=s["k_weight"], q=s["q"],
                             q_weight=s["q_weight"], q_out=h["q_out"], eps=EPS, interleaved=case["pairs"], ws=h["ws"])
            return q, s["k_cache"], s["v_cache"]
        o = nb.paged_attention(s["q"], h["cache"], h["batch"], window=case["window"], out=h["q_out"], lse=h["lse"],
                               ws=h["ws"])
        return o, h["lse"]
    if case["op"] == "rotate":
        return (_rotate(s["q"], s["q_weight"], s["positions"], s["rope"], case["pairs"]).bfloat16(),
                _rotate(s["k"], s["k_weight"], s["positions"], s["rope"], case["pairs"]).bfloat16())
    if case["op"] == "append":
        return _append(s)
    return _attend(s)


def _rotate(x, weight, positions, rope, pairs):
    """Norm and rotation of [T, H, D] in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * weight.float()
    half = rope.shape[1] // 2
    row = rope[positions.long()]
    cos, sin = row[:, None, :half], row[:, None, half:]
    if pairs:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    return torch.cat([turned, x[..., 2 * half:]], dim=2)


def _where(s):
    """Request and cache position of every new token."""
    t = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    return r, s["kv_len"].long()[r] - s["q_start"].long()[r + 1] + t


def _append(s):
    case = s["case"]
    r, pos = _where(s)
    page = s["page_table"].long()[r, pos // case["page"]]
    off = pos % case["page"]
    q = _rotate(s["q"], s["q_weight"], pos, s["rope"], case["pairs"]).bfloat16()
    k = _rotate(s["k"], s["k_weight"], pos, s["rope"], case["pairs"])
    v = s["v"].float()
    if case["fp8"]:
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
    kc, vc = s["k_cache"], s["v_cache"]
    k, v = k.to(kc.dtype), v.to(vc.dtype)
    if case["fp8"]:                                        # moved as bytes
        k, v, kc, vc = (x.view(torch.uint8) for x in (k, v, kc, vc))
    if case["heads_first"]:
        kc[page, :, off] = k
        vc[page, :, off] = v
    else:
        kc[page, off] = k
        vc[page, off] = v
    return q, s["k_cache"], s["v_cache"]


def _gather(s, cache, scale):
    """A cache's pages as [B, Hkv, L, D] in 32 bits."""
    p = s["page_table"].long()
    x = cache.view(torch.uint8)[p].view(torch.float8_e4m3fn) if s["case"]["fp8"] else cache[p]
    x = x.permute(0, 2, 1, 3, 4) if s["case"]["heads_first"] else x.permute(0, 3, 1, 2, 4)
    x = x.flatten(2, 3).float()
    return x if scale is None else x * scale[:, None, None]


def _attend(s):
    case = s["case"]
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["new"]
    b = s["kv_len"].shape[0]
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
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotate":
        t = case["tokens"]
        return {"bytes": t * ((hq + hkv) * d * 4 + case["rot"] * 4 + 4), "flops": t * (hq + hkv) * d * 8}
    ns, lens = _lengths(case)
    t = sum(ns)
    el = 1 if case["fp8"] else 2
    if case["op"] == "append":
        return {"bytes": t * (hq * d * 4 + 2 * hkv * d * (2 + el) + case["rot"] * 4), "flops": t * (hq + 2 * hkv) * d * 8}
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
    return {"bytes": t * hq * (4 * d + 4) + 2 * keys * hkv * d * el, "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def turn(x, weight, pos):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
        half = case["rot"] // 2
        c, sn = s["rope"][pos.long()].double()[:, None].split(half, dim=-1)
        out = x.clone()
        first = slice(0, 2 * half, 2) if case["pairs"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["pairs"] else slice(half, 2 * half)
        out[..., first] = x[..., first] * c - x[..., second] * sn
        out[..., second] = x[..., second] * c + x[..., first] * sn
        return out

    if case["op"] == "rotate":
        return turn(s["q"], s["q_weight"], s["positions"]), turn(s["k"], s["k_weight"], s["positions"])

    ns, lens = _lengths(case)
    page = case["page"]
    begin = [sum(ns[:r]) for r in range(len(ns))]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(length - n, length, device=DEV) for n, length in zip(ns, lens)])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k, v = turn(s["k"], s["k_weight"], pos), s["v"].double()
        if case["fp8"]:
            k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
            v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
        for r, n in enumerate(ns):
            here = slice(begin[r], begin[r] + n)
            where = s["page_table"][r].long()[pos[here] // page], pos[here] % page
            for cache, new in ((kc, k), (vc, v)):
                (cache.transpose(1, 2) if case["heads_first"] else cache)[where] = new[here]
        return turn(s["q"], s["q_weight"], pos), kc, vc

    if work(case)["flops"] > 3e12:
        return None
    o = torch.zeros(sum(ns), hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((sum(ns), hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, (n, length) in enumerate(zip(ns, lens)):
        pages = s["page_table"][r, :-(-length // page)].long()
        here = slice(begin[r], begin[r] + n)
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        j = torch.arange(length, device=DEV)
        hide = (j > pos) | ((j <= pos - case["window"]) if case["window"] else False)
        for kv in range(hkv):
            def rows(cache, scale):
                x = cache.view(torch.uint8)[pages] if case["fp8"] else cache[pages]
                x = (x[:, kv] if case["heads_first"] else x[:, :, kv]).flatten(0, 1)[:length]
                return x.view(torch.float8_e4m3fn).double() * scale[kv].double() if case["fp8"] else x.double()
            k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
            for h in range(kv * (hq // hkv), (kv + 1) * (hq // hkv)):
                a = (s["q"][here, h].double() @ k.T / math.sqrt(d)).masked_fill_(hide, -math.inf)
                lse[here, h] = torch.logsumexp(a, dim=1)
                o[here, h] = torch.softmax(a, dim=1) @ v
    return o, lse
