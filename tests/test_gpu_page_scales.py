"""E4M3 caches with a scale for each page and head: appending to them, attention over
them (64-bit forms and bounds in tests/_serving_reference.py)."""
import math

import pytest
import torch

import _attention_reference as ref
import _serving_reference as sref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD_INDEX = 7
NAN = 0x7F


@pytest.fixture(scope="module")
def nb():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_block_scaled_route_gb300 import binding
    return binding


def rope_table(positions, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def values(raw):
    return raw.view(torch.float8_e4m3fn).double()


class Pages:
    """Requests of (new tokens, cached length) on scattered pages.  Whatever does not
    count is NaN: offsets past a request's length, free pages, their scales; table entries
    past a request's pages point nowhere.  spread: exponents of the scales."""

    def __init__(self, reqs, hk, D, page, heads_first=False, spread=(-3, 3), powers=True, seed=0, extra=3):
        g = torch.Generator().manual_seed(seed + 17 * hk + D + page)
        self.reqs, self.hk, self.D, self.page, self.heads_first = reqs, hk, D, page, heads_first
        need = [-(-max(length, 0) // page) for _, length in reqs]
        n = sum(need) + extra
        order = torch.randperm(n, generator=g)
        self.table = torch.full((len(reqs), max(need + [1]) + 2), 1 << 30, dtype=torch.int32)
        self.raw, self.scale = [], []
        for _ in range(2):
            raw = torch.full((n, page, hk, D), NAN, dtype=torch.uint8)
            self.raw.append(raw)
            self.scale.append(torch.full((n, hk), math.nan))
        at = 0
        for r, (_, length) in enumerate(reqs):
            for i in range(need[r]):
                p = int(order[at])
                at += 1
                self.table[r, i] = p
                m = min(page, length - i * page)
                for raw, scale in zip(self.raw, self.scale):
                    raw[p, :m] = torch.randint(0, 0x7F, (m, hk, D), generator=g, dtype=torch.uint8) \
                        | (torch.randint(0, 2, (m, hk, D), generator=g, dtype=torch.uint8) << 7)
                    # most values of an E4M3 number are tiny: as many of each size as a
                    # page of normal numbers has
                    x = torch.randn(m, hk, D, generator=g) * 100
                    raw[p, :m] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    e = torch.randint(spread[0], spread[1] + 1, (hk,), generator=g) - 8
                    s = torch.exp2(e.double())
                    if not powers:
                        s = s * (1 + torch.rand(hk, generator=g).double())
                    scale[p] = s.float()
        self.q_start = torch.tensor([0] + [n for n, _ in reqs]).cumsum(0).int()
        self.kv_len = torch.tensor([length for _, length in reqs], dtype=torch.int32)
        self.tokens = int(self.q_start[-1])
        self.g = g

    def layout(self, raw):
        return raw.transpose(1, 2).contiguous() if self.heads_first else raw

    def handles(self, nb, max_new=None):
        dev = [self.layout(r).to(DEV).view(torch.float8_e4m3fn) for r in self.raw]
        scales = [s.to(DEV) for s in self.scale]
        cache = nb.PagedKVCache(*dev, heads_first=self.heads_first, k_scale=scales[0], v_scale=scales[1])
        batch = nb.AttnBatch(self.q_start.to(DEV), self.kv_len.to(DEV), self.table.to(DEV),
                             max_new=max_new or max([n for n, _ in self.reqs] + [1]))
        return cache, batch

    def rows(self, which, r, h):
        """(values with their scale, scales) of request r and head h, [length, D], [length]."""
        length = max(self.reqs[r][1], 0)
        pages = self.table[r, :-(-length // self.page)].long()
        s = self.scale[which][pages, h].double().repeat_interleave(self.page)[:length]
        x = values(self.raw[which][pages, :, h].contiguous()).flatten(0, 1)[:length]
        return x * s[:, None], s

    def attention(self, q, scale=None, window=0):
        T, hq, D = q.shape
        scale = D ** -0.5 if scale is None else scale
        group = hq // self.hk
        out = [torch.full((T, hq) + tail, math.nan, dtype=torch.float64) for tail in ((D,), (), (D,), ())]
        for r, (n, length) in enumerate(self.reqs):
            if n == 0:
                continue
            here = slice(int(self.q_start[r]), int(self.q_start[r + 1]))
            for h in range(self.hk):
                heads = slice(h * group, (h + 1) * group)
                k, _ = self.rows(0, r, h)
                v, vs = self.rows(1, r, h)
                got = sref.request_attention(q[here, heads].double(), k, v, vs, length - n, scale, window)
                for o, x in zip(out, got):
                    o[here, heads] = x
        return out


def within(got, want, bound, what):
    got = got.double().cpu()
    err = torch.where(got.isinf() & (got == want), 0.0, (got - want).abs())
    assert not err.isnan().any(), what
    over = err - bound
    assert (over <= 0).all(), f"{what}: {err.max():.3g}, over its bound by {over.max():.3g}"


def check_attention(nb, pages, hq, scale=None, window=0, ws=None, stream=None, q=None):
    if q is None:
        q = (torch.randn(pages.tokens, hq, pages.D, generator=pages.g) * 1.5).bfloat16()
    cache, batch = pages.handles(nb)
    lse = torch.full((pages.tokens, hq), 7.0, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, hq, pages.tokens) if ws is None else ws
    out = nb.paged_attention(q.to(DEV), cache, batch, scale=scale, window=window, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want = pages.attention(q, scale, window)
    within(out, want[0], want[2], "out")
    within(lse, want[1], want[3], "lse")
    return out, lse


# -------------------------------------------------------------- attention --
@pytest.mark.parametrize("powers", [True, False], ids=["powers", "any"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("reqs,hk,hq,page,heads_first,window", [
    ([(1, 1)], 1, 1, 16, False, 0),
    ([(1, 17)], 2, 14, 16, True, 0),
    ([(1, 1000), (1, 15), (1, 128), (1, 129), (0, 40), (1, 500)], 2, 6, 16, False, 0),
    ([(5, 300), (3, 3), (2, 64), (1, 65)], 3, 9, 32, True, 0),
    ([(1, 2049), (1, 1024)], 1, 16, 1024, False, 0),
    ([(4, 700), (1, 260)], 2, 8, 256, True, 100),
    ([(2, 1), (3, 0), (1, 40)], 1, 2, 16, False, 0),             # tokens of negative position
    ([(3, 4000)], 1, 4, 64, False, 0),
])
def test_few_rows(nb, reqs, hk, hq, page, heads_first, window, D, powers):
    pages = Pages(reqs, hk, D, page, heads_first, powers=powers)
    assert max(n for n, _ in reqs) * hq // hk <= 16
    check_attention(nb, pages, hq, window=window)


@pytest.mark.parametrize("powers", [True, False], ids=["powers", "any"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("reqs,hk,hq,page,heads_first,window", [
    ([(17, 17)], 1, 1, 16, False, 0),
    ([(5, 300), (3, 3), (0, 9), (20, 450)], 2, 14, 16, True, 0),
    ([(130, 700), (1, 900), (64, 64)], 2, 4, 32, False, 0),
    ([(200, 1500)], 1, 3, 64, True, 130),
    ([(150, 2100), (33, 1024)], 1, 2, 1024, False, 0),
    ([(257, 257), (255, 400)], 2, 2, 128, True, 0),
    ([(40, 7), (30, 0), (20, 300)], 1, 2, 16, False, 0),         # tokens of negative position
    ([(300, 300)], 8, 8, 256, False, 17),
])
def test_chunks(nb, reqs, hk, hq, page, heads_first, window, D, powers):
    pages = Pages(reqs, hk, D, page, heads_first, powers=powers)
    check_attention(nb, pages, hq, window=window)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("page", [16, 128])
def test_scales_that_lie_far_apart(nb, n, page):
    """Scales over the whole range side by side, queries small so that all pages count."""
    pages = Pages([(n, 700), (n, 90)], 2, 128, page, spread=(-30, 30))
    # (keys as large as usual: only the values' scales spread)
    pages.scale[0] = torch.where(pages.scale[0].isnan(), math.nan, 2.0 ** -8).float()
    check_attention(nb, pages, 4)
    # values of nothing but zeros in pages of the lowest scale take their weight all the same
    pages = Pages([(n, 640)], 1, 128, page)
    for i in range(0, 640 // page, 2):
        p = int(pages.table[0, i])
        pages.raw[1][p], pages.scale[1][p] = 0, 2.0 ** -40
    check_attention(nb, pages, 2)


@pytest.mark.parametrize("n", [2, 40])
def test_scales_past_their_bounds(nb, n):
    """Taken as the nearer bound, NaN and what is not positive as the lower."""
    pages = Pages([(n, 96)], 1, 128, 16)
    odd = [0.0, -3.0, math.nan, 2.0 ** -60, 2.0 ** 70, math.inf]
    want = [2.0 ** -40] * 4 + [2.0 ** 40] * 2
    q = (torch.randn(n, 1, 128, generator=pages.g)).bfloat16()
    for which in range(2):
        for i, s in enumerate(odd):
            pages.scale[which][int(pages.table[0, i])] = s
    cache, batch = pages.handles(nb)
    out = nb.paged_attention(q.to(DEV), cache, batch, scale=2.0 ** -44)
    for which in range(2):
        for i, s in enumerate(want):
            pages.scale[which][int(pages.table[0, i])] = s
    o, _, bound, _ = pages.attention(q, 2.0 ** -44)
    within(out, o, bound, "out")


@pytest.mark.parametrize("n", [1, 50])
def test_like_a_cache_with_scales_of_heads(nb, n):
    """The same scale in every page: within the bounds' sum of the cache with a scale per head."""
    pages = Pages([(n, 900), (n, 333)], 2, 128, 64)
    for which, s in ((0, 2.0 ** -7), (1, 2.0 ** -6)):
        pages.scale[which] = torch.full_like(pages.scale[which], s)
    out, lse = check_attention(nb, pages, 8, q=(q := torch.randn(2 * n, 8, 128).bfloat16()))
    cache, batch = pages.handles(nb)
    heads = [torch.full((2,), s, device=DEV) for s in (2.0 ** -7, 2.0 ** -6)]
    plain = nb.PagedKVCache(cache.k, cache.v, k_scale=heads[0], v_scale=heads[1])
    lse2 = torch.empty_like(lse)
    out2 = nb.paged_attention(q.to(DEV), plain, batch, lse=lse2)
    want = pages.attention(q)
    within(out - out2, torch.zeros_like(want[0]), 2 * want[2], "out")
    within(lse - lse2, torch.zeros_like(want[1]), 2 * want[3], "lse")


@pytest.mark.parametrize("n", [3, 60])
def test_hidden_nan_values(nb, n):
    """NaN at the last tokens' keys reaches those that see them alone."""
    pages = Pages([(n, 400), (n, 130)], 2, 128, 16, spread=(-6, 6))
    q = torch.randn(2 * n, 4, 128, generator=pages.g).bfloat16()
    clean = pages.attention(q)
    for r, length in ((0, 400), (1, 130)):
        p = int(pages.table[r, (length - 1) // 16])
        pages.raw[1][p, (length - 1) % 16] = NAN
    cache, batch = pages.handles(nb)
    out = nb.paged_attention(q.to(DEV), cache, batch).double().cpu()
    last = torch.tensor([n - 1, 2 * n - 1])
    others = torch.tensor([i for i in range(2 * n) if i not in last.tolist()])
    assert out[last].isnan().all()
    within(out[others], clean[0][others], clean[2][others], "rows that do not see them")


@pytest.mark.parametrize("n", [1, 40])
def test_pages_out_of_range_read_as_zeros(nb, n):
    pages = Pages([(n, 300), (n, 100)], 1, 128, 32)
    bad = {1: -1, 4: 1 << 20}
    cache, batch = pages.handles(nb)
    for i, p in bad.items():
        real = int(pages.table[0, i])
        pages.raw[0][real] = pages.raw[1][real] = 0
        pages.scale[0][real] = pages.scale[1][real] = 1.0
        batch.page_table[0, i] = p
    q = torch.randn(2 * n, 2, 128, generator=pages.g).bfloat16()
    ws = nb.paged_attention_workspace(cache, batch, 2)
    out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    want = pages.attention(q)
    within(out, want[0], want[2], "out")


@pytest.mark.parametrize("n", [1, 30])
def test_many_requests(nb, n):
    """More requests than the chunk kernel plans for itself, with empty ones between."""
    reqs = [(0 if i % 7 == 3 else n, n + (i * 37) % 200) for i in range(450)]
    check_attention(nb, Pages(reqs, 1, 64, 16), 2)


@pytest.mark.parametrize("hk", [1, 2])
@pytest.mark.parametrize("batch", [384, 385, 900])
def test_many_requests_of_wide_heads(nb, hk, batch):
    """More requests than a block of the few-row kernel has threads, with empty ones between."""
    reqs = [(0 if i % 7 == 3 else 1 + i % 3, 3 + (i * 37) % 300) for i in range(batch)]
    check_attention(nb, Pages(reqs, hk, 128, 16), 4 * hk)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("reqs,hk,hq", [([(2, 9000)], 1, 5), ([(1, 100), (1, 20000), (3, 129)], 1, 4),
                                        ([(4, 30000)], 2, 8), ([(40, 12000)], 1, 2)])
def test_an_axis_in_many_pieces(nb, reqs, hk, hq, D):
    """A request's keys over most blocks of the GPU: more pieces than a row has lanes in the join."""
    check_attention(nb, Pages(reqs, hk, D, 64, True), hq)


@pytest.mark.parametrize("n", [2, 40])
def test_results_are_the_same_bits_from_a_graph_and_another_stream(nb, n):
    pages = Pages([(n, 700), (n, 41)], 2, 128, 16)
    cache, batch = pages.handles(nb)
    q = torch.randn(2 * n, 6, 128, generator=pages.g).bfloat16().to(DEV)
    ws = nb.paged_attention_workspace(cache, batch, 6)
    first = nb.paged_attention(q, cache, batch, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = nb.paged_attention(q, cache, batch, ws=nb.paged_attention_workspace(cache, batch, 6), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph, third = torch.cuda.CUDAGraph(), torch.empty_like(first)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nb.paged_attention(q, cache, batch, ws=ws, out=third)
    for _ in range(2):
        third.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, second) and torch.equal(first, third)


# ----------------------------------------------------------------- append --
def append_reference(pages, k, v, rope, weight, pairs, eps, old):
    """What attn_kv_append leaves: for each side (values and bounds over the whole cache,
    scales, whether the scale stands away from a border), [pages, page, H, D]."""
    T = pages.tokens
    pos = torch.cat([torch.arange(length - n, length) for n, length in pages.reqs] + [torch.zeros(0).long()])
    kx, mag = ref.transform(k, weight, pos, rope, pairs, eps)
    off = (pages.D + 16) * 2.0 ** -24 * mag                # of the fp32 value before its rounding
    found = []
    for which, x, err in ((0, kx, off), (1, v.double(), torch.zeros(T, pages.hk, pages.D, dtype=torch.float64))):
        raw, scale = old[which][0].clone(), old[which][1].clone()
        val, bound = values(raw), torch.zeros(raw.shape, dtype=torch.float64)
        sure = torch.ones_like(scale, dtype=torch.bool)
        for r, (n, length) in enumerate(pages.reqs):
            at, p = int(pages.q_start[r]), length - n
            while p < length:
                take = min(length - p, pages.page - p % pages.page)
                page, o = int(pages.table[r, p // pages.page]), p % pages.page
                for h in range(pages.hk):
                    here = x[at:at + take, h]
                    finite = torch.where(here.isfinite(), here.abs(), 0.0)
                    top, slack = float(finite.max()), float(err[at:at + take, h].max())
                    s = sref.scale_of(top)
                    if o:
                        had = min(max(float(scale[page, h]), sref.LOW), sref.HIGH) \
                            if not math.isnan(float(scale[page, h])) else sref.LOW
                        if s > had:
                            val[page, :o, h] = sref.e4m3(val[page, :o, h] * (had / s))
                        s = max(s, had)
                    sure[page, h] = sref.scale_of(top - slack) == sref.scale_of(top + slack)
                    scale[page, h] = s
                    val[page, o:o + take, h] = (here / s).clamp(-448, 448)
                    # half a step of E4M3 (2^-4 of the value, 2^-10 among the smallest)
                    bound[page, o:o + take, h] = torch.maximum(
                        2.0 ** -4 * val[page, o:o + take, h].abs(), torch.tensor(2.0 ** -10).double()) \
                        + err[at:at + take, h] / s
                p, at = p + take, at + take
        found.append((val, bound, scale, sure))
    return found


@pytest.mark.parametrize("reqs,hk,hq,D,page,heads_first,rot,norm,pairs,powers", [
    ([(1, 1)], 1, 2, 128, 16, False, 128, True, False, True),
    ([(1, 17), (1, 40), (1, 16), (0, 30), (1, 33)], 2, 6, 128, 16, True, 128, True, False, True),
    ([(5, 70), (3, 3), (2, 64), (4, 66)], 3, 3, 64, 64, False, 32, False, True, True),
    ([(5, 70), (3, 19), (2, 50), (4, 66)], 2, 4, 128, 32, True, 64, True, True, False),
    ([(300, 300), (57, 100), (1, 20), (130, 131)], 2, 4, 128, 16, False, 128, True, False, True),
    ([(300, 310), (200, 700)], 1, 3, 128, 64, True, 128, True, False, True),
    ([(300, 310), (200, 700)], 2, 2, 64, 64, False, 64, False, False, True),
    ([(700, 1001)], 1, 2, 128, 128, False, 128, False, True, False),
    ([(1500, 2300)], 1, 1, 128, 1024, True, 128, True, False, True),      # pages of several rounds
    ([(1500, 1500), (90, 95)], 1, 0, 64, 512, False, 0, True, False, True),
    ([(900, 901)], 2, 2, 64, 256, False, 48, True, True, True)])
def test_append(nb, reqs, hk, hq, D, page, heads_first, rot, norm, pairs, powers):
    pages = Pages(reqs, hk, D, page, heads_first, powers=powers)
    g, T = pages.g, pages.tokens
    qkv = (torch.randn(T, (hq + 2 * hk) * D, generator=g)
           * torch.exp2(torch.randint(-6, 4, (T, 1), generator=g).float())).bfloat16()
    rope = rope_table(max(length for _, length in reqs), rot) if rot else None
    wq, wk = ((1 + torch.randn(D, generator=g) / 4).bfloat16() if norm else None for _ in range(2))
    x = qkv.to(DEV)
    q, k, v = x.split([hq * D, hk * D, hk * D], 1)
    q, k, v = q.unflatten(1, (hq, D)) if hq else None, k.unflatten(1, (hk, D)), v.unflatten(1, (hk, D))
    old = [(raw.clone(), s.clone()) for raw, s in zip(pages.raw, pages.scale)]
    cache, batch = pages.handles(nb)
    ws = nb.attn_workspace()
    put = lambda t: t.to(DEV) if t is not None else None   # noqa: E731
    qo = nb.kv_append(cache, batch, k, v, put(rope), put(wk), q=q, q_weight=put(wq), eps=1e-5, interleaved=pairs,
                      ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    if hq:
        pos = torch.cat([torch.arange(length - n, length) for n, length in reqs])
        y, mag = ref.transform(q.cpu(), wq, pos, rope, pairs, 1e-5)
        within(qo, y, ref.transform_bound(y, mag), "queries")
    want = append_reference(pages, k.cpu(), v.cpu(), rope, wk, pairs, 1e-5, old)
    for side, scale, (val, bound, s, sure), (before, s_before) in zip((cache.k, cache.v),
                                                                      (cache.k_scale, cache.v_scale), want, old):
        raw = side.view(torch.uint8).cpu()
        raw = raw.transpose(1, 2) if heads_first else raw
        got, s_got = values(raw), scale.cpu()
        assert sure.all()                                  # (no scale hangs on a rounding here)
        assert torch.equal(s_got.nan_to_num(-1), s.float().nan_to_num(-1))
        same = val.isnan()
        assert torch.equal(got.isnan(), same)
        over = (got - val).abs() - bound
        assert (over[~same] <= 0).all(), over[~same].max()
        # pages without new tokens, and offsets past a request's length: the bytes as they were
        untouched = (bound == 0) & (val == values(before))
        assert torch.equal(raw[untouched], before[untouched])


def test_a_growing_page_keeps_its_values(nb):
    """Scales double token by token, sixteen times: what the first tokens were stays, to
    the last bit while it is above 2^-6 of the scale; then each doubling rounds it by up to
    2^-10 of the scale, less than 2^-9 of the last one in all."""
    D, page = 128, 16
    pages = Pages([(1, 1)], 1, D, page, extra=0)
    cache, batch = pages.handles(nb)
    batch.page_table[0, 0] = 0
    first = (torch.randn(1, 1, D).clamp(-3.4, 3.4) * 100).bfloat16()
    exact = None
    for i in range(page):
        x = first if i == 0 else torch.full((1, 1, D), 448.0 * 2.0 ** i).bfloat16()
        batch.kv_len.fill_(i + 1)
        nb.kv_append(cache, batch, x.to(DEV), x.to(DEV))
        s = float(cache.v_scale[0, 0])
        if i == 0:
            exact = values(cache.v.view(torch.uint8).cpu())[0, 0, 0] * s
            assert s == sref.scale_of(float(first.abs().max()))
            s0 = s
        assert s == max(s0, 2.0 ** i)
        now = values(cache.v.view(torch.uint8).cpu())[0, 0, 0] * s
        clear = exact.abs() >= 2.0 ** -6 * s
        assert torch.equal(now[clear], exact[clear])
        assert ((now - exact).abs() < 2.0 ** -9 * s).all()
        assert torch.equal(cache.k.view(torch.uint8), cache.v.view(torch.uint8))


def test_scales_at_borders_zeros_and_values_that_are_not_finite(nb):
    """One head for each: 448 s exactly and the next number above, zeros alone, infinities
    (they saturate) and NaN (stays) among numbers, nothing but infinities, the smallest and
    the largest bf16 numbers (beyond the scales' range: 0 and saturated)."""
    D, H = 64, 8
    x = torch.zeros(2, H, D, dtype=torch.float64)
    x[0, 0, 3], x[1, 0, 4] = 448.0, -100.0
    x[0, 1, 3] = 450.0                                     # 1.7578125 * 2^8: the next bf16 number
    x[0, 3, 0], x[0, 3, 1], x[1, 3, 2] = math.inf, 5.0, -math.inf
    x[0, 4, 0], x[1, 4, 1] = math.nan, 3.0
    x[:, 5] = math.inf
    x[0, 6, 0] = 2.0 ** -130
    x[0, 7, 0], x[1, 7, 1] = 3e38, 1.0
    x = x.bfloat16()
    pages = Pages([(2, 2)], H, D, 16, extra=0)
    cache, batch = pages.handles(nb)
    nb.kv_append(cache, batch, x.to(DEV), x.to(DEV))
    p = int(pages.table[0, 0])
    for side, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        got = values(side.view(torch.uint8).cpu())[p, :2]
        assert scale[p].cpu().tolist() == [1.0, 2.0, 2.0 ** -40, 2.0 ** -6, 2.0 ** -7, 2.0 ** -40, 2.0 ** -40, 2.0 ** 40]
        assert got[0, 0, 3] == 448 and got[1, 0, 4] == sref.e4m3(torch.tensor(-100.0).double())
        assert got[0, 1, 3] == sref.e4m3(torch.tensor(225.0).double())
        assert (got[:, 2] == 0).all()
        assert got[0, 3, 0] == 448 and got[1, 3, 2] == -448 and got[0, 3, 1] == 320
        assert got[0, 4, 0].isnan() and got[1, 4, 1] == 384 and not got[:, 4].flatten()[1:].isnan().any()
        assert (got[:, 5] == 448).all() and (got[:, 6] == 0).all()
        assert got[0, 7, 0] == 448 and got[1, 7, 1] == 0


def test_tokens_that_cannot_be_placed_are_reported_and_left_out(nb):
    """Positions below 0 and past the rotation's table, pages outside the cache or the
    table: nothing of those tokens is written, nor counts for a scale; the others are."""
    D, page = 128, 16
    pages = Pages([(3, 2), (20, 30), (2, 48), (18, 36)], 1, D, page, extra=2)
    x = torch.ones(pages.tokens, 1, D)
    x[0], x[3 + 20:3 + 22] = 4000.0, 4000.0                # what must not count
    x[3 + 15 + 4:3 + 20] = 3000.0                          # positions 29: past the rotation's table
    x = x.bfloat16()
    rope = rope_table(29, D)
    rope[:, D // 2:] = 0
    rope[:, :D // 2] = 1                                   # turns nothing
    for scale in pages.scale:
        scale[:] = 2.0 ** -5
    cache, batch = pages.handles(nb)
    batch.page_table[2, 2] = -7                            # of request 2's tokens, 46 and 47
    batch.page_table[3, 1] = cache.k.shape[0]              # of request 3's, 18 .. 31
    before = cache.v.view(torch.uint8).clone()
    ws = nb.attn_workspace()
    q = torch.full((pages.tokens, 1, D), 2.0).bfloat16().to(DEV)
    q_out = torch.full_like(q, 9)
    nb.kv_append(cache, batch, x.to(DEV), x.to(DEV), rope.to(DEV), q=q, q_out=q_out, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    v, s = cache.v.view(torch.uint8).cpu(), cache.v_scale.cpu()
    placed = torch.zeros_like(v, dtype=torch.bool)
    one = sref.scale_of(1.0)
    rows = [False] * pages.tokens
    for r, (n, length) in enumerate(pages.reqs):
        for i in range(n):
            pos = length - n + i
            if pos < 0 or pos >= 29 or (r == 2) or (r == 3 and pos // page == 1):
                continue
            p = int(pages.table[r, pos // page])
            placed[p, pos % page] = True
            rows[int(pages.q_start[r]) + i] = True
            fresh = pos // page * page >= length - n
            assert float(s[p, 0]) == (one if fresh else 2.0 ** -5), (r, pos)
    assert placed.any() and torch.equal(v[~placed], before.cpu()[~placed])
    assert ((values(v) * s.double()[:, None, :, None])[placed] == 1).all()
    rows = torch.tensor(rows)
    got = q_out.cpu()
    assert (got[rows] == 2).all() and (got[~rows] == 9).all()


def test_rows_of_no_request_and_empty_requests(nb):
    pages = Pages([(0, 20), (2, 18), (0, 0)], 1, 64, 16)
    cache, batch = pages.handles(nb, max_new=4)
    batch.q_start.add_(1)                                  # row 0 and rows from 3 on belong to nobody
    x = torch.ones(6, 1, 64).bfloat16().to(DEV)
    q_out = torch.full((6, 1, 64), 9.0).bfloat16().to(DEV)
    before = cache.k.view(torch.uint8).clone()
    ws = nb.attn_workspace()
    nb.kv_append(cache, batch, x, x, q=x, q_out=q_out, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    assert (q_out[1:3] == 1).all() and (q_out[0] == 9).all() and (q_out[3:] == 9).all()
    p = int(pages.table[1, 1])
    changed = (cache.k.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [p]


def test_append_twice_and_from_a_graph(nb):
    """The same tokens again change nothing; a captured append follows lengths and tables."""
    pages = Pages([(3, 20), (1, 16), (2, 70)], 2, 128, 16)
    cache, batch = pages.handles(nb)
    k = torch.randn(6, 2, 128, generator=pages.g).bfloat16().to(DEV) * 3
    v = torch.randn(6, 2, 128, generator=pages.g).bfloat16().to(DEV)
    start = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]

    def state():
        return [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale.nan_to_num(-1),
                                    cache.v_scale.nan_to_num(-1))]

    def restore():
        for t, s in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale), start):
            t.copy_(s)
    nb.kv_append(cache, batch, k, v)
    once = state()
    nb.kv_append(cache, batch, k, v)
    assert all(torch.equal(a, b) for a, b in zip(once, state()))
    restore()
    ws, graph = nb.attn_workspace(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nb.kv_append(cache, batch, k, v, ws=ws)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(once, state()))
    # two tokens on: other offsets, the next page for the first request
    batch.kv_len.add_(13)
    batch.page_table[0, 2] = batch.page_table[1, 1] = batch.page_table[2, 5] = 0
    batch.page_table[0, 2], batch.page_table[1, 1], batch.page_table[2, 5] = [int(p) for p in pages_free(pages)]
    restore()
    graph.replay()
    replayed = state()
    restore()
    nb.kv_append(cache, batch, k, v, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(replayed, state())) and nb.read_status(ws) == 0


def test_append_with_queries_in_place(nb):
    """q_out may be q itself: the same rows as into a buffer of its own."""
    for reqs in ([(3, 20), (1, 16)], [(100, 130), (60, 60)]):
        pages = Pages(reqs, 2, 128, 16)
        x = torch.randn(pages.tokens, 10, 128, generator=pages.g).bfloat16().to(DEV)
        rope = rope_table(130, 128).to(DEV)
        w = torch.ones(128).bfloat16().to(DEV)
        cache, batch = pages.handles(nb)
        q, k, v = x.split([6, 2, 2], 1)
        apart = nb.kv_append(cache, batch, k, v, rope, w, q=q, q_weight=w)
        again = nb.kv_append(cache, batch, k, v, rope, w, q=q, q_weight=w, q_out=q)
        assert again is q and torch.equal(apart, q)


def pages_free(pages):
    used = {int(p) for r, (_, length) in enumerate(pages.reqs)
            for p in pages.table[r, :-(-length // pages.page)]}
    return [p for p in range(pages.raw[0].shape[0]) if p not in used][:3]


def test_pages_past_32_bit_offsets(nb):
    """A cache of 3 GB a side: the append's and the attention's offsets are 64 bits."""
    D, H, page, n = 128, 8, 64, 48000
    shape = (n, page, H, D)
    k = torch.zeros(shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v = torch.zeros(shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = [torch.ones(n, H, device=DEV) for _ in range(2)]
    cache = nb.PagedKVCache(k, v, k_scale=scales[0], v_scale=scales[1])
    batch = nb.AttnBatch(torch.tensor([0, 70], dtype=torch.int32, device=DEV),
                         torch.tensor([70], dtype=torch.int32, device=DEV),
                         torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device=DEV), max_new=70)
    x = torch.randn(70, H, D, device=DEV).bfloat16()
    ws = nb.attn_workspace()
    nb.kv_append(cache, batch, x, x, ws=ws)
    got = torch.cat([v[n - 1].double() * scales[1][n - 1, :, None], v[n - 2].double() * scales[1][n - 2, :, None]])[:70]
    assert nb.read_status(ws) == 0
    bound = torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scales[1][n - 2:].double().max())
    assert ((got - x.double()).abs() <= bound).all()
    assert int(torch.count_nonzero(v[:n - 2].view(torch.uint8))) == 0
    # 70 equal keys, of which a token sees its own and those before: the mean of their values
    for first, rows in ((0, 70), (69, 1)):
        step = nb.AttnBatch(torch.tensor([0, rows], dtype=torch.int32, device=DEV), batch.kv_len, batch.page_table,
                            max_new=rows)
        out = nb.paged_attention(torch.zeros(rows, H, D, device=DEV).bfloat16(), cache, step).double()
        mean = got.cumsum(0) / torch.arange(1, 71, device=DEV)[:, None, None]
        size = got.abs().cumsum(0) / torch.arange(1, 71, device=DEV)[:, None, None]
        assert ((out - mean[first:]).abs() <= 2.0 ** -8 * (mean[first:].abs() + size[first:]) + 2.0 ** -16).all()


@pytest.mark.parametrize("n", [1, 40])
def test_small_weights_beside_large_ones_that_come_later(nb, n):
    """Scores that rise by up to 2^4 and less over the first, so that references stay where
    they are while weights grow, and one key 20 powers of two above thousands whose weights
    together are a hundredth of its own: both within the bounds of single weights."""
    L, D = 4096, 128
    pages = Pages([(n, L)], 1, D, 64)
    for scale in pages.scale:
        scale[:] = 2.0 ** -4
    k = torch.zeros(L, D, dtype=torch.float64)
    k[:, 0] = torch.linspace(0, 1, L).double()             # a slow rise ...
    k[L // 2, 1] = 14.0                                    # ... and one key far above
    raw = sref.e4m3(k * 16)
    v = sref.e4m3(torch.randn(L, D, generator=pages.g).double() * 64 + 64)
    for which, x in ((0, raw), (1, v)):
        for i in range(L // 64):
            pages.raw[which][int(pages.table[0, i]), :, 0] = \
                x[i * 64:(i + 1) * 64].to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.zeros(n, 2, D)
    q[:, 0, 0], q[:, 1, 0] = 4 * math.log(2) * D ** 0.5, 4 * math.log(2) * D ** 0.5
    q[:, 1, 1] = math.log(2) * D ** 0.5
    check_attention(nb, pages, 2, q=q.bfloat16())
