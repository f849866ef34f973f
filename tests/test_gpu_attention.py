"""The attention operators against their 64-bit form (tests/_attention_reference.py):
head norm with rotation, appending to the paged cache, attention over it."""
import math

import pytest
import torch

import _attention_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD_INDEX = 7


@pytest.fixture(scope="module")
def nb():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_block_scaled_route_gb300 import binding
    return binding


def _table(positions, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _within(got, want, bound, what):
    got, err = got.double().cpu(), None
    same_inf = got.isinf() & (got == want)
    err = torch.where(same_inf, torch.zeros_like(want), (got - want).abs())
    assert not err.isnan().any(), what
    over = err - bound
    assert (over <= 0).all(), f"{what}: {err.max():.3g}, over its bound by {over.max():.3g}"


# ------------------------------------------------------- norm and rotation --
@pytest.mark.parametrize("T,hq,hk,D,rot,norm,pairs", [
    (1, 7, 1, 128, 128, True, False), (1, 1, 0, 64, 0, True, False), (5, 56, 8, 128, 128, True, False),
    (3, 3, 3, 64, 32, False, True), (33, 5, 2, 128, 16, True, True), (130, 2, 1, 64, 64, True, False),
    (17, 4, 4, 128, 64, False, False), (2, 9, 3, 64, 16, True, False),
    (700, 56, 8, 128, 128, True, False), (1031, 20, 4, 64, 48, True, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_qk_norm_rope(nb, T, hq, hk, D, rot, norm, pairs, in_place):
    g = torch.Generator().manual_seed(T * 1000 + hq)
    qkv = (torch.randn(T, (hq + 2 * hk) * D, generator=g) * 3).bfloat16()
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    rope = _table(300, rot) if rot else None
    wq = (1 + torch.randn(D, generator=g) / 4).bfloat16() if norm else None
    wk = (1 + torch.randn(D, generator=g) / 4).bfloat16() if norm else None
    x = qkv.to(DEV)
    q, k, rest = x.split([hq * D, hk * D, hk * D], 1)     # strided views of one projection
    q, k = q.unflatten(1, (hq, D)), k.reshape(T, 0, D) if hk == 0 else k.unflatten(1, (hk, D))
    dev = lambda t: t.to(DEV) if t is not None else None   # noqa: E731
    q_cpu, k_cpu, rest_cpu = q.cpu(), k.cpu(), rest.cpu()
    ws = nb.attn_workspace()
    qo, ko = nb.qk_norm_rope(q, k, dev(pos), dev(rope), dev(wq), dev(wk), eps=1e-5,
                             interleaved=pairs, ws=ws, q_out=q if in_place else None,
                             k_out=k if in_place else None)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    for got, src, w in ((qo, q_cpu, wq), (ko, k_cpu, wk)):
        y, mag = ref.transform(src, w, pos, rope, pairs, 1e-5)
        _within(got, y, ref.transform_bound(y, mag), "rows")
    assert torch.equal(rest.cpu(), rest_cpu)


def test_qk_norm_rope_zero_and_infinite_rows(nb):
    """A zero row stays zero (eps keeps the norm finite); an infinite element
    past the rotated part does not reach the others without a norm."""
    D, rot = 64, 32
    q = torch.zeros(2, 1, D).bfloat16()
    q[1, 0, 60] = math.inf
    q[1, 0, 0] = 2.0
    rope = _table(4, rot)
    pos = torch.tensor([3, 3], dtype=torch.int32)
    k = torch.zeros(2, 1, D).bfloat16().to(DEV)
    qo, _ = nb.qk_norm_rope(q.to(DEV), k, pos.to(DEV), rope.to(DEV))
    out = qo.cpu().double()
    assert (out[0] == 0).all() and out[1, 0, 60] == math.inf
    rest = torch.cat([out[1, 0, :60], out[1, 0, 61:]])
    assert rest.isfinite().all() and abs(out[1, 0, 0] - 2 * math.cos(3)) < 0.02
    w = torch.ones(D).bfloat16().to(DEV)
    qo, _ = nb.qk_norm_rope(q[:1].to(DEV), k[:1], pos[:1].to(DEV), rope.to(DEV), w, w)
    assert (qo == 0).all()


def test_qk_norm_rope_bad_position_is_reported(nb):
    T, D = 9, 128
    q = torch.randn(T, 4, D, device=DEV).bfloat16()
    k = torch.randn(T, 1, D, device=DEV).bfloat16()
    pos = torch.arange(T, dtype=torch.int32)
    pos[2], pos[5] = -1, 9
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    ws = nb.attn_workspace()
    nb.qk_norm_rope(q, k, pos.to(DEV), _table(T, D).to(DEV), q_out=qo, k_out=ko, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    bad = torch.tensor([2, 5])
    good = torch.tensor([0, 1, 3, 4, 6, 7, 8])
    assert (qo[bad] == 7).all() and (ko[bad] == 7).all()
    y, mag = ref.transform(q.cpu()[good], None, pos[good], _table(T, D), False, 0)
    _within(qo[good.to(DEV)], y, ref.transform_bound(y, mag), "valid rows")


# ------------------------------------------------------------ paged caches --
class Paged:
    """Requests of (new tokens, cached length) on a cache of scattered pages.
    Everything past a request's length is NaN: the unused part of its last
    page, free pages; table entries past its pages point nowhere."""

    def __init__(self, reqs, hk, D, page, heads_first=False, fp8=False, seed=0, extra=3):
        g = torch.Generator().manual_seed(seed + 17 * hk + D + page)
        self.reqs, self.hk, self.D, self.page = reqs, hk, D, page
        self.heads_first, self.fp8 = heads_first, fp8
        need = [-(-max(length, 0) // page) for _, length in reqs]
        pages = sum(need) + extra
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(reqs), max(need + [1]) + 1), -123456, dtype=torch.int32)
        shape = (pages, hk, page, D) if heads_first else (pages, page, hk, D)
        self.k_scale = torch.rand(hk, generator=g) * 0.02 + 0.01 if fp8 else None
        self.v_scale = torch.rand(hk, generator=g) * 0.02 + 0.01 if fp8 else None

        def values():
            x = torch.randn(shape, generator=g)
            return (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.bfloat16()
        self.k, self.v = values(), values()
        used = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for r, (n, length) in enumerate(reqs):
            mine = order[at:at + need[r]]
            self.table[r, :need[r]] = mine.int()
            at += need[r]
            for j in range(length):
                used[mine[j // page], j % page] = True
        hole = ~used[:, None, :, None] if heads_first else ~used[:, :, None, None]
        for c in (self.k, self.v):
            raw = c.view(torch.uint8) if fp8 else c
            raw.copy_(torch.where(hole, torch.full_like(raw, 0x7F if fp8 else math.nan), raw))
        self.q_start = torch.tensor([0] + [n for n, _ in reqs]).cumsum(0).int()
        self.kv_len = torch.tensor([length for _, length in reqs], dtype=torch.int32)
        self.T = int(self.q_start[-1])

    def handles(self, nb, max_new=None):
        dev = lambda t: t.to(DEV) if t is not None else None   # noqa: E731
        self.kd, self.vd = dev(self.k), dev(self.v)
        cache = nb.PagedKVCache(self.kd, self.vd, heads_first=self.heads_first,
                                k_scale=dev(self.k_scale), v_scale=dev(self.v_scale))
        top = max([n for n, _ in self.reqs] + [1])
        batch = nb.AttnBatch(dev(self.q_start), dev(self.kv_len), dev(self.table),
                             max_new=max_new or top)
        return cache, batch

    def reference(self, q, **kw):
        return ref.attention(q, self.k, self.v, self.q_start, self.kv_len, self.table,
                             self.heads_first, self.k_scale, self.v_scale, **kw)


ONE = [(1, 1), (1, 16), (1, 17), (1, 500), (0, 40), (1, 129), (1, 64), (1, 300)]
FEW = [(3, 3), (5, 200), (0, 0), (2, 129), (1, 1), (5, 5), (4, 700)]
CHUNK = [(37, 37), (130, 400), (1, 77), (0, 9), (64, 129), (128, 128)]
EMPTY = [(4, 2), (3, 0), (1, 1), (6, 5)]          # the first tokens have no position


def _check(nb, case, hq, window=0, scale=None, tag="", strided=False, max_new=None):
    g = torch.Generator().manual_seed(hq)
    if strided:
        wide = (torch.randn(case.T, hq + 3, case.D + 8, generator=g) * 1.5).bfloat16().to(DEV)
        q = wide[:, 1:hq + 1, :case.D]
        out = torch.full((case.T, hq + 1, case.D), 5.0, device=DEV).bfloat16()[:, :hq]
    else:
        q = (torch.randn(case.T, hq, case.D, generator=g) * 1.5).bfloat16().to(DEV)
        out = torch.full_like(q, 5.0)
    cache, batch = case.handles(nb, max_new)
    lse = torch.full((case.T, hq), 5.0, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, hq, case.T)
    for _ in range(2):                             # the workspace as the first call left it
        nb.paged_attention(q, cache, batch, scale=scale, window=window, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q.cpu(), window=window, scale=scale)
    _within(out, want, b_out, f"out {tag}")
    _within(lse, wlse, b_lse, f"lse {tag}")
    if strided:
        assert (out._base[:, hq] == 5.0).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("reqs", [ONE, FEW, CHUNK, EMPTY], ids=["one", "few", "chunk", "empty"])
@pytest.mark.parametrize("hq,hk,D,page,heads_first", [
    (7, 1, 128, 16, False), (16, 2, 64, 32, True), (3, 3, 128, 128, True), (16, 1, 64, 16, False),
    (10, 2, 128, 256, False)])
def test_paged_attention(nb, reqs, hq, hk, D, page, heads_first, fp8):
    _check(nb, Paged(reqs, hk, D, page, heads_first, fp8), hq)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 15, 64, 128, 130, 1000])
@pytest.mark.parametrize("reqs", [ONE, FEW, CHUNK], ids=["one", "few", "chunk"])
def test_paged_attention_window(nb, reqs, window, fp8):
    _check(nb, Paged(reqs, 2, 64, 16, True, fp8, seed=3), 6, window=window)


@pytest.mark.parametrize("reqs,hq,hk", [([(1, 4000)], 8, 1), ([(1, 2500), (1, 1)], 4, 2),
                                        ([(40, 3000)], 8, 1), ([(300, 900), (1, 800)], 2, 1),
                                        ([(9, 2000), (2, 1990)], 16, 1)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_paged_attention_long_axis(nb, reqs, hq, hk, fp8):
    """Few rows over many keys: the work is split along the keys and joined."""
    _check(nb, Paged(reqs, hk, 128, 64, False, fp8, seed=5), hq)


def test_paged_attention_strided_and_scaled(nb):
    for reqs in (ONE, FEW, CHUNK):
        _check(nb, Paged(reqs, 2, 64, 16, seed=9), 6, scale=0.3, strided=True)


def test_paged_attention_loose_max_new(nb):
    """max_new is a bound: batches of shorter chunks give the same results."""
    for top in (1, 2, 9, 33, 300):
        _check(nb, Paged(ONE, 1, 128, 16, seed=top), 8, max_new=top)


@pytest.mark.parametrize("hq,D", [(8, 128), (4, 64)])
@pytest.mark.parametrize("n", [1, 40])
def test_paged_attention_large_scores(nb, hq, D, n):
    """Scores far apart: one key takes (almost) all the weight, early and late
    in the axis, and scores of a size where exp without the maximum overflows."""
    case = Paged([(n, 700), (n, n)], 1, D, 32, seed=21)
    q = torch.randn(case.T, hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    q *= 40
    cache, batch = case.handles(nb)
    lse = torch.empty(case.T, hq, device=DEV)
    out = nb.paged_attention(q.to(DEV), cache, batch, lse=lse)
    want, wlse, b_out, b_lse = case.reference(q)
    _within(out, want, b_out, "out")
    _within(lse, wlse, b_lse, "lse")


def test_paged_attention_on_another_stream(nb):
    case = Paged(FEW, 2, 128, 16, seed=2)
    q = torch.randn(case.T, 8, 128, device=DEV).bfloat16()
    cache, batch = case.handles(nb)
    want = nb.paged_attention(q, cache, batch)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = nb.paged_attention(q, cache, batch)
        s.synchronize()
    assert torch.equal(got, want)
    got2 = torch.empty_like(q)
    ws = nb.paged_attention_workspace(cache, batch, 8, case.T)
    torch.cuda.synchronize()
    nb.paged_attention(q, cache, batch, out=got2, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(got2, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 70])
def test_paged_attention_e4m3_uneven_queries(nb, n, D):
    """Query rows with elements far above the rest, rows of zeros and of the smallest
    numbers, on an E4M3 cache.  Queries are scaled by a row's maximum and held to 16
    bits or two E4M3 numbers: an element to within 2^-17 of the maximum, so that a
    score may be off by scale * 2^-17 max|q| sum|k| beside the usual bound."""
    case = Paged([(n, n + 90)], 1, D, 16, seed=4, fp8=True)
    g = torch.Generator().manual_seed(n + D)
    q = torch.randn(n, 8, D, generator=g)
    q[:, 0, 3] *= 300
    q[:, 1, ::2] *= 2.0 ** -9
    q[:, 2] = 0
    q[:, 3] = 1e-39
    q[:, 4] *= 2.0 ** -60
    q[:, 5, D // 2:] = 0
    q = q.bfloat16()
    cache, batch = case.handles(nb)
    lse = torch.empty(n, 8, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, 8, n)
    out = nb.paged_attention(q.to(DEV), cache, batch, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q)
    k, v = (ref.key_rows(c, case.table[0], 16, n + 90, 0, False, sc)
            for c, sc in ((case.k, case.k_scale), (case.v, case.v_scale)))
    extra = D ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * k.abs().sum(1).max()
    _within(out, want, b_out + 2 * extra[..., None] * v.abs().max(), "out")
    _within(lse, wlse, b_lse + extra, "lse")


@pytest.mark.parametrize("count,hq,hk,D,fp8", [(400, 32, 1, 64, False), (1100, 17, 1, 128, True),
                                               (1100, 20, 10, 64, False)],
                         ids=["400", "1100-e4m3", "1100-few"])
def test_paged_attention_many_requests(nb, count, hq, hk, D, fp8):
    """More requests than a CTA has threads to plan them with, empty ones among them."""
    case = Paged([((i * 5 % 7) > 1, (i * 7) % 19 + 1) for i in range(count)], hk, D, 16, seed=8, fp8=fp8)
    _check(nb, case, hq)


def test_paged_attention_in_a_graph_follows_the_batch(nb):
    """Captured once; lengths and pages are device data, refilled in place."""
    a, b = Paged([(1, 300), (1, 70)], 2, 128, 16, seed=1), Paged([(1, 33), (1, 301)], 2, 128, 16, seed=1)
    q = torch.randn(2, 8, 128, device=DEV).bfloat16()
    cache, batch = a.handles(nb)
    ws = nb.paged_attention_workspace(cache, batch, 8, 2)
    out = torch.empty_like(q)
    nb.paged_attention(q, cache, batch, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nb.paged_attention(q, cache, batch, out=out, ws=ws)
    for case in (a, b):
        a.kd.copy_(case.k[:a.k.shape[0]]) if case.k.shape[0] >= a.k.shape[0] else a.kd[:case.k.shape[0]].copy_(case.k)
        a.vd.copy_(case.v[:a.v.shape[0]]) if case.v.shape[0] >= a.v.shape[0] else a.vd[:case.v.shape[0]].copy_(case.v)
        batch.kv_len.copy_(case.kv_len)
        w = min(batch.page_table.shape[1], case.table.shape[1])
        batch.page_table[:, :w].copy_(case.table[:, :w])
        graph.replay()
        torch.cuda.synchronize()
        want, _, bound, _ = case.reference(q.cpu())
        _within(out, want, bound, "replayed")
    assert nb.read_status(ws) == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("reqs,hq,hk,D", [([(5, 200), (3, 3)], 6, 2, 128), ([(5, 133)], 4, 4, 64),
                                          ([(90, 300), (20, 20)], 4, 2, 128), ([(90, 90)], 1, 1, 64),
                                          ([(300, 450)], 2, 1, 128), ([(260, 260)], 3, 3, 64)])
def test_paged_attention_hidden_values_that_are_not_finite(nb, reqs, hq, hk, D, window, fp8):
    """Infinities and NaN in keys and values reach the tokens that see them, and no
    others: they stand at keys that the window or the causal order hides from some
    tokens of the same chunk."""
    case = Paged(reqs, hk, D, 16, seed=31, fp8=fp8)
    g = torch.Generator().manual_seed(5)
    inf = math.nan if fp8 else math.inf                # (E4M3 has no infinity)
    for r, (n, length) in enumerate(reqs):
        for back, what in ((2, "v"), (n // 2, "v"), (n, "v"), (min(length, n + 30), "v"), (1, "k")):
            j = length - back
            p, o = int(case.table[r, j // 16]), j % 16
            for c, nm in ((case.k, "k"), (case.v, "v")):
                if nm == what:
                    x = c[p, o].float()
                    x[:, int(torch.randint(0, D, (1,), generator=g))] = inf
                    x[0, int(torch.randint(0, D, (1,), generator=g))] = math.nan if what == "v" else inf
                    x[-1, 3] = -inf
                    c[p, o] = x.to(c.dtype)
    q = torch.randn(case.T, hq, D, generator=g).bfloat16()
    cache, batch = case.handles(nb)
    lse = torch.empty(case.T, hq, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, hq, case.T)
    out = nb.paged_attention(q.to(DEV), cache, batch, window=window, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q, window=window)
    for got, w, b in ((out, want, b_out), (lse, wlse, b_lse)):
        got = got.double().cpu()
        fine = w.isfinite()
        assert fine.any()
        assert torch.equal(got.isfinite(), fine)
        over = (got - w).abs()[fine] - b[fine]
        assert (over <= 0).all(), over.max()


@pytest.mark.parametrize("n", [1, 60])
def test_paged_attention_reports_bad_input(nb, n):
    """A page id out of range reads as zeros and is reported; a length past the
    page table row and more new tokens than max_new are reported."""
    case = Paged([(n, 200), (n, 100)], 1, 128, 16, seed=4)
    cache, batch = case.handles(nb)
    q = torch.randn(case.T, 4, 128).bfloat16()
    ws = nb.paged_attention_workspace(cache, batch, 4, case.T)
    batch.page_table[0, 2] = case.k.shape[0]
    out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    zero = case.k.shape[0]
    case.k = torch.cat([case.k, torch.zeros_like(case.k[:1])])
    case.v = torch.cat([case.v, torch.zeros_like(case.v[:1])])
    case.table[0, 2] = zero
    want, _, bound, _ = case.reference(q)
    _within(out, want, bound, "zero page")
    assert nb.lib().nvmoe_clear_status(nb._ptr(ws), nb._stream()) == 0
    batch.page_table[0, 2] = 0
    batch.kv_len[1] = batch.page_table.shape[1] * case.page + 1
    batch.page_table[1].clamp_(min=0)
    nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX


def test_paged_attention_leaves_rows_of_no_request(nb):
    for reqs in ([(1, 30), (2, 40)], [(40, 90), (70, 71)]):
        case = Paged(reqs, 1, 64, 16, seed=6)
        cache, batch = case.handles(nb)
        q = torch.randn(case.T + 5, 4, 64, device=DEV).bfloat16()
        out = torch.full_like(q, 5.0)
        ws = nb.paged_attention_workspace(cache, batch, 4, case.T + 5)
        nb.paged_attention(q, cache, batch, out=out, ws=ws)
        torch.cuda.synchronize()
        assert (out[case.T:] == 5).all()
        want, _, bound, _ = case.reference(q[:case.T].cpu())
        _within(out[:case.T], want, bound, "rows")
        # more new tokens than max_new: the first ones are computed, the rest left
        short = nb.AttnBatch(batch.q_start, batch.kv_len, batch.page_table, max_new=1)
        out.fill_(5.0)
        nb.paged_attention(q, cache, short, out=out, ws=ws)
        torch.cuda.synchronize()
        assert nb.read_status(ws) == BAD_INDEX
        first = case.q_start[:-1].long()
        _within(out[first.to(DEV)], want[first], bound[first], "first tokens")
        rest = torch.ones(case.T + 5, dtype=torch.bool)
        rest[first] = False
        assert (out[rest.to(DEV)] == 5).all()


# ------------------------------------------------------------------ append --
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("reqs", [ONE, FEW, CHUNK], ids=["one", "few", "chunk"])
@pytest.mark.parametrize("hq,hk,D,page,heads_first,rot,norm,pairs,with_q", [
    (7, 1, 128, 16, False, 128, True, False, True), (16, 2, 64, 32, True, 32, True, True, True),
    (3, 3, 128, 128, True, 0, False, False, False), (8, 8, 64, 16, False, 64, False, False, True)])
def test_kv_append(nb, reqs, hq, hk, D, page, heads_first, rot, norm, pairs, with_q, fp8):
    case = Paged(reqs, hk, D, page, heads_first, fp8, seed=11)
    g = torch.Generator().manual_seed(hq)
    q, k, v = ((torch.randn(case.T, h, D, generator=g) * 2).bfloat16() for h in (hq, hk, hk))
    rope = _table(1024, rot) if rot else None
    wq = (1 + torch.randn(D, generator=g) / 4).bfloat16() if norm else None
    wk = (1 + torch.randn(D, generator=g) / 4).bfloat16() if norm else None
    dev = lambda t: t.to(DEV) if t is not None else None   # noqa: E731
    cache, batch = case.handles(nb)
    ws = nb.attn_workspace()
    qo = nb.kv_append(cache, batch, dev(k), dev(v), rope=dev(rope), k_weight=dev(wk),
                      q=dev(q) if with_q else None, q_weight=dev(wq), eps=1e-5,
                      interleaved=pairs, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    pos = torch.cat([torch.arange(length - n, length) for n, length in reqs])
    req = torch.cat([torch.full((n,), r) for r, (n, _) in enumerate(reqs)]).long()
    if with_q:
        y, mag = ref.transform(q, wq, pos, rope, pairs, 1e-5)
        _within(qo, y, ref.transform_bound(y, mag), "q")
    ky, mag = ref.transform(k, wk, pos, rope, pairs, 1e-5)
    kb = ref.transform_bound(ky, mag)
    vy, vb = v.double(), torch.zeros(v.shape, dtype=torch.float64)
    if fp8:
        # half a step of E4M3 (2^-4 relative, 2^-10 below 2^-6) on the value over
        # its scale, the fp32 value's own error beside it
        def stored(y, bound, sc):
            y = y / sc.double()[:, None]
            at = y.clamp(-448, 448)
            return at, (bound - ref.U * y.abs() * sc.double()[:, None]).clamp(min=0) / \
                sc.double()[:, None] * 2 + at.abs() * 2.0 ** -22 + torch.maximum(
                    at.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
        ky, kb = stored(ky, kb, case.k_scale)
        vy, vb = stored(vy, vb, case.v_scale)
    page_of = case.table[req, pos // page].long()
    off = pos % page
    for got, old, want, bound, what in ((case.kd, case.k, ky, kb, "k"), (case.vd, case.v, vy, vb, "v")):
        got = got.cpu()
        new = got.float()                     # (torch does not index 8-bit floats on the CPU)
        new = new[page_of, :, off] if heads_first else new[page_of, off]
        _within(new, want, bound, what)
        # nothing else changed
        raw, was = got.view(torch.uint8).clone(), old.view(torch.uint8).clone()
        for t in (raw, was):
            if heads_first:
                t[page_of, :, off] = 0
            else:
                t[page_of, off] = 0
        assert torch.equal(raw, was)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
def test_cache_offsets_past_32_bits(nb, n, fp8):
    """Pages at the far end of a cache of 2.4e9 elements hold and give what pages
    of a small cache do, bit for bit."""
    hq, hk, D, page = 16, 8, 128, 16
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(n)
    q, k, v = (torch.randn(40, h, D, generator=g, device=DEV).bfloat16() for h in (hq, hk, hk))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    got = []
    for pages, ids in ((3, (2, 0, 1)), (146500, (146499, 0, 140000))):
        kc, vc = (torch.empty(pages, page, hk, D, dtype=dtype, device=DEV) for _ in range(2))
        cache, table = nb.PagedKVCache(kc, vc), i32(*ids)[None]
        everything = nb.AttnBatch(i32(0, 40), i32(40), table, max_new=40)
        nb.kv_append(cache, everything, k, v)
        batch = nb.AttnBatch(i32(0, n), i32(40), table, max_new=n)
        out = nb.paged_attention(q[:n].contiguous(), cache, batch)
        got.append([out] + [c[table[0].long()].view(torch.uint8).flatten(0, 1)[:40].cpu()
                            for c in (kc, vc)])
        del kc, vc, cache
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].isfinite().all()


def test_kv_append_e4m3_rounds_to_nearest_and_saturates(nb):
    """Without a scale the stored bytes are torch's cast of the clamped value."""
    D, page = 128, 16
    case = Paged([(3, 40)], 1, D, page, fp8=True)
    case.k_scale = case.v_scale = None
    cache, batch = case.handles(nb)
    v = torch.linspace(-600, 600, 3 * D).reshape(3, 1, D).bfloat16()
    v[0, 0, :8] = torch.tensor([17.0, 19.0, 0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, -1e30])
    k = (torch.randn(3, 1, D) * 2.0 ** -5).bfloat16()
    nb.kv_append(cache, batch, k.to(DEV), v.to(DEV))
    torch.cuda.synchronize()
    for i, j in enumerate(range(37, 40)):
        p, o = int(case.table[0, j // page]), j % page
        for got, src in ((case.kd, k), (case.vd, v)):
            want = src[i, 0].float().clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(got[p, o, 0].cpu().view(torch.uint8), want.view(torch.uint8))


def test_kv_append_bad_pages_and_positions_are_reported(nb):
    D, page = 64, 16
    reqs = [(2, 33), (3, 2), (1, 16), (2, 20)]
    case = Paged(reqs, 1, D, page, seed=8)
    cache, batch = case.handles(nb)
    before_k = case.kd.clone()
    batch.page_table[0, 2] = -1                       # the second token of request 0
    batch.page_table[2, 0] = case.k.shape[0]          # the token of request 2
    k = torch.randn(case.T, 1, D, device=DEV).bfloat16()
    qo = torch.full((case.T, 2, D), 7.0, device=DEV).bfloat16()
    q = torch.randn(case.T, 2, D, device=DEV).bfloat16()
    ws = nb.attn_workspace()
    nb.kv_append(cache, batch, k, k, q=q, q_out=qo, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    # request 1 has fewer cached tokens than new ones: its first has no position
    lost, kept = [1, 2, 5], [0, 3, 4, 6, 7]
    assert (qo[lost] == 7).all() and torch.equal(qo[kept], q[kept])
    where = {0: (0, 31), 3: (1, 0), 4: (1, 1), 6: (3, 18), 7: (3, 19)}
    want = before_k.cpu()
    for t, (r, j) in where.items():
        want[int(case.table[r, j // page]), j % page] = k[t].cpu()
    assert torch.equal(case.kd.cpu().view(torch.int16), want.view(torch.int16))


def test_append_then_attend_is_attention_of_the_whole_prompt(nb):
    """A prompt appended in three uneven chunks and attended chunk by chunk
    equals its attention in one piece."""
    D, hq, hk, page, n = 128, 8, 2, 16, 150
    g = torch.Generator().manual_seed(3)
    q, k, v = ((torch.randn(n, h, D, generator=g)).bfloat16().to(DEV) for h in (hq, hk, hk))
    rope = _table(n, D).to(DEV)
    w = (1 + torch.randn(D, generator=g) / 4).bfloat16().to(DEV)
    outs = []
    for cuts in ([0, n], [0, 101, 102, n]):
        case = Paged([(n, n)], hk, D, page, seed=13)
        cache, _ = case.handles(nb)
        parts = []
        for a, e in zip(cuts, cuts[1:]):
            batch = nb.AttnBatch(torch.tensor([0, e - a], dtype=torch.int32, device=DEV),
                                 torch.tensor([e], dtype=torch.int32, device=DEV),
                                 case.table.to(DEV), max_new=e - a)
            qr = nb.kv_append(cache, batch, k[a:e], v[a:e], rope=rope, k_weight=w, q=q[a:e], q_weight=w)
            parts.append(nb.paged_attention(qr, cache, batch))
        outs.append(torch.cat(parts).double().cpu())
        case.k, case.v = case.kd.cpu(), case.vd.cpu()
    qr, _ = nb.qk_norm_rope(q, k, torch.arange(n, dtype=torch.int32, device=DEV), rope, w, w)
    want, _, bound, _ = case.reference(qr.cpu())
    for o in outs:
        _within(o, want, bound, "prompt")


def _dense(q, k, v, pos, window):
    """Attention in 64 bits on the GPU, one request: q [n, Hq, D] at positions pos,
    k and v [L, Hkv, D] -> (out, lse, bounds) as tests/_attention_reference.py has them."""
    n, hq, D = q.shape
    g = hq // k.shape[1]
    scale = D ** -0.5
    j = torch.arange(k.shape[0], device=DEV)
    see = j <= pos[:, None]
    if window:
        see &= j > pos[:, None] - window
    outs = []
    for h in range(hq):
        x, kk, vv = q[:, h].double(), k[:, h // g].double(), v[:, h // g].double()
        s = (x @ kk.T * scale).masked_fill(~see, -math.inf)
        ds = (x.abs() @ kk.abs().T * scale).masked_fill(~see, 0).amax(1) * (D + 8) * 2.0 ** -23
        p = torch.softmax(s, 1)
        o, ev, ls = p @ vv, p @ vv.abs(), torch.logsumexp(s, 1)
        outs.append((o, ls, (ref.U + 2 * ds[:, None] + 2.0 ** -18) * ev + ref.U * o.abs(),
                     ds + 2.0 ** -18 * (1 + ls.abs())))
    return tuple(torch.stack(t, 1).cpu() for t in zip(*outs))


@pytest.mark.parametrize("n,prior,hq,hk,D,window", [
    (2000, 0, 32, 16, 128, 0), (1999, 1500, 24, 24, 64, 0), (3001, 500, 16, 8, 128, 300),
    (700, 9000, 56, 8, 128, 0), (4, 9000, 56, 8, 128, 0), (1, 20000, 64, 64, 64, 0),
    (1, 3000, 64, 64, 128, 0), (1, 40000, 56, 8, 128, 0), (2, 5000, 48, 3, 128, 1000)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_paged_attention_many_segments(nb, n, prior, hq, hk, D, window, fp8):
    """Enough work that every SM walks through several heads and row blocks;
    the same bits every time."""
    g = torch.Generator(device=DEV).manual_seed(n + hq)
    L, page = n + prior, 64
    pages = -(-L // page)
    k, v = (torch.randn(pages, page, hk, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = (torch.randn(n, hq, D, generator=g, device=DEV) * 1.5).bfloat16()
    table = torch.randperm(pages, generator=g, device=DEV).int()
    scales = torch.rand(2, hk, generator=g, device=DEV) * 0.02 + 0.01
    if fp8:
        k, v = ((x / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for x, sc in zip((k, v), scales))
        cache = nb.PagedKVCache(k, v, k_scale=scales[0], v_scale=scales[1])
        k, v = (x.double() * sc[:, None] for x, sc in zip((k, v), scales))
    else:
        cache = nb.PagedKVCache(k, v)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    batch = nb.AttnBatch(i32(0, n), i32(L), table[None], max_new=n)
    lse = torch.empty(n, hq, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    out = nb.paged_attention(q, cache, batch, window=window, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    flat = lambda t: t[table.long()].flatten(0, 1)[:L]   # noqa: E731
    want, wlse, b_out, b_lse = _dense(q, flat(k), flat(v), torch.arange(prior, L, device=DEV), window)
    _within(out, want, b_out, "out")
    _within(lse, wlse, b_lse, "lse")
    again = [nb.paged_attention(q, cache, batch, window=window, ws=ws) for _ in range(20)]
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    assert all(torch.equal(a, out) for a in again)


@pytest.mark.parametrize("n,prior,window", [(1600, 100, 0), (3100, 0, 200)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_paged_attention_many_blocks(nb, n, prior, window, fp8):
    """More row blocks than are planned in place."""
    test_paged_attention_many_segments(nb, n, prior, 32, 1, 64, window, fp8)
