"""The attention operators at the edges of their ranges: rounding into E4M3 pages,
weights far apart, values that are not finite, page ids, windows, token offsets and
streams.  Bounds as in tests/_attention_reference.py unless a test says otherwise."""
import math

import pytest
import torch

import _attention_reference as ref
from test_gpu_attention import BAD_INDEX, DEV, Paged, _within, nb  # noqa: F401

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ append --
def _appended(nb, x, scale):
    """Bytes of an E4M3 cache after x [T, H, D] went in as keys and as values, one
    request from position 0 on."""
    T, H, D = x.shape
    page = 16
    pages = -(-T // page)
    kc, vc = (torch.zeros(pages, page, H, D, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    sc = scale.to(DEV)
    cache = nb.PagedKVCache(kc, vc, k_scale=sc, v_scale=sc)
    batch = nb.AttnBatch(_i32(0, T), _i32(T), torch.arange(pages, dtype=torch.int32, device=DEV)[None],
                         max_new=T)
    ws = nb.attn_workspace()
    nb.kv_append(cache, batch, x.to(DEV), x.to(DEV), ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    return [c.view(torch.uint8).flatten(0, 1)[:T].cpu() for c in (kc, vc)]


@pytest.mark.parametrize("D", [64, 128])
def test_kv_append_divides_by_the_scale(nb, D):
    """The stored byte is that of the fp32 quotient, ties included: scales for which
    quotients fall on or beside the middle between two E4M3 numbers, where a product
    with the rounded reciprocal goes to the other side, and the ends of the range, where
    the reciprocal is infinite or subnormal."""
    ties = torch.arange(17, 32, 2).float()
    tops = torch.arange(128, 256).float()
    scale = torch.cat([(tops[:, None] / ties).flatten()[::23], torch.tensor(
        [7.0, 1e-39, 2.0 ** -149, 2.0 ** -128, 3e38, 1.0])])
    H = scale.numel()
    x = torch.cat([tops, -tops, tops * 2.0 ** -9, torch.zeros(64), 7 * ties,
                   torch.tensor([2.0 ** -126, -2.0 ** -126, 2.0 ** -133, 3e38, -3e38])])
    x = torch.nn.functional.pad(x, (0, -x.numel() % D)).view(-1, 1, D).expand(-1, H, D)
    x = x.bfloat16().contiguous()
    quotient = (x.float() / scale[:, None]).clamp(-448, 448)
    want = quotient.to(torch.float8_e4m3fn).view(torch.uint8)
    other = (x.float() * (1 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert (other.view(torch.uint8)[:, :-6] != want[:, :-6]).sum() > 9    # the cases are there
    for got in _appended(nb, x, scale):
        assert torch.equal(got, want)


# ----------------------------------------------------------------- weights --
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("nats", [12.0, 18.0])
@pytest.mark.parametrize("sink", [0, 300, 610])
def test_paged_attention_beside_a_dominant_key(nb, sink, nats, n, D, fp8):
    """One key far above the rest whose value is zero: the output is made of the small
    weights alone.  They lie within 2^-27 of the largest, where every weight is held to
    within 2^-8, so the usual bound holds."""
    L, page, hq = 650, 16, 8
    case = Paged([(n, L)], 1, D, page, fp8=fp8, seed=41)
    g = torch.Generator().manual_seed(7)
    step = 0.25 if fp8 else 1.0
    if fp8:
        case.k_scale, case.v_scale = torch.tensor([step]), torch.tensor([0.01])
    k = torch.randn(L, D, generator=g) * 0.04
    k[sink] = nats / (0.5 * D ** 0.5)
    v = torch.rand(L, D, generator=g) + 0.5
    v[sink] = 0.0
    for j in range(L):
        p, o = int(case.table[0, j // page]), j % page
        case.k[p, o, 0] = (k[j] / step).to(case.k.dtype)
        case.v[p, o, 0] = (v[j] / (0.01 if fp8 else 1.0)).to(case.v.dtype)
    q = torch.full((n, hq, D), 0.5).bfloat16()
    cache, batch = case.handles(nb)
    lse = torch.empty(n, hq, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    out = nb.paged_attention(q.to(DEV), cache, batch, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q)
    assert (want[-1] > 0).all() and want[-1].max() < 0.05
    _within(out, want, b_out, "out")
    _within(lse, wlse, b_lse, "lse")


@pytest.mark.parametrize("hq,D", [(8, 128), (4, 64)])
@pytest.mark.parametrize("n", [1, 40])
def test_paged_attention_large_scores_e4m3(nb, hq, D, n):
    """Scores far apart on an E4M3 cache.  A query element counts to within 2^-17 of its
    row's maximum (its score then to scale * 2^-17 max|q| sum|k|), and a weight is held
    to within 2^-8 down to 2^-27 of the largest and to within 2^-35 of that below."""
    case = Paged([(n, 700), (n, n)], 1, D, 32, seed=21, fp8=True)
    q = torch.randn(case.T, hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    q *= 40
    cache, batch = case.handles(nb)
    lse = torch.empty(case.T, hq, device=DEV)
    out = nb.paged_attention(q.to(DEV), cache, batch, lse=lse)
    want, wlse, b_out, b_lse = case.reference(q)
    k, v = (torch.cat([ref.key_rows(c, case.table[r], 32, length, 0, False, sc)
                       for r, (_, length) in enumerate(case.reqs)])
            for c, sc in ((case.k, case.k_scale), (case.v, case.v_scale)))
    extra = D ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * k.abs().sum(1).max()
    _within(out, want, b_out + 2 * extra[..., None] * v.abs().max() + 700 * 2.0 ** -35 * v.abs().max(),
            "out")
    _within(lse, wlse, b_lse + extra, "lse")


# ------------------------------------------------- values that are not finite --
def _timed(f):
    f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = math.inf
    for _ in range(3):
        start.record()
        f()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    return best


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,prior,hq,hk,D", [(1, 1024, 1200, 32, 4, 128), (4, 1000, 0, 8, 8, 64),
                                               (160, 2, 6000, 16, 2, 128)])
def test_paged_attention_visible_nan_costs_little(nb, B, n, prior, hq, hk, D, fp8):
    """A NaN in a value that every row sees makes that element NaN in every row and leaves
    the others as they were, bit for bit.  No row has to be done once more for it, so the
    call takes about as long as without it: at most twice the time and 0.2 ms."""
    L, page = n + prior, 64
    pages = -(-L // page)
    g = torch.Generator(device=DEV).manual_seed(n)
    k, v = (torch.randn(pages, page, hk, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    if fp8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    q = torch.randn(B * n, hq, D, generator=g, device=DEV).bfloat16()
    cache = nb.PagedKVCache(k, v)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    batch = nb.AttnBatch(n * torch.arange(B + 1, dtype=torch.int32, device=DEV), _i32(*[L] * B), table,
                         max_new=n)
    ws = nb.paged_attention_workspace(cache, batch, hq, B * n)
    out = torch.empty_like(q)

    def call():
        nb.paged_attention(q, cache, batch, out=out, ws=ws)
    clean_ms = _timed(call)
    clean = out.clone()
    at = v.view(torch.uint8)[0, 0, :, 9] if fp8 else v[0, 0, :, 9]
    at.fill_(0x7F if fp8 else math.nan)
    nan_ms = _timed(call)
    assert nb.read_status(ws) == 0
    assert out[..., 9].isnan().all()
    rest = [i for i in range(D) if i != 9]
    assert torch.equal(out[..., rest], clean[..., rest]) and clean.isfinite().all()
    assert nan_ms < 2 * clean_ms + 0.2, (clean_ms, nan_ms)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,hq,hk,D", [(4, 4, 1, 128), (70, 4, 2, 64), (150, 6, 1, 128)])
def test_paged_attention_visible_and_hidden_nan(nb, n, hq, hk, D, fp8):
    """The same element NaN in a key that all rows see and in one that some do not, and
    another element NaN only where some rows do not see it: each row's output is NaN just
    where a key that it sees is."""
    L = n + 200
    case = Paged([(n, L)], hk, D, 16, fp8=fp8, seed=51)
    nan = math.nan

    def put(j, d, value):
        p, o = int(case.table[0, j // 16]), j % 16
        x = case.v[p, o].float()
        x[:, d] = value
        case.v[p, o] = x.to(case.v.dtype)
    put(7, 3, nan)                       # everyone
    put(L - 1, 3, nan)                   # the last token alone sees this one,
    put(L - 1, 8, nan)                   # and this one
    put(L - 1 - n // 2, 20, nan)         # the later half
    q = torch.randn(n, hq, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    cache, batch = case.handles(nb)
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    for _ in range(2):
        out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, _, bound, _ = case.reference(q)
    got = out.double().cpu()
    fine = want.isfinite()
    assert not fine[..., 3].any() and fine[0, :, 8].all() and not fine[-1, :, 8].any()
    assert torch.equal(got.isfinite(), fine)
    over = (got - want).abs()[fine] - bound[fine]
    assert (over <= 0).all(), over.max()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [4, 60])
def test_paged_attention_bad_page_beside_a_hidden_nan(nb, n, fp8):
    """A page id out of range reads as zeros in rows that are done once more, too."""
    L, D, hq = 200, 128, 4
    case = Paged([(n, L)], 1, D, 16, fp8=fp8, seed=61)
    # (page 9, whose id is bad, lies in the same 128 keys)
    p, o = int(case.table[0, (L - 1) // 16]), (L - 1) % 16
    x = case.v[p, o].float()
    x[:, 5] = math.nan                   # the last token alone sees it
    case.v[p, o] = x.to(case.v.dtype)
    cache, batch = case.handles(nb)
    batch.page_table[0, 9] = case.k.shape[0] + 7
    q = torch.randn(n, hq, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    case.table[0, 9] = case.k.shape[0]

    def with_zeros(c):
        return torch.cat([c.view(torch.uint8), torch.zeros_like(c[:1].view(torch.uint8))]).view(c.dtype)
    case.k, case.v = with_zeros(case.k), with_zeros(case.v)
    want, _, bound, _ = case.reference(q)
    got = out.double().cpu()
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine) and fine[:-1].all()
    over = (got - want).abs()[fine] - bound[fine]
    assert (over <= 0).all(), over.max()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_paged_attention_hidden_nan_in_a_long_chunk(nb, D, fp8):
    """A NaN at the last key, which the last token alone sees: the other rows of its block
    are done once more, 16 by each warp.  They come out as without it, and in at most
    0.4 us a row and key (0.18 measured at full clock)."""
    n, prior, hq, hk, page = 1024, 4096, 56, 8, 64
    L = n + prior
    g = torch.Generator(device=DEV).manual_seed(D)
    k, v = (torch.randn(L // page, page, hk, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    if fp8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    q = torch.randn(n, hq, D, generator=g, device=DEV).bfloat16()
    cache = nb.PagedKVCache(k, v)
    batch = nb.AttnBatch(_i32(0, n), _i32(L),
                         torch.arange(L // page, dtype=torch.int32, device=DEV)[None], max_new=n)
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    out = torch.empty_like(q)

    def call():
        nb.paged_attention(q, cache, batch, out=out, ws=ws)
    clean_ms = _timed(call)
    clean = out.clone()
    (v.view(torch.uint8) if fp8 else v)[-1, -1, :, 9].fill_(0x7F if fp8 else math.nan)
    nan_ms = _timed(call)
    assert nb.read_status(ws) == 0
    assert out[-1, :, 9].isnan().all()
    rest = [i for i in range(D) if i != 9]
    assert torch.equal(out[:-128], clean[:-128]) and torch.equal(out[-1][:, rest], clean[-1][:, rest])
    # rows done once more have other roundings: two of bf16 and of 16-bit weights
    flat = lambda t: t.flatten(0, 1)[:L]                   # noqa: E731
    for h in (0, hq - 1):
        x = q[-128:-1, h].double()
        kk, vv = flat(k)[:, h // 7].double(), flat(v)[:, h // 7].double()
        s = (x @ kk.T * D ** -0.5).masked_fill(
            torch.arange(L, device=DEV) > torch.arange(L - 128, L - 1, device=DEV)[:, None], -math.inf)
        p = torch.softmax(s, 1)[:, :-1]
        want, ev = p @ vv[:-1], p @ vv[:-1].abs()
        ds = (x.abs() @ kk.abs().T * D ** -0.5).amax(1, True) * (D + 8) * 2.0 ** -23
        extra = D ** -0.5 * 2.0 ** -17 * x.abs().amax(1, True) * kk.abs().sum(1).max() if fp8 else 0.0
        over = (out[-128:-1, h].double() - want).abs() - (
            (ref.U + 2 * (ds + extra) + 2.0 ** -18) * ev + ref.U * want.abs())
        assert (over <= 0).all(), over.max()
    assert nan_ms < 2 * clean_ms + 16 * L * 0.4e-3, (clean_ms, nan_ms)


# ----------------------------------------------------------------- streams --
def test_buffers_made_in_a_call_belong_to_its_stream(nb, monkeypatch):
    """Calls with stream= and no workspace or outputs make and zero them on that stream:
    nothing of theirs waits in, or returns to, the current one, which is busy meanwhile."""
    made = []

    def spy(name):
        real = getattr(torch, name)

        def f(*a, **kw):
            t = real(*a, **kw)
            if t.is_cuda:
                made.append((name, torch.cuda.current_stream().cuda_stream))
            return t
        return f
    case = Paged([(5, 200), (3, 3), (64, 300)], 2, 128, 16, seed=2)
    T, hq, D = case.T, 8, 128
    q = torch.randn(T, hq, D, device=DEV).bfloat16()
    k = torch.randn(T, 2, D, device=DEV).bfloat16()
    x = torch.randn(T, 256, device=DEV).bfloat16()
    w = torch.randn(16, 256, device=DEV).bfloat16()
    h = torch.randn(4, 256, 128, device=DEV)
    cache, batch = case.handles(nb)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)

    def calls(**kw):
        ids, wts = nb.router_topk(x, w, 2, **kw)
        route = nb.route_permute(ids, 16, **kw)
        got = [nb.paged_attention(q, cache, batch, **kw), *nb.qk_norm_rope(q, k, pos, None, **kw),
               nb.kv_append(cache, batch, k, k, q=q, **kw), ids, wts, route.slot_of,
               *nb.quantize_act(x, **kw)[:2], nb.amax(x, **kw), *nb.quantize_weights(h, **kw)]
        return got + [nb.paged_attention(q, cache, batch, **kw)]
    s = torch.cuda.Stream()
    calls()
    # (what the first calls appended is there from now on)
    want = calls()
    torch.cuda.synchronize()
    calls(stream=s)                                  # its pool has memory from here on
    torch.cuda.synchronize()
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, spy(name))
    busy = torch.cuda.Event()
    torch.cuda._sleep(600_000_000)                   # some 0.3 s of the current stream
    busy.record()
    got = calls(stream=s)
    s.synchronize()
    assert not busy.query(), "the current stream was not busy"
    monkeypatch.undo()
    assert len(made) > 20 and all(stream == s.cuda_stream for _, stream in made), made
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------- windows and offsets --
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("reqs", [[(8, 2), (7, 0), (1, 90), (9, 3)], [(60, 40), (150, 400), (30, 5)]],
                         ids=["few", "chunk"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20])
def test_paged_attention_window_without_end(nb, reqs, window, fp8):
    """A window of almost 2^31 positions is no window, also for tokens whose position is
    negative."""
    case = Paged(reqs, 1, 64, 16, fp8=fp8, seed=71)
    q = torch.randn(case.T, 1, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    cache, batch = case.handles(nb)
    lse = torch.full((case.T, 1), 5.0, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, 1, case.T)
    out = nb.paged_attention(q.to(DEV), cache, batch, window=window, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q)
    _within(out, want, b_out, "out")
    _within(lse, wlse, b_lse, "lse")


@pytest.mark.parametrize("n", [3, 60])
@pytest.mark.parametrize("cut", ["end", "begin"])
def test_paged_attention_token_offsets_outside_the_rows(nb, n, cut):
    """A request whose token offsets reach past the rows of q is reported, and the rows
    that are there keep their positions: those at which its keys were appended."""
    L, D, hq, beyond = 200, 128, 4, 2
    case = Paged([(n, L)], 1, D, 16, seed=81)
    q = torch.randn(n, hq, D, generator=torch.Generator().manual_seed(5)).bfloat16()
    cache, batch = case.handles(nb)
    batch.q_start.copy_(_i32(0, n + beyond) if cut == "end" else _i32(-beyond, n))
    batch = nb.AttnBatch(batch.q_start, batch.kv_len, batch.page_table, max_new=n + beyond)
    ws = nb.paged_attention_workspace(cache, batch, hq, n)
    out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    pad = torch.zeros(beyond, hq, D).bfloat16()
    case.q_start = torch.tensor([0, n + beyond])
    want, _, bound, _ = case.reference(torch.cat([q, pad] if cut == "end" else [pad, q]))
    rows = slice(0, n) if cut == "end" else slice(beyond, n + beyond)
    _within(out, want[rows], bound[rows], "rows")


@pytest.mark.parametrize("m", [1, 30])
def test_paged_attention_token_offsets_that_descend(nb, m):
    """Offsets that do not ascend are reported; requests whose own do are computed."""
    D, page = 64, 16
    case = Paged([(3 * m, 3 * m + 40), (1, 40), (2 * m, 2 * m + 20)], 1, D, page, seed=82)
    cache, batch = case.handles(nb)
    batch.q_start.copy_(_i32(0, 3 * m, 2 * m, 4 * m))
    q = torch.randn(4 * m, 2, D, generator=torch.Generator().manual_seed(7)).bfloat16()
    ws = nb.paged_attention_workspace(cache, batch, 2, 4 * m)
    out = nb.paged_attention(q.to(DEV), cache, batch, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == BAD_INDEX
    # rows of two requests hold either's; the others their own
    for r, rows in ((0, slice(0, 2 * m)), (2, slice(3 * m, 4 * m))):
        first, n = (0, 3 * m) if r == 0 else (2 * m, 2 * m)
        want, _, bound, _ = ref.attention(q[first:first + n], case.k, case.v, [0, n],
                                          [case.reqs[r][1]], case.table[r:r + 1])
        mine = slice(rows.start - first, rows.stop - first)
        _within(out[rows], want[mine], bound[mine], f"request {r}")


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_paged_attention_e4m3_scores_that_vanish(nb, n, D):
    """Scales and queries so small that the factor of the scores is below the smallest
    fp32 number: all scores are zero, hidden keys still count for nothing."""
    case = Paged([(n, n + 70)], 1, D, 16, fp8=True, seed=91)
    case.k_scale = torch.tensor([1e-30])
    q = (torch.randn(n, 4, D, generator=torch.Generator().manual_seed(6)) * 1e-25).bfloat16()
    cache, batch = case.handles(nb)
    lse = torch.empty(n, 4, device=DEV)
    ws = nb.paged_attention_workspace(cache, batch, 4, n)
    out = nb.paged_attention(q.to(DEV), cache, batch, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == 0
    want, wlse, b_out, b_lse = case.reference(q)
    _within(out, want, b_out, "out")
    _within(lse, wlse, b_lse, "lse")
