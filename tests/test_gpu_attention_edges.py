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
