"""What the serving operators promise about single weights and running sums, held apart
from the roundings that hide them elsewhere."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def nb():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_block_scaled_route_gb300 import binding
    return binding


# ------------------------------------------------- weights of single tokens --
def two_keys(nb, group, low, high, a, seed):
    """Attention over two keys that count, of which the first has weight 1 and value a_d in
    dimension d, the second, a tile later, a weight w spread over its logarithm between 2^low
    and 2^high and the value 1.  (out, w) in 64 bits, [B, heads, group, 128] and [.., 1].

    The other keys have scores of -200 and less: weights of 0.  512 requests of 4 key heads
    and two tiles each: most of them are not cut, so a row's reference is that of its first
    tile, score 0, when the second comes in."""
    B, H, D, page = 512, 4, 128, 128
    g = torch.Generator().manual_seed(seed)
    k = torch.zeros(2 * B, page, H, D)
    k[..., 1] = -256.0
    k[:, 0] = 0.0
    k[B:, 0, :, 0] = 1.0
    v = torch.zeros(2 * B, page, H, D)
    v[:B, 0] = a
    v[B:, 0] = 1.0
    ones = torch.ones(2 * B, H)
    # the score of the second key is q k_scale: any scale will do
    k_scale = ones.clone()
    k_scale[B:] = 1 + torch.rand(B, H, generator=g)
    y = low + (high - low) * torch.rand(B, H, group, generator=g)
    q = torch.zeros(B, H, group, D)
    q[..., 0] = y * float(np.log(2)) / k_scale[B:, :, None]
    q[..., 1] = 1.0
    q = q.bfloat16()
    w = torch.exp(q[..., :1].double() * k_scale[B:, :, None, None].double())
    cache = nb.PagedKVCache(k.to(torch.float8_e4m3fn).to(DEV), v.to(torch.float8_e4m3fn).to(DEV),
                            k_scale=k_scale.to(DEV), v_scale=ones.to(DEV))
    table = torch.stack([torch.arange(B), torch.arange(B, 2 * B)], 1).int().to(DEV)
    batch = nb.AttnBatch(torch.arange(B + 1, dtype=torch.int32, device=DEV),
                         torch.full((B,), 2 * page, dtype=torch.int32, device=DEV), table, max_new=1)
    out = nb.paged_attention(q.flatten(1, 2).to(DEV), cache, batch, scale=1.0)
    return out.double().cpu().unflatten(1, (H, group)), w


@pytest.mark.parametrize("group", [7, 8, 14, 16])
def test_weights_above_their_reference(nb, group):
    """Weights of up to 2^4 times the first are fp16 numbers, right to within 2^-11: values
    of the other sign take away what is common to both keys.  Of out = (a + w) / (1 + w) the
    first weight is exact, w is off by 2^-11 of itself and 2^-18 for the score, its
    exponential and the sums in 32 bits, the output by 2^-8."""
    a = torch.tensor([1.0, 1.5, 2.0, 3.0, 4.0, 4.5, 5.0, 5.5, 6.0, 6.5, 7.0, 7.5, 8.0, 9.0, 10.0, 11.0,
                      12.0, 13.0, 14.0, 15.0, 16.0]).repeat(7)[:128].neg()
    out, w = two_keys(nb, group, 0.0, 4.0, a, group)
    want = (a.double() + w) / (1 + w)
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 * w + 2.0 ** -18 * (a.double().abs() + w)) / (1 + w)
    assert ((out - want).abs() <= bound).all()


@pytest.mark.parametrize("group", [7, 14])
def test_weights_far_below_their_reference(nb, group):
    """Weights down to 2^-22 of the largest are right to within 2^-8, those below to within
    2^-31 of the largest; the output by 2^-8."""
    for low, high in ((-22.0, -2.0), (-34.0, -22.0)):
        out, w = two_keys(nb, group, low, high, torch.zeros(128), group)
        want = w / (1 + w)
        bound = 2.0 ** -7 * want + 2.0 ** -18 * want + torch.where(w < 2.0 ** -22, 2.0 ** -31, 0.0)
        assert ((out - want).abs() <= bound).all()


# --------------------------------------------------- sums of the vocabulary --
def numbers_away_from_borders(weights, count, runs, rng, margin):
    """fp32 numbers u for which the token is decided: u times the whole is `margin` of it or
    more away from the running sums on either side.  (u, tokens)."""
    upto = np.cumsum(weights.astype(np.longdouble))
    whole, V = upto[-1], len(weights)
    us, tokens = [], []
    while len(us) < count:
        # behind the large numbers at the front of a run
        at = rng.integers(0, runs) * (V // runs) + rng.integers(128, V // runs)
        u = np.float32(upto[at] / whole)
        x = np.longdouble(u) * whole
        i = int(np.searchsorted(upto, x, side="right"))
        if 0 < i < V and min(x - upto[i - 1], upto[i] - x) >= margin * whole:
            us.append(u)
            tokens.append(i)
    return torch.tensor(np.array(us)), tokens


@pytest.mark.parametrize("requests,runs,vocab", [(400, 8, 1 << 21), (400, 8, 1 << 20), (30, 64, 24 * 8192 - 64),
                                                 (30, 64, 1 << 21)])
@pytest.mark.parametrize("given", [False, True])
def test_running_sums_of_small_numbers_behind_large_ones(nb, given, requests, runs, vocab):
    """Running sums are off by 2^-38 of themselves at most, however many small numbers come
    behind large ones: 400 requests have a CTA each, and each of its threads adds up
    thousands of numbers (30: eight CTAs).  The whole and the running sum may both be off, so
    numbers that are 2^-37 away from the borders have to find their token."""
    if given and requests * vocab > 1 << 29:
        vocab >>= 1
    rng = np.random.default_rng(vocab)
    weights = np.full(vocab, 1.37 * 2.0 ** -34, np.float32)
    weights.reshape(runs, -1)[:, :128] = 0.91 * 2.0 ** -7 / runs
    rows, p, draft = requests, torch.from_numpy(weights), None
    q_start = torch.arange(requests + 1, dtype=torch.int32, device=DEV)
    if given:                                              # p - q, which 24 bits do not hold
        p, q = torch.from_numpy(weights * np.float32(1.7)), torch.from_numpy(weights * np.float32(0.31))
        p[5] = q[5] = 0.0                                  # the drafted token: never stands
        weights = p.double().numpy() - q.double().numpy()
        rows, q_start = 2 * requests, 2 * q_start
        draft = q.to(DEV).expand(rows, vocab).contiguous()
    u, want = numbers_away_from_borders(weights, requests, runs, rng, 2.0 ** -37)
    batch = nb.AttnBatch(q_start, torch.full((requests,), 9, dtype=torch.int32, device=DEV),
                         torch.zeros(requests, 1, dtype=torch.int32, device=DEV), max_new=2)
    target = p.to(DEV).expand(rows, vocab).contiguous()
    accepted, nxt = nb.draft_verify(target, draft, torch.full((rows,), 5, dtype=torch.int32, device=DEV), batch,
                                    torch.full((rows,), 0.5, device=DEV), u.to(DEV))
    assert accepted.tolist() == [0] * requests
    assert nxt.tolist() == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("requests,vocab", [(3, 300001), (320, 40003), (300, 600011)])
def test_long_rows_at_any_alignment(nb, requests, vocab, given, dtype):
    """Sums from blocks and from stretches of blocks, rows that begin anywhere, the draft's at
    another place of 16 bytes than the target's."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    drafts = 1 if requests > 9 else 4
    rows = requests * (drafts + 1)

    def distributions(pad):
        wide = torch.zeros(rows, vocab + 9, device=DEV, dtype=dtype)
        x = torch.randn(1, vocab, generator=g, device=DEV).expand(rows, vocab)
        row = torch.softmax(2 * x[:1] + torch.randn(1, vocab, generator=g, device=DEV), 1)
        wide[:, pad:pad + vocab] = row
        return wide[:, pad:pad + vocab]
    p, q = distributions(1), distributions(2) if given else None
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV, dtype=torch.int32)
    u, v = torch.rand(rows, generator=g, device=DEV), torch.rand(requests, generator=g, device=DEV)
    q_start = torch.arange(0, rows + 1, drafts + 1, dtype=torch.int32, device=DEV)
    batch = nb.AttnBatch(q_start, torch.full((requests,), 9, dtype=torch.int32, device=DEV),
                         torch.zeros(requests, 1, dtype=torch.int32, device=DEV), max_new=drafts + 1)
    accepted, nxt = nb.draft_verify(p, q, tokens, batch, u, v)
    # one row of probabilities for all: what is drawn from it, in 64 bits
    pd = p[0].double()
    weights = (pd - q[0].double()).clamp(min=0) if given else pd
    for r in range(requests):
        k = 0
        while k < drafts:
            x = int(tokens[r * (drafts + 1) + k + 1])
            if not float(u[r * (drafts + 1) + k]) * (float(q[0, x]) if given else 1.0) < float(p[0, x]):
                break
            k += 1
        w = pd if k == drafts else weights
        if k < drafts and not given:
            w = pd.clone()
            w[int(tokens[r * (drafts + 1) + k + 1])] = 0
        upto = w.cumsum(0)
        want = int(torch.searchsorted(upto, (float(v[r]) * upto[-1]).reshape(1), right=True))
        assert (int(accepted[r]), int(nxt[r])) == (k, want), r
