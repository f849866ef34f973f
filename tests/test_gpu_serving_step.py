"""Planning of a serving step and verification of drafted tokens (64-bit forms in
tests/_serving_reference.py), and the operators of a step together."""
import random

import pytest
import torch

import _serving_reference as sref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD_INDEX, RANGE = 7, 8


@pytest.fixture(scope="module")
def nb():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_block_scaled_route_gb300 import binding
    return binding


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


# ------------------------------------------------------------------- plan --
class Requests:
    """Lengths, tables and a pool as a server has them, on the host."""

    def __init__(self, rng, B, page, max_pages, spare, top):
        self.page, self.max_pages = page, max_pages
        self.before = [rng.choice([0, rng.randint(0, top)]) for _ in range(B)]
        held = [-(-n // page) for n in self.before]
        pages = list(range(sum(held) + spare))
        rng.shuffle(pages)
        self.table = [[-1] * max_pages for _ in range(B)]
        at = 0
        for r, n in enumerate(held):
            self.table[r][:n] = pages[at:at + n]
            at += n
        free, size = pages[at:], max(1, len(pages))
        first = rng.randrange(size)
        self.ring = [-9] * size
        for i, p in enumerate(free):
            self.ring[(first + i) % size] = p
        self.state = [first, len(free)]


def run_plan(nb, s, new, cached=None, rows=None, in_place=False, outputs=True, stream=None):
    """attn_plan_pages on copies of s, against the host's; returns what it left."""
    B = len(new)
    # (rows count for every request of the step, taken up or not)
    rows = min(sum(max(n, 0) for n in new) + 3, 1 << 20) if rows is None else rows
    want = sref.plan(s.ring, s.state, s.before, cached, new, s.table, s.page, rows if outputs else 2 ** 31 - 1)
    total = want[1][-1]
    table = ints(s.table).view(B, s.max_pages)
    pool = nb.PagePool(ints(s.ring), ints(s.state))
    before = ints(s.before)
    batch = nb.AttnBatch(torch.full((B + 1,), -5, dtype=torch.int32, device=DEV),
                         before if in_place else torch.full((B,), -5, dtype=torch.int32, device=DEV), table, max_new=1)
    out = None if in_place else ints([-5, -5])
    pos = torch.full((rows,), -5, dtype=torch.int32, device=DEV) if outputs else None
    slots = torch.full((rows,), -5, dtype=torch.int64, device=DEV) if outputs else None
    ws = nb.attn_workspace()
    nb.plan_pages(pool, batch, s.page, ints(new), cached=None if cached is None else ints(cached),
                  kv_before=None if in_place else before, state_out=out, positions=pos, slots=slots, ws=ws,
                  stream=stream)
    torch.cuda.synchronize()
    kv_len, q_start, tab, positions, slot, ring, state, faults = want
    got = nb.read_status(ws)
    assert (got in faults) if faults else got == 0
    assert batch.kv_len.tolist() == kv_len and batch.q_start.tolist() == q_start
    assert table.tolist() == tab and pool.ring.tolist() == ring
    assert (pool.state if in_place else out).tolist() == state
    if outputs:
        assert pos.tolist() == positions + [-5] * (rows - total)
        assert slots.tolist() == slot + [-5] * (rows - total)
    return want


@pytest.mark.parametrize("B,page,top,most", [(1, 16, 40, 5), (3, 16, 100, 40), (7, 64, 300, 130), (40, 16, 500, 9),
                                             (300, 32, 200, 60), (1500, 16, 60, 3), (2100, 128, 300, 40),
                                             (2, 1024, 5000, 9000), (1, 16, 20000, 30000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(nb, B, page, top, most, in_place):
    """Requests that grow, stay, shrink and end; tokens turned down; enough pages."""
    rng = random.Random(B + page)
    for _ in range(3):
        s = Requests(rng, B, page, -(-(top + most) // page), B * (most // page + 2), top)
        new = [rng.choice([-1, 0, 1, rng.randint(0, most), most]) for _ in range(B)]
        cached = [rng.choice([n, max(0, n - rng.randint(0, 2 * page)), 0]) for n in s.before]
        run_plan(nb, s, new, rng.choice([None, cached]), in_place=in_place)
        run_plan(nb, s, new, cached, in_place=in_place, outputs=False)


@pytest.mark.parametrize("B", [5, 60, 1300])
def test_plan_without_enough_pages_or_rows(nb, B):
    """Requests past the last page or row bring nothing; what they had stays, and others
    that need none go on."""
    rng = random.Random(B)
    for spare in (0, 1, B // 2, B):
        s = Requests(rng, B, 16, 8, spare, 60)
        new = [rng.choice([-1, 0, 1, rng.randint(1, 60)]) for _ in range(B)]
        cached = [max(0, n - rng.randint(0, 20)) for n in s.before]
        want = run_plan(nb, s, new, cached)
        assert want[6][1] >= 0
        for rows in (0, 1, want[1][-1] // 2):
            run_plan(nb, s, new, cached, rows=rows)


def test_plan_of_bad_lengths(nb):
    """Lengths below 0, past the table or shorter than what stands: those requests are left
    as they are."""
    s = Requests(random.Random(1), 7, 16, 4, 20, 40)
    s.before = [-3, 65, 20, 20, 60, 2 ** 31 - 1, 5]
    run_plan(nb, s, [1, 1, 1, 45, 1, 1, 2], [0, 60, 21, 20, 60, 3, 5])
    run_plan(nb, s, [-1, -1, -1, -1, 5, -1, 2 ** 31 - 1], None)
    run_plan(nb, s, [1] * 7, [0, 0, -1, 20, 60, -2 ** 31, 5])


def test_plan_of_a_bad_pool(nb):
    for state in ([-1, 3], [9, 3], [0, 10], [0, -1]):
        s = Requests(random.Random(2), 3, 16, 4, 9, 0)
        s.before, s.state = [0, 0, 0], state
        assert len(s.ring) == 9
        run_plan(nb, s, [1, 0, 20])
    # pages given back to a ring that has no room for them
    s = Requests(random.Random(3), 4, 16, 4, 2, 60)
    s.before = [60, 60, 60, 60]
    s.table = [[4 * r + i for i in range(4)] for r in range(4)]
    s.ring, s.state = list(range(100, 107)), [3, 4]
    want = run_plan(nb, s, [-1, 1, -1, 0])
    assert want[6] == [3, 7] and want[7] == {BAD_INDEX}


@pytest.mark.parametrize("state", [[-1, 3], [9, 3], [0, 10], [0, -1]])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,rows", [(5, 40), (1200, 4000)])
def test_plan_on_a_bad_pool_leaves_it_as_it_is(nb, state, in_place, B, rows):
    """Pages given back have no place to go: the ring stays, and a pool planned in place
    says the same the next time."""
    pool, out = nb.PagePool(ints(range(100, 109)), ints(state)), ints([-5, -5])
    before, table = ints([40] * B), ints([[3 * r, 3 * r + 1, 3 * r + 2, -1] for r in range(B)])
    new = [-1, 1, 5, -1, 9] * (B // 5)
    batch = nb.AttnBatch(ints([-5] * (B + 1)), ints([-5] * B), table, max_new=9)
    pos, slots = ints([-5] * rows), ints([-5] * rows, torch.int64)
    for _ in range(2):
        ws = nb.attn_workspace()
        nb.plan_pages(pool, batch, 16, ints(new), kv_before=before, state_out=None if in_place else out, positions=pos,
                      slots=slots, ws=ws)
        assert nb.read_status(ws) in (BAD_INDEX, RANGE)
        assert pool.ring.tolist() == list(range(100, 109)) and pool.state.tolist() == state
        assert in_place or out.tolist() == [0, 0]
        # 41 and 45 tokens fit the pages that are there, 49 do not
        assert batch.kv_len.tolist() == [0, 41, 45, 0, 40] * (B // 5)
        assert int(batch.q_start[-1]) == 6 * (B // 5)
        assert slots[:6].tolist() == [3 * 16 + 40] + [6 * 16 + i for i in range(40, 45)] and pos[0] == 40
        assert slots[6 * (B // 5):].eq(-5).all()


def test_plan_of_nothing(nb):
    s = Requests(random.Random(4), 0, 16, 4, 3, 0)
    pool = nb.PagePool(ints(s.ring), ints(s.state))
    batch = nb.AttnBatch(ints([7]), ints([]), torch.zeros(0, 4, dtype=torch.int32, device=DEV), max_new=1)
    nb.plan_pages(pool, batch, 16, ints([]))
    assert batch.q_start.tolist() == [0] and pool.state.tolist() == s.state
    run_plan(nb, Requests(random.Random(4), 3, 16, 4, 3, 0), [0, 0, 0])


def test_steps_keep_every_page_once(nb):
    """A thousand requests over thirty steps, in place, from a graph: after each, the pool
    and the requests hold every page exactly once, and the lengths are the host's."""
    rng = random.Random(9)
    B, page, pages, max_pages = 1100, 16, 14000, 12
    pool = nb.PagePool(ints(rng.sample(range(pages), pages)), ints([17, pages]))
    batch = nb.AttnBatch(ints([0] * (B + 1)), ints([0] * B), ints([[0] * max_pages] * B), max_new=32)
    new, cached, ws = ints([0] * B), ints([0] * B), nb.attn_workspace()
    pos, slots = ints([0] * 40 * B), ints([0] * 40 * B, torch.int64)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nb.plan_pages(pool, batch, page, new, cached=cached, positions=pos, slots=slots, ws=ws)
    length = [0] * B
    for _ in range(30):
        stand = [max(0, n - rng.choice([0, 0, 3])) for n in length]
        add = [-1 if n > 100 and rng.random() < 0.3 else min(rng.randint(0, 32), page * max_pages - c)
               for n, c in zip(length, stand)]
        new.copy_(ints(add))
        cached.copy_(ints(stand))
        graph.replay()
        length = [0 if n < 0 else c + n for c, n in zip(stand, add)]
        assert batch.kv_len.tolist() == length and nb.read_status(ws) == 0
        table, (first, free), ring = batch.page_table.tolist(), pool.state.tolist(), pool.ring.tolist()
        held = [p for r, n in enumerate(length) for p in table[r][:-(-n // page)]]
        assert sorted(held + [ring[(first + i) % pages] for i in range(free)]) == list(range(pages))
        n = sum(max(0, x) for x in add)
        want = [table[r][p // page] * page + p % page for r, x in enumerate(add)
                for p in range(length[r] - max(0, x), length[r])]
        assert slots[:n].tolist() == want and len(set(want)) == n


def test_plan_on_another_stream(nb):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = Requests(random.Random(5), 30, 16, 9, 100, 100)
    run_plan(nb, s, [3] * 30, stream=side)


# ----------------------------------------------------------------- verify --
def drafted(g, counts, vocab, sharp=3.0, off=0.3, dtype=torch.float32):
    """Distributions and tokens for requests of counts[r] drafted tokens (-1: no rows)."""
    q_start = torch.tensor([0] + [n + 1 for n in counts]).cumsum(0)
    T = int(q_start[-1])
    p = torch.softmax(torch.randn(T, vocab, generator=g) * sharp, 1)
    q = p * (1 - off) + off * torch.softmax(torch.randn(T, vocab, generator=g) * sharp, 1)
    tokens = torch.zeros(T, dtype=torch.int32)
    if T > 1:
        tokens[1:] = torch.multinomial(q, 1, generator=g)[:-1, 0].int()
    return (p.to(dtype), q.to(dtype), tokens, q_start.int(), torch.rand(T, generator=g),
            torch.rand(len(counts), generator=g))


def run_verify(nb, p, q, tokens, q_start, u, v, status=0, stream=None, pad=0):
    B = len(q_start) - 1

    def put(t):
        if t is None or not pad:
            return None if t is None else t.to(DEV)
        wide = torch.full((t.shape[0], t.shape[1] + pad), 0.7, dtype=t.dtype, device=DEV)
        wide[:, pad // 2:pad // 2 + t.shape[1]] = t.to(DEV)
        return wide[:, pad // 2:pad // 2 + t.shape[1]]     # a view: strides and alignment of its own
    kv_len = torch.arange(100, 100 + B, dtype=torch.int32, device=DEV)
    batch = nb.AttnBatch(q_start.to(DEV), kv_len, torch.zeros(B, 1, dtype=torch.int32, device=DEV), max_new=9)
    cached, ws = ints([-5] * B), nb.attn_workspace()
    accepted, nxt = nb.draft_verify(put(p), put(q), tokens.to(DEV), batch, u.to(DEV), v.to(DEV), cached=cached, ws=ws,
                                    stream=stream)
    torch.cuda.synchronize()
    assert nb.read_status(ws) == status
    want = sref.verify(p, q, tokens, q_start, u, v)
    assert accepted.tolist() == want[0]
    assert nxt.tolist() == want[1]
    drafts = (q_start[1:] - q_start[:-1] - 1).clamp(min=0).tolist()
    assert cached.tolist() == [100 + r - (n - k) for r, (n, k) in enumerate(zip(drafts, want[0]))]
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,vocab,pad", [
    ([0], 1, 0), ([1, 0, 3], 2, 0), ([4], 5, 0), ([2, -1, 0, 7], 37, 0), ([5] * 9, 1000, 3), ([3, 40, 1], 333, 1),
    ([1] * 30, 4099, 0), ([4, 2, 5], 32003, 0), ([4, 2, 5], 32003, 5), ([5, 5, 1, 0], 129280, 0), ([2, 3], 262145, 7)])
@pytest.mark.parametrize("given", [True, False])
def test_verify(nb, counts, vocab, pad, dtype, given):
    g = torch.Generator().manual_seed(vocab + pad)
    for off in (0.05, 0.6):
        p, q, *rest = drafted(g, counts, vocab, off=off, dtype=dtype)
        run_verify(nb, p, q if given else None, *rest, pad=pad)


@pytest.mark.parametrize("requests", [19, 40, 72, 90, 110, 140, 180, 290, 350])
def test_verify_shares_of_any_number_of_blocks(nb, requests):
    """Blocks of a request: 1 to 8, by how many requests fit the GPU at once."""
    g = torch.Generator().manual_seed(requests)
    p, q, *rest = drafted(g, [2] * requests, 59999, off=0.8)
    run_verify(nb, p, q, *rest)


def test_verify_rows_that_differ_in_alignment(nb):
    g = torch.Generator().manual_seed(3)
    p, q, tokens, q_start, u, v = drafted(g, [3, 2, 4], 5001)
    wide = torch.zeros(12, 5008, device=DEV)
    wide[:, 1:5002] = q.to(DEV)
    batch = nb.AttnBatch(q_start.to(DEV), ints([9] * 3), torch.zeros(3, 1, dtype=torch.int32, device=DEV), max_new=9)
    got = nb.draft_verify(p.to(DEV), wide[:, 1:5002], tokens.to(DEV), batch, u.to(DEV), v.to(DEV))
    assert [x.tolist() for x in got] == list(sref.verify(p, q, tokens, q_start, u, v))


def test_verify_over_the_numbers(nb):
    """Every way through: 600 requests a row each, flat distributions whose running sums
    pass the number anywhere along the row."""
    g = torch.Generator().manual_seed(8)
    p, q, *rest = drafted(g, [1] * 600, 20011, sharp=0.5)
    accepted, nxt = run_verify(nb, p, q, *rest)
    assert 100 < sum(accepted) < 590
    assert min(nxt) < 200 and max(nxt) > 19800


def test_verify_numbers_at_their_ends_and_at_borders(nb):
    """Sums that are exact: a number at a border takes the next token, one past the end
    the last that has any probability, one below 0 and NaN the first."""
    p = torch.tensor([0.0, 0.25, 0.0, 0.25, 0.25, 0.25, 0.0, 0.0]).repeat(9, 1)
    v = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.9999999, 1.0, 3.0, -1.0, float("nan")])
    tokens, q_start = torch.zeros(9, dtype=torch.int32), torch.arange(10, dtype=torch.int32)
    _, nxt = run_verify(nb, p, None, tokens, q_start, torch.zeros(9), v)
    assert nxt == [1, 3, 4, 5, 5, 5, 5, 1, 1]
    # a drafted token stands while u q < p, not at u q = p; NaN as a number never
    p = torch.tensor([[0.25, 0.75]]).repeat(8, 1)
    q = torch.tensor([[0.5, 0.5]]).repeat(8, 1)
    tokens, q_start = torch.zeros(8, dtype=torch.int32), torch.arange(0, 10, 2, dtype=torch.int32)
    u = torch.tensor([0.5, 0, 0.49999997, 0, 0.0, 0, float("nan"), 0])
    accepted, nxt = run_verify(nb, p, q, tokens, q_start, u, torch.tensor([0.1, 0.1, 0.3, 0.0]))
    assert accepted == [0, 1, 1, 0] and nxt == [1, 0, 1, 1]


def test_verify_small_remainders(nb):
    """p and q that differ in their last bits alone, and remainders of one token."""
    V = 3001
    base = torch.rand(1, V, generator=torch.Generator().manual_seed(1)) / V
    p, q = base.repeat(40, 1), base.repeat(40, 1)
    g = torch.Generator().manual_seed(2)
    bump = torch.rand(40, V, generator=g) < 0.01
    p = torch.where(bump, torch.nextafter(p, torch.tensor(1.0)), p)
    p[::2, 7] = 0.0                                        # the drafted token: always turned down
    tokens = torch.full((40,), 7, dtype=torch.int32)
    q_start = torch.arange(0, 42, 2, dtype=torch.int32)
    accepted, _ = run_verify(nb, p, q, tokens, q_start, torch.rand(40, generator=g), torch.rand(20, generator=g))
    assert sum(accepted) == 0
    p = torch.zeros(2, V)
    p[0, 2999] = 2.0 ** -100
    run_verify(nb, p, torch.rand(2, V), tokens[:2], q_start[:2], torch.tensor([0.5, 0.5]), torch.tensor([0.99]))


def test_verify_of_rows_that_are_no_distributions(nb):
    """NaN, infinities, negative numbers and numbers above 1; a remainder of nothing takes
    the target's row; a row of nothing gives no token, and says so."""
    V = 40
    g = torch.Generator().manual_seed(5)
    p, q = torch.rand(12, V, generator=g), torch.rand(12, V, generator=g)
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.5, 7.0, 0.0])
    p[:, 3:33:5] = odd
    q[:, 5:35:5] = odd
    tokens = torch.randint(0, V, (12,), generator=g, dtype=torch.int32)
    q_start = torch.arange(0, 14, 2, dtype=torch.int32)
    run_verify(nb, p, q, tokens, q_start, torch.rand(12, generator=g), torch.rand(6, generator=g))
    run_verify(nb, p, None, tokens, q_start, torch.rand(12, generator=g), torch.rand(6, generator=g))
    p = torch.full((4, V), 0.02)
    q = torch.full((4, V), 0.9)
    accepted, _ = run_verify(nb, p, q, tokens[:4], q_start[:3], torch.full((4,), 0.9), torch.tensor([0.3, 0.8]))
    assert accepted == [0, 0]
    p[2:] = 0.0
    _, nxt = run_verify(nb, p, q, tokens[:4], q_start[:3], torch.full((4,), 0.9), torch.tensor([0.3, 0.8]),
                        status=RANGE)
    assert nxt[1] == -1 and nxt[0] >= 0
    p[2:, 3] = 1.0                                         # guessed for sure, and nothing else there: p itself
    run_verify(nb, p, None, torch.full((4,), 3, dtype=torch.int32), q_start[:3], torch.full((4,), 1.0),
               torch.tensor([0.3, 0.8]))


def test_verify_of_bad_tokens_and_offsets(nb):
    g = torch.Generator().manual_seed(6)
    p, q, tokens, q_start, u, v = drafted(g, [3, 2, 2], 50)
    tokens[2], tokens[5], tokens[9] = 50, -1, 2 ** 31 - 1
    run_verify(nb, p, q, tokens, q_start, u * 0, v, status=BAD_INDEX)
    run_verify(nb, p, None, tokens, q_start, u * 0, v, status=BAD_INDEX)
    for bad in ([-1, 4, 7, 10], [0, 4, 2, 10], [0, 4, 7, 11]):
        batch = nb.AttnBatch(ints(bad), ints([9] * 3), torch.zeros(3, 1, dtype=torch.int32, device=DEV), max_new=9)
        ws = nb.attn_workspace()
        accepted, nxt = nb.draft_verify(p.to(DEV), q.to(DEV), torch.zeros(10, dtype=torch.int32, device=DEV), batch,
                                        u.to(DEV), v.to(DEV), ws=ws)
        torch.cuda.synchronize()
        assert nb.read_status(ws) == BAD_INDEX
        for r in range(3):
            wrong = bad[r] < 0 or bad[r + 1] < bad[r] or bad[r + 1] > 10
            assert (int(nxt[r]) == -1) == wrong and (not wrong or int(accepted[r]) == 0)


def test_verified_tokens_have_the_targets_distribution(nb):
    """2^17 requests with one drafted token each from q: the first token that comes out
    (the drafted one where it stands) has the distribution p.  A count of N p tokens has
    the standard deviation sqrt(N p (1 - p)); six of them are allowed, each token."""
    N, V = 1 << 17, 8
    g = torch.Generator(device=DEV).manual_seed(11)
    p = torch.tensor([0.3, 0.01, 0.2, 0.0, 0.09, 0.25, 0.05, 0.1], device=DEV)
    q = torch.tensor([0.1, 0.2, 0.2, 0.1, 0.05, 0.05, 0.2, 0.1], device=DEV)
    x = torch.multinomial(q, N, replacement=True, generator=g).int()
    tokens = torch.zeros(2 * N, dtype=torch.int32, device=DEV)
    tokens[1::2] = x
    batch = nb.AttnBatch(torch.arange(0, 2 * N + 1, 2, dtype=torch.int32, device=DEV), ints([9] * N),
                         torch.zeros(N, 1, dtype=torch.int32, device=DEV), max_new=2)
    accepted, nxt = nb.draft_verify(p.repeat(2 * N, 1), q.repeat(2 * N, 1), tokens, batch,
                                    torch.rand(2 * N, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV))
    first = torch.where(accepted == 1, x, nxt)
    count = torch.bincount(first.long(), minlength=V).double()
    want = p.double() / p.double().sum()
    assert ((count - N * want).abs() <= 6 * (N * want * (1 - want)).sqrt()).all()
    # and the token behind one that stands has it too
    behind = nxt[accepted == 1]
    n = len(behind)
    count = torch.bincount(behind.long(), minlength=V).double()
    assert ((count - n * want).abs() <= 6 * (n * want * (1 - want)).sqrt()).all()


def test_verify_from_a_graph_and_on_another_stream(nb):
    g = torch.Generator().manual_seed(12)
    p, q, tokens, q_start, u, v = drafted(g, [4] * 20, 7001)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run_verify(nb, p, q, tokens, q_start, u, v, stream=side)
    args = [t.to(DEV) for t in (p, q, tokens, u, v)]
    batch = nb.AttnBatch(q_start.to(DEV), ints([9] * 20), torch.zeros(20, 1, dtype=torch.int32, device=DEV), max_new=5)
    ws, accepted, nxt = nb.attn_workspace(), ints([0] * 20), ints([0] * 20)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nb.draft_verify(args[0], args[1], args[2], batch, args[3], args[4], accepted=accepted, next_token=nxt, ws=ws)
    for seed in (13, 14):
        p, q, tokens, q_start, u, v = drafted(torch.Generator().manual_seed(seed), [4] * 20, 7001)
        for t, x in zip(args, (p, q, tokens, u, v)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = sref.verify(p, q, tokens, q_start, u, v)
        assert accepted.tolist() == want[0] and nxt.tolist() == want[1]


def test_verify_rows_past_32_bit_offsets(nb):
    """Rows of 2^18 tokens past element 2^31."""
    V, rows = 1 << 18, 8300
    p = torch.zeros(rows, V, dtype=torch.bfloat16, device=DEV)
    p[rows - 3:, 5], p[rows - 3:, V - 9] = 0.25, 0.75
    tokens = torch.full((rows,), 5, dtype=torch.int32, device=DEV)
    batch = nb.AttnBatch(ints([rows - 3, rows]), ints([50]), torch.zeros(1, 1, dtype=torch.int32, device=DEV), max_new=3)
    u = torch.full((rows,), 0.9, device=DEV)
    u[rows - 3] = 0.2
    accepted, nxt = nb.draft_verify(p, p, tokens, batch, u * 0.99, ints([0], torch.float32) + 0.3)
    assert accepted.tolist() == [2] and nxt.tolist() == [V - 9]
    accepted, nxt = nb.draft_verify(p, None, tokens, batch, u, ints([0], torch.float32) + 0.3)
    assert accepted.tolist() == [1] and nxt.tolist() == [V - 9]


# --------------------------------------------------------------- together --
@pytest.fixture(scope="module")
def ex():
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import decoder_block
    return decoder_block


@pytest.mark.parametrize("page_scales", [False, True], ids=["bf16", "page-scales"])
def test_drafted_steps_from_a_graph(nb, ex, monkeypatch, page_scales):
    """Steps of three drafted tokens from a graph: each step's answer is that of its own
    numbers, the lengths go on from the tokens that stand, every page is held once, and the
    attention of the last step is that of what the cache holds."""
    from _serving_reference import request_attention, verify
    seen = {}
    inner = nb.paged_attention

    def recorded(q, cache, batch, **kw):
        seen["q"], seen["out"] = q, inner(q, cache, batch, **kw)
        return seen["out"]
    monkeypatch.setattr(nb, "paged_attention", recorded)
    torch.manual_seed(3)
    R, n, prompt = 3, 3, 37
    block = ex.DecoderBlock(hidden=512, q_heads=4, inter=256, positions=256)
    pages = ex.PageTable(R, 160, 16)
    cache = block.cache(pages, page_scales=page_scales)
    ex.prefill(block, cache, pages, torch.randn(R, prompt, 512, device=DEV).bfloat16(), 20)
    embed = torch.nn.functional.normalize(torch.randn(300, 512, device=DEV)).bfloat16()
    decode = ex.DraftedDecoder(block, cache, pages, embed, ints([5, 6, 7]), n)
    cached, stood = [prompt] * R, 0
    assert decode.cached.tolist() == cached
    for _ in range(8):
        last = decode.last.tolist()
        tokens, accepted, following = (t.cpu() for t in decode())
        assert decode.status() == 0
        assert tokens[:, 0].tolist() == last
        assert pages.kv_len.tolist() == [c + n + 1 for c in cached]
        q_start = pages.q_start.cpu()
        assert q_start.tolist() == [i * (n + 1) for i in range(R + 1)]
        want = verify(decode.target.cpu(), decode.draft.flatten(0, 1).cpu(), tokens.flatten(), q_start,
                      decode.accept_u.cpu(), decode.sample_u.cpu())
        assert accepted.tolist() == want[0] and following.tolist() == want[1]
        cached = [c + 1 + k for c, k in zip(cached, want[0])]
        assert decode.cached.tolist() == cached
        stood += sum(want[0])
        table, ring, (first, free) = pages.table.tolist(), pages.pool.ring.tolist(), pages.pool.state.tolist()
        held = [p for r, length in enumerate(pages.kv_len.tolist()) for p in table[r][:-(-length // 16)]]
        assert sorted(held + [ring[(first + i) % len(ring)] for i in range(free)]) == list(range(pages.num_pages))
    assert 0 < stood < 8 * R * n                           # some stand, some do not
    k, v = cache.k.double().cpu(), cache.v.double().cpu()
    if page_scales:
        k, v = (x * s.double().cpu()[:, None, :, None] for x, s in ((k, cache.k_scale), (v, cache.v_scale)))
    for r in range(R):
        length = int(pages.kv_len[r])
        at = torch.tensor(table[r][:-(-length // 16)])
        vs = cache.v_scale.double().cpu()[at] if page_scales else torch.ones(len(at), block.hk).double()
        rows = slice(r * (n + 1), (r + 1) * (n + 1))
        for h in range(block.hk):
            g = block.hq // block.hk
            out, _, bound, _ = request_attention(
                seen["q"][rows, h * g:(h + 1) * g].double().cpu(), k[at, :, h].flatten(0, 1)[:length],
                v[at, :, h].flatten(0, 1)[:length], vs[:, h].repeat_interleave(16)[:length], length - n - 1,
                block.D ** -0.5, 0)
            err = (seen["out"][rows, h * g:(h + 1) * g].double().cpu() - out).abs()
            assert (err <= bound).all(), (err - bound).max()


def test_the_example_runs_with_drafted_tokens(ex, capsys):
    y, whole, last = ex.main(["--requests", "2", "--prompt", "100", "--chunk", "33", "--new", "5", "--drafts", "2",
                              "--page-scales"])
    assert y.isfinite().all() and whole.isfinite().all() and last.shape == (2,)
    assert "drafted tokens" in capsys.readouterr().out


def test_two_steps_on_two_streams(nb):
    """Plans, appends and attention of two batches at once, on streams and workspaces of
    their own, give what they give one after the other."""
    def make(seed):
        g = torch.Generator().manual_seed(seed)
        pool = nb.PagePool(torch.randperm(64, generator=g).int().to(DEV), ints([0, 64]))
        batch = nb.AttnBatch(ints([0] * 4), ints([0] * 3), ints([[0] * 8] * 3), max_new=40)
        side = [torch.zeros(64, 16, 2, 128, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        cache = nb.PagedKVCache(*side, k_scale=torch.ones(64, 2, device=DEV), v_scale=torch.ones(64, 2, device=DEV))
        x = torch.randn(120, 8, 128, generator=g).bfloat16().to(DEV)
        new = [ints([40, 23, 7]), ints([1, 3, 2])]
        ws = [nb.attn_workspace(), nb.paged_attention_workspace(cache, batch, 4, 120)]
        return pool, batch, cache, x, new, ws

    def steps(state, stream):
        pool, batch, cache, x, new, (ws, ws_attn) = state
        outs = []
        for add, rows in zip(new, (70, 6)):
            nb.plan_pages(pool, batch, 16, add, ws=ws, stream=stream)
            q, k, v = x[:rows, :4], x[:rows, 4:6], x[:rows, 6:]
            nb.kv_append(cache, batch, k, v, ws=ws, stream=stream)
            outs.append(nb.paged_attention(q, cache, batch, ws=ws_attn, stream=stream))
        return outs + [cache.k.view(torch.uint8), cache.v_scale, batch.kv_len, pool.ring]
    alone = [[t.clone() for t in steps(make(seed), None)] for seed in (1, 2)]
    states = [make(seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [steps(state, stream) for state, stream in zip(states, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
