"""The operators of a serving step refuse bad arguments on the host, before anything is
enqueued (no GPU needed)."""
import pytest
import torch

from test_attention_args import FAKE, INVALID, MISALIGNED, SHAPE, SMALL, _append, _batch, _cache, _forward, nb  # noqa: F401
from test_attention_host import Device


# ------------------------------------------------------------ page scales --
def test_page_scales_are_not_optional(nb):
    paged = dict(dtype=nb.E4M3_PAGES, k_scale=FAKE, v_scale=FAKE)
    for call in (_append, _forward):
        assert call(nb, _cache(nb, **paged), _batch(nb), n=0) == SMALL        # (all but the workspace)
        for missing in ("k_scale", "v_scale"):
            assert call(nb, _cache(nb, **{**paged, missing: None}), _batch(nb)) == INVALID
            assert call(nb, _cache(nb, **{**paged, missing: FAKE + 2}), _batch(nb)) == MISALIGNED
        assert call(nb, _cache(nb, **{**paged, "dtype": 5}), _batch(nb)) == INVALID
        assert call(nb, _cache(nb, **{**paged, "token_stride": 136}), _batch(nb)) == MISALIGNED


class Workspace(Device):
    def __init__(self):
        super().__init__(256, dtype=torch.uint8)

    def numel(self):
        return 256


class Cache(Device):
    """A dense cache side, as the handle reads it."""

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]


def _sides():
    return [Cache(5, 16, 2, 128, dtype=torch.float8_e4m3fn) for _ in range(2)]


def test_a_cache_handle_tells_scales_of_pages_from_those_of_heads(nb):
    f32 = torch.float32
    by_head = nb.PagedKVCache(*_sides(), k_scale=Device(2, dtype=f32), v_scale=Device(2, dtype=f32))
    assert by_head.struct.dtype == nb.E4M3
    by_page = nb.PagedKVCache(*_sides(), k_scale=Device(5, 2, dtype=f32), v_scale=Device(5, 2, dtype=f32))
    assert by_page.struct.dtype == nb.E4M3_PAGES and by_page.struct.k_scale == 1 << 20
    for k, v in [((5, 2), (2,)), ((2,), (5, 2)), ((5, 2), None), ((4, 2), (5, 2)), ((5, 2), (5, 3))]:
        with pytest.raises(ValueError, match="_scale must be"):
            nb.PagedKVCache(*_sides(), k_scale=Device(*k, dtype=f32),
                            v_scale=None if v is None else Device(*v, dtype=f32))
    with pytest.raises(ValueError, match="k_scale must be"):
        nb.PagedKVCache(*_sides(), k_scale=Device(5, 2, dtype=torch.float64), v_scale=Device(5, 2, dtype=f32))
    with pytest.raises(ValueError):                                # bf16 caches have none
        nb.PagedKVCache(*[Cache(5, 16, 2, 128, dtype=torch.bfloat16) for _ in range(2)],
                        k_scale=Device(5, 2, dtype=f32), v_scale=Device(5, 2, dtype=f32))


# -------------------------------------------------------------- page plan --
def _plan(nb, ring=FAKE, size=8, state=FAKE, out=FAKE, batch=2, page=16, max_pages=4, before=FAKE, cached=FAKE,
          new=FAKE, kv_len=FAKE, q_start=FAKE, table=FAKE, positions=FAKE, slots=FAKE, rows=10, ws=FAKE, n=256):
    return nb.lib().attn_plan_pages(ring, size, state, out, batch, page, max_pages, before, cached, new, kv_len,
                                    q_start, table, positions, slots, rows, ws, n, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(ring=None)), (INVALID, dict(size=0)), (SHAPE, dict(size=1 << 31)), (INVALID, dict(state=None)),
    (INVALID, dict(out=None)), (INVALID, dict(batch=-1)), (SHAPE, dict(page=8)), (SHAPE, dict(page=48)),
    (SHAPE, dict(page=2048)), (INVALID, dict(max_pages=-1)), (SHAPE, dict(max_pages=1 << 27)),
    (INVALID, dict(before=None)), (INVALID, dict(new=None)), (INVALID, dict(kv_len=None)),
    (INVALID, dict(q_start=None)), (INVALID, dict(table=None)), (INVALID, dict(rows=-1)), (SHAPE, dict(rows=1 << 31)),
    (INVALID, dict(ws=None)), (MISALIGNED, dict(ws=FAKE + 4)), (SMALL, dict(n=255))])
def test_plan_pages_refuses(nb, want, kw):
    assert _plan(nb, **kw) == want


def test_plan_pages_binding_refuses(nb):
    pool = nb.PagePool(Device(8), Device(2))
    batch = nb.AttnBatch(Device(3), Device(2), Device(2, 4), max_new=5)
    ws = Workspace()
    for kw in (dict(new_tokens=Device(3)), dict(new_tokens=Device(2, dtype=torch.int64)),
               dict(cached=Device(1)), dict(kv_before=Device(3)), dict(state_out=Device(3)),
               dict(positions=Device(7, dtype=torch.int64)), dict(slots=Device(7))):
        with pytest.raises(ValueError, match="must be"):
            nb.plan_pages(pool, batch, 16, **{"new_tokens": Device(2), "ws": ws, **kw})
    with pytest.raises(ValueError, match="state must be"):
        nb.PagePool(Device(8), Device(3))


# ----------------------------------------------------------- verification --
def _verify(nb, target=FAKE, ts=100, draft=FAKE, ds=100, dtype=1, rows=6, vocab=100, tokens=FAKE, batch=2,
            q_start=FAKE, kv_len=FAKE, accept=FAKE, sample=FAKE, accepted=FAKE, nxt=FAKE, cached=FAKE, ws=FAKE,
            n=256):
    return nb.lib().draft_verify(target, ts, draft, ds, dtype, rows, vocab, tokens, batch, q_start, kv_len, accept,
                                 sample, accepted, nxt, cached, ws, n, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(target=None)), (MISALIGNED, dict(target=FAKE + 2)), (MISALIGNED, dict(draft=FAKE + 1)),
    (MISALIGNED, dict(dtype=0, target=FAKE + 1)), (INVALID, dict(ts=99)), (INVALID, dict(ds=99)),
    (INVALID, dict(ts=1 << 31)), (INVALID, dict(dtype=2)), (INVALID, dict(dtype=3)), (INVALID, dict(rows=-1)),
    (SHAPE, dict(rows=1 << 31)), (INVALID, dict(vocab=0)), (SHAPE, dict(vocab=(1 << 30) + 1)),
    (INVALID, dict(tokens=None)), (INVALID, dict(batch=-1)), (SHAPE, dict(batch=1 << 28)),
    (INVALID, dict(q_start=None)), (INVALID, dict(kv_len=None)), (INVALID, dict(accept=None)),
    (INVALID, dict(sample=None)), (INVALID, dict(accepted=None)), (INVALID, dict(nxt=None)), (INVALID, dict(ws=None)),
    (MISALIGNED, dict(ws=FAKE + 8)), (SMALL, dict(n=0)),
    (0, dict(batch=0, target=None, tokens=None, q_start=None, accepted=None))])
def test_draft_verify_refuses(nb, want, kw):
    assert _verify(nb, **kw) == want


def test_draft_verify_binding_refuses(nb):
    class Rows(Cache):
        device = "cuda"

        def __init__(self, *shape, dtype=torch.float32, strides=None):
            super().__init__(*shape, dtype=dtype)
            self.strides = strides

        def stride(self, i=None):
            return self.strides or super().stride(i)
    f32 = torch.float32
    batch = nb.AttnBatch(Device(3), Device(2), Device(2, 4), max_new=5)
    good = dict(target=Rows(6, 50), draft=Rows(6, 50), tokens=Device(6), accept_u=Device(6, dtype=f32),
                sample_u=Device(2, dtype=f32), accepted=Device(2), next_token=Device(2),
                ws=Workspace())
    for kw in (dict(target=Rows(6, 50, dtype=torch.float16)), dict(draft=Rows(6, 49)), dict(draft=Rows(5, 50)),
               dict(draft=Rows(6, 50, dtype=torch.bfloat16)), dict(target=Rows(6, 50, strides=(1, 6))),
               dict(tokens=Device(5)), dict(tokens=Device(6, dtype=torch.int64)), dict(accept_u=Device(6)),
               dict(sample_u=Device(3, dtype=f32)), dict(accepted=Device(3)), dict(next_token=Device(1)),
               dict(cached=Device(3))):
        with pytest.raises(ValueError, match="must"):
            nb.draft_verify(batch=batch, **{**good, **kw})


# --------------------------------------------------------- the extension --
def test_the_extension_checks_head_rows(nb):
    class Rows(Cache):
        def __init__(self, *shape, dtype=torch.bfloat16, strides=None):
            super().__init__(*shape, dtype=dtype)
            self.strides = strides

        def stride(self, i=None):
            return self.strides or super().stride(i)
    rows = nb._calls().rows
    assert rows(Rows(5, 4, 128), torch.bfloat16, "q") == (1 << 20, 512, 128)
    assert rows(Rows(5, 4, 128, strides=(1024, 128, 1)), torch.bfloat16, "q") == (1 << 20, 1024, 128)
    for bad in (Rows(5, 4, 128, dtype=torch.float16), Rows(5, 128)):
        with pytest.raises(ValueError, match="q must be a bf16 CUDA tensor"):
            rows(bad, torch.bfloat16, "q")
    cpu = Rows(5, 4, 128)
    cpu.is_cuda = False
    with pytest.raises(ValueError, match="q must be a bf16 CUDA tensor"):
        rows(cpu, torch.bfloat16, "q")
    with pytest.raises(ValueError, match="head_dim must be contiguous"):
        rows(Rows(5, 4, 128, strides=(512, 1, 4)), torch.bfloat16, "q")
    with pytest.raises(AttributeError):
        rows(3, torch.bfloat16, "q")


def test_the_extension_checks_vectors(nb):
    vector = nb._calls().vector
    assert vector(None, 3, torch.int32, "x") is None
    assert vector(Device(3), 3, torch.int32, "x") == 1 << 20
    for bad, n in ((Device(3), 4), (Device(3, dtype=torch.int64), 3), (Device(3, 1), 3)):
        with pytest.raises(ValueError, match=r"x must be torch.int32 \[%d\]" % n):
            vector(bad, n, torch.int32, "x")
    loose = Device(3)
    loose.is_contiguous = lambda: False
    with pytest.raises(ValueError, match="x must be a dense CUDA tensor"):
        vector(loose, 3, torch.int32, "x")
    with pytest.raises(TypeError):
        vector(Device(3), 3)


def test_the_extension_takes_any_dense_tensor_as_memory(nb):
    dense = nb._calls().dense
    assert dense(Workspace()) == (1 << 20, 256)
    host, loose = Workspace(), Workspace()
    host.is_cuda, loose.is_contiguous = False, lambda: False
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        dense(host)
    with pytest.raises(ValueError, match="expected a contiguous tensor"):
        dense(loose)


def test_the_extension_passes_arguments_as_they_are(nb):
    """Each call's refusals are those of the entry point itself; what is no argument at all
    raises before it."""
    host = nb._calls()
    plan = [FAKE, 8, FAKE, FAKE, 2, 16, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 10, FAKE, 0, None]
    assert host.attn_plan_pages(*plan) == SMALL
    for at, value, want in ((1, 0, INVALID), (5, 24, SHAPE), (6, 1 << 40, SHAPE), (0, None, INVALID),
                            (15, 1 << 31, SHAPE), (16, None, INVALID), (16, FAKE + 4, SMALL)):
        assert host.attn_plan_pages(*plan[:at], value, *plan[at + 1:]) == want
    with pytest.raises(TypeError):
        host.attn_plan_pages(*plan[:-1])
    with pytest.raises(TypeError):
        host.attn_plan_pages("ring", *plan[1:])
    with pytest.raises(OverflowError):
        host.attn_plan_pages(FAKE, 1 << 70, *plan[2:])
    cache = nb.KvCache(FAKE, FAKE, nb.E4M3_PAGES, 2, 128, 16, 8, 16 * 256, 256, 128, FAKE, FAKE)
    batch = nb.AttnBatchArgs(2, 1, 2, 4, FAKE, FAKE, FAKE)
    call = [FAKE, 512, 128, 4, cache, batch, 1.0, 0, FAKE + 4096, 512, 128, None, FAKE, 0, None]
    assert host.attn_paged_forward(*call) == SMALL
    assert host.attn_paged_forward(*call[:6], float("nan"), *call[7:]) == INVALID
    assert host.attn_paged_forward(*call[:7], -1, *call[8:]) == INVALID
    with pytest.raises(TypeError):
        host.attn_paged_forward(*call[:4], 7, *call[5:])
    append = [cache, batch, FAKE, 256, 128, FAKE, 256, 128, None, 0, 0, 0, None, 0, 0, None, 0, 0, 0, None, None, 1e-6,
              FAKE, 0, None]
    assert host.attn_kv_append(*append) == SMALL
    assert host.attn_kv_append(*append[:21], -1.0, FAKE, 256, None) == INVALID
    verify = [FAKE, 100, FAKE, 100, 1, 6, 100, FAKE, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None]
    assert host.draft_verify(*verify) == SMALL
    rope = [FAKE, 512, 128, 4, FAKE, 256, 128, 2, 3, 128, FAKE, FAKE, 16, 128, 0, FAKE, FAKE, 1e-6, FAKE, 512, 128,
            FAKE, 256, 128, FAKE, 0, None]
    assert host.attn_qk_norm_rope(*rope) == SMALL


@pytest.mark.parametrize("head_dim,ctas", [(64, 256), (128, 304)])
@pytest.mark.parametrize("rows", [1, 7, 16])
def test_the_workspace_of_few_rows_holds_the_pieces_that_there_are(nb, head_dim, ctas, rows):
    """Two pieces of every CTA, each a row's sums with its maximum and weight sum: 256 CTAs, or
    two on each of 152 SMs for the kernel that takes 128-wide heads over pages with scales."""
    size = nb.lib().attn_paged_workspace_size(64, 64, 1, 8 * rows, 8, head_dim)
    pieces = 2 * ctas * rows * (head_dim * 4 + 8)
    assert pieces <= size <= pieces + 32768
