"""The attention entry points refuse bad arguments on the host, before anything
is enqueued (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = 1 << 20                      # never dereferenced: every call fails its checks first
INVALID, SHAPE, MISALIGNED, SMALL = 1, 2, 3, 4


@pytest.fixture(scope="module")
def nb():
    import __graft_entry__
    __graft_entry__.build()
    from nvfp4_block_scaled_route_gb300 import binding
    return binding


def _cache(nb, **kw):
    d = dict(k=FAKE, v=FAKE, dtype=nb.BF16, kv_heads=2, head_dim=128, page_size=16, num_pages=8,
             page_stride=16 * 256, token_stride=256, head_stride=128, k_scale=None, v_scale=None)
    d.update(kw)
    return ctypes.byref(nb.KvCache(**d))


def _batch(nb, **kw):
    d = dict(batch=2, max_new=1, tokens=2, max_pages=4, q_start=FAKE, kv_len=FAKE, page_table=FAKE)
    d.update(kw)
    return ctypes.byref(nb.AttnBatchArgs(**d))


def _rope_args(q=FAKE, qs=(512, 128), hq=4, k=FAKE, ks=(256, 128), hk=2, T=3, D=128, pos=FAKE,
               rope=FAKE, npos=16, rot=128, wq=FAKE, wk=FAKE, eps=1e-6, qo=FAKE, qos=(512, 128),
               ko=FAKE, kos=(256, 128), ws=FAKE, n=256):
    return (q, *qs, hq, k, *ks, hk, T, D, pos, rope, npos, rot, 0, wq, wk, eps, qo, *qos, ko, *kos,
            ws, n, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=-1)), (INVALID, dict(hq=-1)), (INVALID, dict(ws=None)), (SMALL, dict(n=255)),
    (MISALIGNED, dict(ws=FAKE + 8)), (SHAPE, dict(D=96)), (SHAPE, dict(D=256)),
    (SHAPE, dict(T=1 << 30)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(npos=0)), (SHAPE, dict(rot=8)), (SHAPE, dict(rot=24)), (SHAPE, dict(rot=144)),
    (MISALIGNED, dict(rope=FAKE + 4)), (MISALIGNED, dict(wq=FAKE + 2)), (INVALID, dict(pos=None)),
    (INVALID, dict(q=None)), (INVALID, dict(ko=None)), (MISALIGNED, dict(q=FAKE + 8)),
    (MISALIGNED, dict(qs=(516, 128))), (INVALID, dict(ks=(256, 64))), (INVALID, dict(qs=(-512, 128))),
    (0, dict(T=0, q=None, k=None)), (0, dict(hq=0, hk=0))])
def test_qk_norm_rope_refuses(nb, want, kw):
    assert nb.lib().attn_qk_norm_rope(*_rope_args(**kw)) == want


CACHES = [
    (INVALID, dict(kv_heads=0)), (INVALID, dict(dtype=1)), (SHAPE, dict(head_dim=96)),
    (SHAPE, dict(page_size=8)), (SHAPE, dict(page_size=48)), (SHAPE, dict(page_size=2048)),
    (INVALID, dict(k=None)), (MISALIGNED, dict(v=FAKE + 8)), (INVALID, dict(token_stride=0)),
    (MISALIGNED, dict(token_stride=260)), (INVALID, dict(num_pages=-1)),
    (SHAPE, dict(num_pages=1 << 31)), (INVALID, dict(page_stride=1 << 40))]
BATCHES = [
    (INVALID, dict(batch=-1)), (INVALID, dict(max_new=0)), (INVALID, dict(tokens=-1)),
    (INVALID, dict(q_start=None)), (INVALID, dict(kv_len=None)), (INVALID, dict(page_table=None)),
    (SHAPE, dict(max_pages=1 << 27)), (SHAPE, dict(tokens=1 << 31)), (0, dict(tokens=0, q_start=None))]


def _append(nb, cache, batch, k=FAKE, q=FAKE, hq=4, qo=FAKE, ws=FAKE, n=256, rope=FAKE, rot=128):
    return nb.lib().attn_kv_append(cache, batch, k, 256, 128, FAKE, 256, 128, q, 512, 128, hq, qo,
                                   512, 128, rope, 16, rot, 0, FAKE, FAKE, 1e-6, ws, n, None)


def _forward(nb, cache, batch, q=FAKE, hq=4, scale=1.0, window=0, out=FAKE, ws=FAKE, n=1 << 40):
    return nb.lib().attn_paged_forward(q, 512, 128, hq, cache, batch, scale, window, out, 512, 128,
                                       None, ws, n, None)


@pytest.mark.parametrize("want,kw", CACHES)
def test_bad_caches_are_refused(nb, want, kw):
    assert _append(nb, _cache(nb, **kw), _batch(nb)) == want
    assert _forward(nb, _cache(nb, **kw), _batch(nb)) == want


@pytest.mark.parametrize("want,kw", BATCHES)
def test_bad_batches_are_refused(nb, want, kw):
    assert _append(nb, _cache(nb), _batch(nb, **kw)) == want
    assert _forward(nb, _cache(nb), _batch(nb, **kw)) == want


def test_kv_append_refuses(nb):
    c, b = _cache(nb), _batch(nb)
    assert _append(nb, None, b) == INVALID and _append(nb, c, None) == INVALID
    assert _append(nb, c, b, k=None) == INVALID
    assert _append(nb, c, b, q=None) == INVALID
    assert _append(nb, c, b, qo=FAKE + 4) == MISALIGNED
    assert _append(nb, c, b, hq=-1) == INVALID
    assert _append(nb, c, b, ws=None) == INVALID
    assert _append(nb, c, b, n=0) == SMALL
    assert _append(nb, c, b, rot=20) == SHAPE
    assert _append(nb, c, _batch(nb, tokens=1 << 30)) == SHAPE


def test_paged_forward_refuses(nb):
    c, b = _cache(nb), _batch(nb)
    need = nb.lib().attn_paged_workspace_size(2, 2, 1, 4, 2, 128)
    assert need >= 256
    assert _forward(nb, None, b) == INVALID and _forward(nb, c, None) == INVALID
    assert _forward(nb, c, b, hq=0) == INVALID
    assert _forward(nb, c, b, hq=3) == SHAPE
    assert _forward(nb, c, b, window=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _forward(nb, c, b, scale=scale) == INVALID
    assert _forward(nb, c, b, q=None) == INVALID
    assert _forward(nb, c, b, out=FAKE + 8) == MISALIGNED
    assert _forward(nb, c, b, ws=None) == INVALID
    assert _forward(nb, c, b, ws=FAKE + 8) == MISALIGNED
    assert _forward(nb, c, b, n=need - 1) == SMALL
    assert _forward(nb, c, _batch(nb, tokens=1 << 30)) == SHAPE


def test_workspace_size_of_bad_shapes_is_zero(nb):
    f = nb.lib().attn_paged_workspace_size
    assert f(-1, 1, 1, 4, 2, 128) == 0 and f(1, -1, 1, 4, 2, 128) == 0
    assert f(1, 1, 0, 4, 2, 128) == 0 and f(1, 1, 1, 3, 2, 128) == 0
    assert f(1, 1, 1, 4, 0, 128) == 0 and f(1, 1, 1, 4, 2, 96) == 0
    assert f(0, 0, 1, 4, 2, 128) >= 256
