"""The decoder block example: the attention operators next to the experts, as a
serving loop runs them."""
import os
import sys

import pytest
import torch

from _attention_reference import attention

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_block
    return decoder_block


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_steps_attend_to_what_the_cache_holds(ex, monkeypatch, fp8):
    """Prompts of 90 tokens in chunks of 37, then four single tokens, 3 requests:
    each step's attention against the 64-bit one over the cache at that time,
    and the cache lengths."""
    nb, seen = ex.nb, []
    inner = nb.paged_attention

    def recorded(q, cache, batch, **kw):
        out = inner(q, cache, batch, **kw)
        seen.append([t.cpu().clone() for t in (q, out, cache.k, cache.v, batch.q_start,
                                               batch.kv_len, batch.page_table)])
        return out
    monkeypatch.setattr(nb, "paged_attention", recorded)
    torch.manual_seed(1)
    block = ex.DecoderBlock(hidden=512, q_heads=4, inter=256, positions=128)
    pages = ex.PageTable(3, 100, 16)
    cache = block.cache(pages, fp8)
    y = ex.prefill(block, cache, pages, torch.randn(3, 90, 512, device=DEV).bfloat16(), 37)
    assert y.isfinite().all()
    q_start = torch.arange(4, dtype=torch.int32, device=DEV)
    step = ex.Step(block, cache, nb.AttnBatch(q_start, pages.kv_len, pages.table, max_new=1), 3)
    x = y[:, -1].contiguous()
    for _ in range(4):
        pages.grow([1, 1, 1])
        x = step(x).clone()
    assert step.status() == 0 and x.isfinite().all()
    assert [int(s[5][0]) for s in seen] == [37, 74, 90, 91, 92, 93, 94]
    ks = None if cache.k_scale is None else cache.k_scale.cpu()
    vs = None if cache.v_scale is None else cache.v_scale.cpu()
    for q, out, k, v, start, lens, table in seen:
        want, _, bound, _ = attention(q, k, v, start, lens, table, k_scale=ks, v_scale=vs)
        over = (out.double() - want).abs() - bound
        assert (over <= 0).all(), over.max()


def test_decoding_from_a_graph_is_decoding(ex):
    """The captured step gives bit for bit what the calls give, as the requests grow
    over page borders, and leaves the cache as it found it when it is captured."""
    nb = ex.nb
    got = []
    for graph in (False, True):
        torch.manual_seed(2)
        block = ex.DecoderBlock(hidden=512, q_heads=4, inter=256, positions=128)
        pages = ex.PageTable(2, 80, 16)
        cache = block.cache(pages)
        x = torch.randn(2, 30, 512, device=DEV).bfloat16()
        token = ex.prefill(block, cache, pages, x, 30)[:, -1].contiguous()
        if graph:
            before = cache.k.clone()
            run = ex.Decoder(block, cache, pages, 2, 512)
            assert torch.equal(cache.k, before)
        else:
            q_start = torch.arange(3, dtype=torch.int32, device=DEV)
            step = ex.Step(block, cache, nb.AttnBatch(q_start, pages.kv_len, pages.table, 1), 2)

            def run(t):
                pages.grow([1, 1])
                return step(t)
        for _ in range(20):
            token = run(token).clone()
        got.append(token)
    assert got[0].isfinite().all() and torch.equal(got[0], got[1])


def test_the_example_runs(ex, capsys):
    y, whole, token = ex.main(["--requests", "2", "--prompt", "100", "--chunk", "33", "--new", "5"])
    assert token.shape == (2, 1024) and token.isfinite().all()
    assert y.isfinite().all() and whole.isfinite().all()
    assert "us a step" in capsys.readouterr().out
