"""A decoder block on the attention operators and the NVFP4 experts, served step
by step: prompts in chunks, then single or drafted tokens replayed from a CUDA graph.

    python examples/decoder_block.py [--prompt 600] [--chunk 256] [--new 64] [--fp8-cache]
                                     [--page-scales] [--drafts 4]

A step's launches are those of a serving loop: ``plan_pages`` (lengths and page
tables, on the GPU); one product for q, k and v; ``kv_append`` (norm, rotation and
append, queries in the same launch); ``paged_attention`` over the pages; the output
product; ``router_topk`` and ``FusedLayer`` for the experts; with drafted tokens
``draft_verify`` behind them, whose answer the next step's plan starts from.  Weights
are random, so it shows how the calls fit together.  However a prompt is cut, the block
gives the same answers up to the experts' FP4 rounding: a step's activations share one
global scale, from the largest of them, so the grid that they are rounded to goes by the
step.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_route_gb300 import binding as nb  # noqa: E402


def rope_table(positions: int, rotary_dim: int, base: float = 1e4, device="cuda"):
    """float32 [positions, rotary_dim]: cosines, then sines, of position * base^(-2 i / dim)."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] \
        * base ** (-2 * i / rotary_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class PageTable:
    """Requests' pages from one pool, planned on the device as the requests grow."""

    def __init__(self, requests: int, max_len: int, page_size: int, device="cuda"):
        self.page_size, self.device = page_size, device
        self.max_pages = -(-max_len // page_size)
        self.num_pages = requests * self.max_pages
        self.pool = nb.PagePool(torch.randperm(self.num_pages).int().to(device),
                                torch.tensor([0, self.num_pages], dtype=torch.int32, device=device))
        self.lengths = [0] * requests
        self.table = torch.zeros(requests, self.max_pages, dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(requests, dtype=torch.int32, device=device)
        self.q_start = torch.zeros(requests + 1, dtype=torch.int32, device=device)
        self.new = torch.zeros(requests, dtype=torch.int32, device=device)
        self.ws = nb.attn_workspace(device)

    def batch(self, max_new: int) -> nb.AttnBatch:
        """The step's requests as the operators take them, of up to max_new new tokens each."""
        return nb.AttnBatch(self.q_start, self.kv_len, self.table, max_new=max_new)

    def grow(self, new):
        """new[r] more tokens for each request; the device tensors follow in place."""
        for r, n in enumerate(new):
            if self.lengths[r] + n > self.max_pages * self.page_size:
                raise ValueError(f"request {r} has outgrown its pages")
        self.lengths = [have + n for have, n in zip(self.lengths, new)]
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        nb.plan_pages(self.pool, self.batch(max(1, *new)), self.page_size, self.new, ws=self.ws)


class DecoderBlock:
    """x + attention, then + experts; bf16 in and out, one NVFP4 expert layer."""

    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, experts=8, inter=512,
                 topk=2, positions=4096, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(*shape, generator=g, device=device)
        self.hq, self.hk, self.D, self.k = q_heads, kv_heads, head_dim, topk
        heads = q_heads + 2 * kv_heads
        self.w_qkv = (rand(heads * head_dim, hidden) * hidden ** -0.5).bfloat16()
        self.w_out = (rand(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5).bfloat16()
        self.w_router = (rand(experts, hidden) * hidden ** -0.5).bfloat16()
        self.w_in = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.w_mid = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.q_weight = (1 + 0.1 * rand(head_dim)).bfloat16()
        self.k_weight = (1 + 0.1 * rand(head_dim)).bfloat16()
        self.rope = rope_table(positions, head_dim, device=device)
        q1, s1, g1 = nb.quantize_weights(rand(experts, hidden, 2 * inter) * hidden ** -0.5)
        q2, s2, g2 = nb.quantize_weights(rand(experts, inter, hidden) * inter ** -0.5)
        self.experts = nb.PreparedWeights.from_checkpoint(q1, s1, g1, q2, s2, g2)

    def cache(self, pages: PageTable, fp8: bool = False,
              page_scales: bool = False) -> nb.PagedKVCache:
        shape = (pages.num_pages, pages.page_size, self.hk, self.D)
        dtype = torch.float8_e4m3fn if fp8 or page_scales else torch.bfloat16
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=pages.device).to(dtype)
                for _ in range(2))
        if page_scales:                                         # set by the append
            ks, vs = (torch.ones(pages.num_pages, self.hk, device=pages.device) for _ in range(2))
            return nb.PagedKVCache(k, v, k_scale=ks, v_scale=vs)
        # keys after the norm stay within sqrt(D) or so times their weight, values within a few
        scale = [torch.full((self.hk,), s, device=pages.device) if fp8 else None
                 for s in (self.D ** 0.5 / 256, 8 / 256)]
        return nb.PagedKVCache(k, v, k_scale=scale[0], v_scale=scale[1])


class Step:
    """The block over up to `tokens` rows of one batch shape, on buffers of its own."""

    def __init__(self, block: DecoderBlock, cache: nb.PagedKVCache, batch: nb.AttnBatch,
                 tokens: int):
        self.block, self.kv, self.batch, self.tokens = block, cache, batch, tokens
        dev = cache.k.device
        self.ws_append = nb.attn_workspace(dev)
        self.ws_attn = nb.paged_attention_workspace(cache, batch, block.hq, tokens)
        self.layer = nb.FusedLayer(block.experts, tokens, block.k, device=dev)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        b = self.block
        h = F.rms_norm(x, (x.shape[1],), b.w_in, 1e-6)
        qkv = (h @ b.w_qkv.T).view(self.tokens, b.hq + 2 * b.hk, b.D)
        q, k, v = qkv.split((b.hq, b.hk, b.hk), dim=1)         # strided views, as they are
        q = nb.kv_append(self.kv, self.batch, k, v, b.rope, b.k_weight, q=q,
                         q_weight=b.q_weight, ws=self.ws_append)
        a = nb.paged_attention(q, self.kv, self.batch, ws=self.ws_attn)
        x = x + a.view(self.tokens, -1) @ b.w_out.T
        h = F.rms_norm(x, (x.shape[1],), b.w_mid, 1e-6)
        ids, wts = nb.router_topk(h, b.w_router, b.k)
        return x + self.layer.forward(h, ids, wts)

    def status(self) -> int:
        return (nb.read_status(self.ws_append) or nb.read_status(self.ws_attn)
                or self.layer.status())


def prefill(block, cache, pages, x, chunk):
    """Prompts x [requests, length, hidden], up to `chunk` tokens of each a step."""
    R, length, _ = x.shape
    y = torch.empty_like(x)
    for at in range(0, length, chunk):
        n = min(chunk, length - at)
        pages.grow([n] * R)
        step = Step(block, cache, pages.batch(n), R * n)
        y[:, at:at + n] = step(x[:, at:at + n].reshape(R * n, -1)).view(R, n, -1)
        if step.status():
            raise RuntimeError(f"device status {step.status()}")
    return y


def captured(fn, keep):
    """A graph of fn and what it returned.  Warm-up and capture leave the tensors `keep`
    as they were."""
    saved = [(t, t.clone()) for t in keep]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    for t, old in saved:
        t.copy_(old)
    return graph, out


def cache_tensors(cache):
    return [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]


class Decoder:
    """One token of every request a step, replayed from a graph: the page table
    and the lengths are read on the device, so they may move under it."""

    def __init__(self, block, cache, pages, requests, hidden):
        q_start = torch.arange(requests + 1, dtype=torch.int32, device=pages.device)
        batch = nb.AttnBatch(q_start, pages.kv_len, pages.table, max_new=1)
        self.pages, self.step = pages, Step(block, cache, batch, requests)
        self.x = torch.zeros(requests, hidden, dtype=torch.bfloat16, device=pages.device)
        # (warm-up and capture write at the requests' last positions)
        self.graph, self.y = captured(lambda: self.step(self.x), cache_tensors(cache))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        self.pages.grow([1] * x.shape[0])
        self.x.copy_(x)
        self.graph.replay()
        return self.y


class DraftedDecoder:
    """`drafts` tokens guessed for every request and held against the block's own
    distributions, a step from a graph that takes nothing from the host: which tokens
    stand, the next step's lengths and its pages stay on the device.

    The block stands between an embedding and its transpose; the draft is the embedding
    alone, a token's distribution going by the token before."""

    def __init__(self, block, cache, pages, embed, last, drafts=4, temperature=0.05):
        R, dev = last.shape[0], pages.device
        self.pages, self.embed, self.temperature = pages, embed, temperature
        self.drafts, self.requests, V = drafts, R, embed.shape[0]
        self.batch = pages.batch(drafts + 1)
        self.step = Step(block, cache, self.batch, R * (drafts + 1))
        self.ws = nb.attn_workspace(dev)
        self.new = torch.full((R,), drafts + 1, dtype=torch.int32, device=dev)
        self.tokens = torch.zeros(R, drafts + 1, dtype=torch.int32, device=dev)
        self.draft = torch.zeros(R, drafts + 1, V, device=dev)
        self.accepted = torch.zeros(R, dtype=torch.int32, device=dev)
        self.last = last.clone()                    # each request's newest token, not yet cached
        self.cached = pages.kv_len.clone()          # tokens that stand
        keep = [*cache_tensors(cache), pages.pool.ring, pages.pool.state, pages.table,
                pages.kv_len, pages.q_start, self.last, self.cached, self.accepted]
        self.graph, _ = captured(self._step, keep)

    def _distribution(self, x):
        return torch.softmax(x.float() @ self.embed.float().T / self.temperature, dim=-1)

    def _step(self):
        R, n, dev = self.requests, self.drafts, self.pages.device
        self.tokens[:, 0] = self.last
        for i in range(n):
            q = self._distribution(F.rms_norm(self.embed[self.tokens[:, i].long()], (self.embed.shape[1],)))
            self.draft[:, i] = q
            passed = q.double().cumsum(1) > torch.rand(R, 1, dtype=torch.float64, device=dev)
            self.tokens[:, i + 1] = passed.int().argmax(1).int()
        nb.plan_pages(self.pages.pool, self.batch, self.pages.page_size, self.new,
                      cached=self.cached, ws=self.ws)
        tokens = self.tokens.view(-1)
        y = self.step(self.embed[tokens.long()])
        self.target = self._distribution(F.rms_norm(y, (y.shape[1],)))
        self.accept_u, self.sample_u = torch.rand(R * (n + 1), device=dev), torch.rand(R, device=dev)
        nb.draft_verify(self.target, self.draft.flatten(0, 1), tokens, self.batch, self.accept_u,
                        self.sample_u, accepted=self.accepted, next_token=self.last,
                        cached=self.cached, ws=self.ws)

    def __call__(self):
        """One step: (tokens, accepted, last): of request r the tokens [r, 1 .. accepted[r]]
        stand, and last[r] follows them."""
        self.graph.replay()
        return self.tokens, self.accepted, self.last

    def status(self) -> int:
        return nb.read_status(self.ws) or self.step.status()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--new", type=int, default=64)
    ap.add_argument("--fp8-cache", action="store_true")
    ap.add_argument("--page-scales", action="store_true",
                    help="an E4M3 cache with a scale for each page and head")
    ap.add_argument("--drafts", type=int, default=0, help="tokens guessed a step")
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    # (drafted tokens that are turned down have had their places)
    total = args.prompt + args.new * (args.drafts + 1) + args.drafts + 1
    block = DecoderBlock(positions=total)
    hidden = block.w_in.numel()
    x = torch.randn(args.requests, args.prompt, hidden, device="cuda").bfloat16()

    def serve(chunk):
        pages = PageTable(args.requests, total, 64)
        cache = block.cache(pages, args.fp8_cache, args.page_scales)
        return prefill(block, cache, pages, x, chunk), pages, cache
    whole, _, _ = serve(args.prompt)
    y, pages, cache = serve(args.chunk)
    same = F.cosine_similarity(y.float(), whole.float(), dim=-1)
    print(f"prompts in chunks of {args.chunk} against whole: cosine {same.mean():.5f} on average, "
          f"{same.min():.5f} at least")

    if args.drafts:
        embed = F.normalize(torch.randn(2000, hidden, device="cuda")).bfloat16()
        decode = DraftedDecoder(block, cache, pages, embed, torch.arange(args.requests).int().cuda(),
                                args.drafts)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        stood = torch.zeros(args.requests, device="cuda")
        start.record()
        for _ in range(args.new):
            stood += decode()[1]
        end.record()
        torch.cuda.synchronize()
        if decode.status():
            raise RuntimeError(f"device status {decode.status()}")
        print(f"{args.new} steps of {args.drafts} drafted tokens for {args.requests} requests: "
              f"{start.elapsed_time(end) / args.new * 1e3:.0f} us a step, "
              f"{float(stood.mean()) / args.new:.2f} of them stand")
        return y, whole, decode.last
    decode = Decoder(block, cache, pages, args.requests, hidden)
    token = y[:, -1].contiguous()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(args.new):
        # a stand-in for sampling and embedding
        token = F.rms_norm(decode(token), (hidden,))
    end.record()
    torch.cuda.synchronize()
    if decode.step.status():
        raise RuntimeError(f"device status {decode.step.status()}")
    print(f"{args.new} tokens of {args.requests} requests at length {args.prompt}..{total}: "
          f"{start.elapsed_time(end) / args.new * 1e3:.0f} us a step")
    return y, whole, token


if __name__ == "__main__":
    main()
