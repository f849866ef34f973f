"""A decoder block on the attention operators and the NVFP4 experts, served step
by step: prompts in chunks, then single tokens replayed from a CUDA graph.

    python examples/decoder_block.py [--prompt 600] [--chunk 256] [--new 64] [--fp8-cache]

A step's launches are those of a serving loop: one product for q, k and v;
``kv_append`` (norm, rotation and append, queries in the same launch);
``paged_attention`` over the pages; the output product; ``router_topk`` and
``FusedLayer`` for the experts.  Weights are random, so it shows how the calls
fit together.  However a prompt is cut, the block gives the same answers up to the
experts' FP4 rounding: a step's activations share one global scale, from the largest
of them, so the grid that they are rounded to goes by the step.
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
    """Requests' pages from one pool, filled as the requests grow."""

    def __init__(self, requests: int, max_len: int, page_size: int, device="cuda"):
        self.page_size, self.device = page_size, device
        self.max_pages = -(-max_len // page_size)
        self.num_pages = requests * self.max_pages
        self.free = torch.randperm(self.num_pages).tolist()
        self.lengths = [0] * requests
        self.host = torch.zeros(requests, self.max_pages, dtype=torch.int32)
        self.table = self.host.to(device)
        self.kv_len = torch.zeros(requests, dtype=torch.int32, device=device)

    def grow(self, new):
        """new[r] more tokens for each request; the device tensors follow in place."""
        for r, n in enumerate(new):
            have = -(-self.lengths[r] // self.page_size)
            self.lengths[r] += n
            need = -(-self.lengths[r] // self.page_size)
            if need > self.max_pages:
                raise ValueError(f"request {r} has outgrown its pages")
            for p in range(have, need):
                self.host[r, p] = self.free.pop()
        self.table.copy_(self.host)
        self.kv_len.copy_(torch.tensor(self.lengths, dtype=torch.int32))


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

    def cache(self, pages: PageTable, fp8: bool = False) -> nb.PagedKVCache:
        shape = (pages.num_pages, pages.page_size, self.hk, self.D)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=pages.device).to(dtype)
                for _ in range(2))
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
        q_start = torch.arange(R + 1, dtype=torch.int32, device=x.device) * n
        batch = nb.AttnBatch(q_start, pages.kv_len, pages.table, max_new=n)
        step = Step(block, cache, batch, R * n)
        y[:, at:at + n] = step(x[:, at:at + n].reshape(R * n, -1)).view(R, n, -1)
        if step.status():
            raise RuntimeError(f"device status {step.status()}")
    return y


class Decoder:
    """One token of every request a step, replayed from a graph: the page table
    and the lengths are read on the device, so they may move under it."""

    def __init__(self, block, cache, pages, requests, hidden):
        q_start = torch.arange(requests + 1, dtype=torch.int32, device=pages.device)
        batch = nb.AttnBatch(q_start, pages.kv_len, pages.table, max_new=1)
        self.pages, self.step = pages, Step(block, cache, batch, requests)
        self.x = torch.zeros(requests, hidden, dtype=torch.bfloat16, device=pages.device)
        # warm-up and capture write at the requests' last positions; what they
        # leave there is put back, as nothing has been decoded yet
        saved = [(t, t.clone()) for t in (cache.k, cache.v)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(self.x)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.step(self.x)
        for t, old in saved:
            t.copy_(old)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        self.pages.grow([1] * x.shape[0])
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--new", type=int, default=64)
    ap.add_argument("--fp8-cache", action="store_true")
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    total = args.prompt + args.new
    block = DecoderBlock(positions=total)
    hidden = block.w_in.numel()
    x = torch.randn(args.requests, args.prompt, hidden, device="cuda").bfloat16()

    def serve(chunk):
        pages = PageTable(args.requests, total, 64)
        cache = block.cache(pages, args.fp8_cache)
        return prefill(block, cache, pages, x, chunk), pages, cache
    whole, _, _ = serve(args.prompt)
    y, pages, cache = serve(args.chunk)
    same = F.cosine_similarity(y.float(), whole.float(), dim=-1)
    print(f"prompts in chunks of {args.chunk} against whole: cosine {same.mean():.5f} on average, "
          f"{same.min():.5f} at least")

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
