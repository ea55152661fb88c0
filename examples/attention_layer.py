"""Causal attention of one layer in serving: INT8 projections around a paged NVFP4 cache.

    python examples/attention_layer.py

A step takes the tokens of some requests, whole prompts, parts of them or one token each, mixed as they come.
``hq_rotate_quant_int8`` and ``hq_gemm_int8`` project them to queries, keys and values; ``hq_kv_append_nvfp4`` turns
queries and keys to their positions, rotates all three and puts keys and values into the requests' pages;
``hq_kv_attention_nvfp4`` reads the pages; quantizer and product again project the result.  A step of one token each
has no size that depends on the requests' lengths, so it can be captured into a graph and replayed.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hadamard_rotation_gb300 as hq  # noqa: E402

ROTATE = 256  # groups of the projections' rotation
GROUP = 16    # of the cache's


def rotary_tables(rows, rotary, base=10000.0, device="cuda"):
    angle = torch.arange(rows, device=device)[:, None] * base ** (-torch.arange(rotary // 2, device=device) / (rotary // 2))
    return angle.cos(), angle.sin()


class Attention:
    """Weights qkv [(q_heads + 2 kv_heads) D, width] and o [width, q_heads D], bf16; their cache.

    ``kv_amax`` [2]: the largest rotated key and value that the cache is to hold without saturating."""

    def __init__(self, qkv, o, q_heads, kv_heads, D, kv_amax, pages, page_size=64, rows=4096):
        self.heads, self.D, self.page_size = (q_heads, kv_heads, kv_heads), D, page_size
        self.qkv, self.o = (hq.hq_rotate_quant_int8(w, ROTATE) for w in (qkv, o))
        self.tables = rotary_tables(rows, D, device=qkv.device)
        self.kv_amax = kv_amax
        self.cache = torch.zeros(pages, kv_heads, page_size // 16, 18 * D, dtype=torch.uint8, device=qkv.device)

    def project(self, x):
        """x [T, width] -> q [T, q_heads, D], k, v [T, kv_heads, D], views of one product."""
        y = hq.hq_gemm_int8(*hq.hq_rotate_quant_int8(x, ROTATE), *self.qkv)
        return (t.unflatten(1, (-1, self.D)) for t in y.split([h * self.D for h in self.heads], 1))

    def step(self, x, positions, slots, page_table, kv_len, q_start, max_q=None, out=None):
        """The layer's output [T, width] for T tokens; kv_len counts them too.  max_q, the most tokens of a request, chooses the
        attention's kernel for all of them: 1 for a step of single tokens (without it, they take three times as long)."""
        q = hq.hq_kv_append_nvfp4(*self.project(x), *self.tables, positions, slots, self.kv_amax, self.cache, GROUP)
        a = hq.hq_kv_attention_nvfp4(q, self.cache, page_table, kv_len, q_start, self.kv_amax, self.D ** -0.5, GROUP,
                                     max_q=max_q, out=out)
        return hq.hq_gemm_int8(*hq.hq_rotate_quant_int8(a.flatten(1), ROTATE), *self.o)


def places(page_table, page_size, before, new):
    """Of requests with ``before`` tokens in the cache and ``new`` ones (lists): a step's arguments."""
    dev = page_table.device
    at = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)]).to(dev)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(dev)
    slots = page_table[seq, at // page_size].long() * page_size + at % page_size
    kv_len = torch.tensor([b + n for b, n in zip(before, new)], dtype=torch.int32, device=dev)
    q_start = torch.tensor([0, *new]).cumsum(0).to(torch.int32).to(dev)
    return at.int(), slots, page_table, kv_len, q_start


def parameters(width, q_heads, kv_heads, D, seed=0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)

    def draw(*shape):
        return (torch.randn(*shape, generator=g, device=device) * shape[1] ** -0.5).to(torch.bfloat16)

    return draw((q_heads + 2 * kv_heads) * D, width), draw(width, q_heads * D)


class Decode:
    """A captured step of at most ``requests`` requests with a token each.  Request i is row i; idle ones come last."""

    def __init__(self, layer, requests, pages_each, width, device="cuda"):
        def new(*shape, dtype=torch.int32):
            return torch.zeros(*shape, dtype=dtype, device=device)

        self.x = new(requests, width, dtype=torch.bfloat16)
        self.positions, self.slots, self.kv_len = new(requests), new(requests, dtype=torch.int64) - 1, new(requests)
        self.page_table, self.q_start = new(requests, pages_each), new(requests + 1)
        self.out = new(requests, layer.heads[0], layer.D, dtype=torch.bfloat16)

        def step():
            return layer.step(self.x, self.positions, self.slots, self.page_table, self.kv_len, self.q_start, 1, self.out)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # (all idle: it stores nothing)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = step()

    def __call__(self, x, positions, slots, page_table, kv_len, q_start):
        n = len(x)
        self.x[:n], self.positions[:n], self.page_table[:n] = x, positions, page_table
        self.slots.fill_(-1)
        self.slots[:n] = slots
        self.kv_len.zero_()
        self.kv_len[:n] = kv_len
        self.q_start.fill_(n)
        self.q_start[:n + 1] = q_start
        self.graph.replay()
        return self.y[:n]


def main():
    width, q_heads, kv_heads, D, page_size = 512, 8, 2, 64, 16
    layer = Attention(*parameters(width, q_heads, kv_heads, D), q_heads, kv_heads, D, torch.full((2,), 6.0, device="cuda"), 64, page_size)
    page_table = torch.randperm(64, device="cuda").int()[:60].view(3, 20)
    before, new = [0, 0, 0], [200, 17, 64]
    x = torch.randn(sum(new), width, device="cuda").to(torch.bfloat16)
    y = layer.step(x, *places(page_table, page_size, before, new), max_q=max(new))
    print("prompts:", tuple(y.shape))
    decode = Decode(layer, 4, 20, width)
    x = y[torch.tensor(new).cumsum(0) - 1]  # (as if the layer's output were the next token)
    for _ in range(5):
        before, new = [b + n for b, n in zip(before, new)], [1, 1, 1]
        x = decode(x, *places(page_table, page_size, before, new))
    print("decoding:", tuple(x.shape), "lengths", [b + 1 for b in before])


if __name__ == "__main__":
    main()
