"""The INT8 projections, the paged cache and the attention over it together, as the example's layer runs them: prompts,
parts of prompts, single tokens, mixed, captured, on two streams, against a plain layer.

Tolerances.  INT8 codes of rotated, normally distributed rows of some 500 values have steps of amax / 127, amax about
3.3 to 4 deviations: rms error (4 / 127) / sqrt(12) = 0.009 of a value, 0.013 of a product of two.  NVFP4 codes of such
values have 0.095: a key's error moves a score of deviation s by 0.095 s, and its weight by as much of itself; with the
values' own error the output of the attention is off by 0.095 sqrt(1 + s^2) of its norm.  Scores here have s = 1 (queries
and keys of unit variance, scale D^-1/2), so 0.135; with both projections 0.137.  0.2 is allowed.
Between two ways to run the same tokens the cache is the same to the bit, since the INT8 sums are exact (512 * 127^2 < 2^24)
and rows do not depend on one another; attention's outputs then differ by their rounding to bf16 (2 * 2^-9 in norm at most
with the weights' 2^-11), and that by at most as many INT8 steps behind it as the rounding turns: 2^-7 + 0.009.
"""
import os
import sys

import pytest
import torch

import hadamard_rotation_gb300 as hq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
WIDTH, ROWS = 512, 1024


@pytest.fixture(scope="module")
def example():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    import attention_layer

    yield attention_layer
    assert hq.hq_read_fault() == 0


def make(example, q_heads, kv_heads, D, page_size, requests, pages_each, seed=0):
    qkv, o = example.parameters(WIDTH, q_heads, kv_heads, D, seed)
    pages = requests * pages_each + 3
    g = torch.Generator("cuda").manual_seed(seed)
    layer = example.Attention(qkv, o, q_heads, kv_heads, D, torch.full((2,), 7.0, device="cuda"), pages, page_size, ROWS)
    table = torch.randperm(pages, generator=g, device="cuda").int()[:requests * pages_each].view(requests, pages_each)
    return layer, table, (qkv.float(), o.float())


def plain(example, layer, weights, x):
    """One request's whole layer in fp32."""
    Hq, Hkv, _ = layer.heads
    D, T = layer.D, len(x)
    q, k, v = (t.unflatten(1, (-1, D)) for t in (x.float() @ weights[0].t()).split([h * D for h in layer.heads], 1))
    cos, sin = (t[:T, None] for t in layer.tables)

    def turn(t):
        a, b = t.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = turn(q), turn(k)
    k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(T, T, device="cuda", dtype=torch.bool).triu(1), -torch.inf)
    return torch.einsum("hqk,khd->qhd", s.softmax(-1), v).flatten(1) @ weights[1].t()


def off(got, want):
    return float((got.float() - want.float()).norm() / want.float().norm())


def tokens(n, seed):
    return torch.randn(n, WIDTH, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


SHAPES = [(8, 2, 64, 16), (4, 1, 128, 48), (2, 2, 256, 64)]


@pytest.mark.parametrize("q_heads,kv_heads,D,page_size", SHAPES)
def test_prompts_against_a_plain_layer(example, q_heads, kv_heads, D, page_size):
    lens = [300, 1, 77]
    layer, table, w = make(example, q_heads, kv_heads, D, page_size, 3, 320 // page_size + 1)
    x = tokens(sum(lens), 1)
    got = layer.step(x, *example.places(table, page_size, [0] * 3, lens))
    for a, b in zip(got.split(lens), x.split(lens)):
        assert off(a, plain(example, layer, w, b)) < 0.2


@pytest.mark.parametrize("q_heads,kv_heads,D,page_size", SHAPES)
def test_parts_and_single_tokens_leave_the_same_cache(example, q_heads, kv_heads, D, page_size):
    lens, each = [300, 40, 77], 320 // page_size + 1
    layer, table, _ = make(example, q_heads, kv_heads, D, page_size, 3, each)
    other, _, _ = make(example, q_heads, kv_heads, D, page_size, 3, each)
    x = tokens(sum(lens), 2)
    want = layer.step(x, *example.places(table, page_size, [0] * 3, lens))
    rows, got = x.split(lens), [[], [], []]
    before = [0, 0, 0]
    for new in ([200, 1, 60], [1, 35, 1], [40, 0, 15], [58, 3, 0], *[[int(s == 0), int(s == 1), int(s == 2)] for s in (2, 0, 1)]):
        part = torch.cat([r[b:b + n] for r, b, n in zip(rows, before, new)])
        y = other.step(part, *example.places(table, page_size, before, new))
        for g, t in zip(got, y.split(new)):
            g.append(t)
        before = [b + n for b, n in zip(before, new)]
    assert before == lens
    assert torch.equal(other.cache, layer.cache)
    for a, b in zip(got, want.split(lens)):
        assert off(torch.cat(a), b) < 2 ** -7 + 0.009


def test_captured_steps_with_idle_rows(example):
    q_heads, kv_heads, D, page_size = 8, 2, 128, 32
    lens = [100, 31, 5]
    layer, table, _ = make(example, q_heads, kv_heads, D, page_size, 3, 8)
    twin, _, _ = make(example, q_heads, kv_heads, D, page_size, 3, 8)
    x = tokens(sum(lens), 3)
    for t in (layer, twin):
        t.step(x, *example.places(table, page_size, [0] * 3, lens))
    decode = example.Decode(layer, 5, 8, WIDTH)
    assert torch.equal(layer.cache, twin.cache)  # (capturing stores nothing)
    again = example.Decode(layer, 2, 8, WIDTH)   # a second graph on the same cache, with buffers of its own
    before = lens
    for i in range(40):
        n = 3 if i % 3 else 2
        run = decode if n == 3 or i % 2 else again
        x, args = tokens(n, 10 + i), example.places(table[:n], page_size, before[:n], [1] * n)
        got = run(x, *args).clone()
        want = twin.step(x, *args, max_q=1)
        assert torch.equal(got, want)
        before = [b + (s < n) for s, b in enumerate(before)]
    assert torch.equal(layer.cache, twin.cache)


def test_two_streams_at_once(example):
    q_heads, kv_heads, D, page_size = 8, 2, 128, 64
    lens = [700, 300]
    layers = [make(example, q_heads, kv_heads, D, page_size, 2, 12, seed) for seed in (0, 1)]
    x = tokens(sum(lens), 4)
    args = [example.places(t, page_size, [0, 0], lens) for _, t, _ in layers]
    want = [layer.step(x, *a) for (layer, _, _), a in zip(layers, args)]
    one = [layer.cache.clone() for layer, _, _ in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for (layer, _, _), a, s, g in zip(layers, args, streams, got):
            with torch.cuda.stream(s):
                g.append(layer.step(x, *a))
    torch.cuda.synchronize()
    for g, w, c, (layer, _, _) in zip(got, want, one, layers):
        assert all(torch.equal(t, w) for t in g)
        assert torch.equal(layer.cache, c)


def test_main_runs(example, capsys):
    example.main()
    text = capsys.readouterr().out
    assert "prompts: (281, 512)" in text and "decoding: (3, 512) lengths [205, 22, 69]" in text
