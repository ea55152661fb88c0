"""Attention over the paged cache against the definition in 64 bits: head layouts, ragged and empty sequences, windows,
pages, long contexts, garbage behind the sequences' ends.

Tolerance.  With w the weights of a row, A = sum w |V| per channel and V's largest magnitude Vm:
  - a weight is carried in f16: half a step, 2^-11 of it, and where it leaves f16's normal range at most 2^-25 / 2^7 of
    the reference weight, which is at most 2^0 of the largest: n 2^-32 Vm for n keys;
  - a score is off by e = (D / 16 + 8) 2^-22 |scale| sum |q k| at most (D / 16 sums of the tensor core, the scales and
    the power of two's argument, which are products in fp32), and 2^-21 for ex2.approx and the argument's own
    rounding, relative to the weight; numerator and sum move by it, so twice;
  - sums over keys in fp32: (n / 16 + 64) 2^-23 of A twice (the tensor core's additions, the joining of parts).
The rotation back adds the errors of a block's channels with sign, so at most their sum over sqrt(group); the output's
rounding is 2^-8 of it.
lse: e, 2^-21, (n / 16 + 64) 2^-23 and 2^-22 of itself.
"""
import math

import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu

GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def hadamard(group):
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < group:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return (h / math.sqrt(group)).cuda()


def random_cache(pages, Hkv, page_size, D, seed, garbage=False):
    """Codes of every kind; scales over four binades.  garbage: any byte at all."""
    g = torch.Generator("cuda").manual_seed(seed)
    cache = torch.randint(0, 256, (pages, Hkv, page_size // 16, 18 * D), generator=g, device="cuda", dtype=torch.uint8)
    if not garbage:
        s = (2.0 ** (torch.rand((pages, Hkv, page_size // 16, 2 * D), generator=g, device="cuda") * 4 - 2)).to(torch.float8_e4m3fn)
        cache[..., 16 * D:] = s.view(torch.uint8)
    return cache


def values(cache, pages, head, n, which, sg):
    """float64 K (which = 0) or V of the first n tokens of the pages."""
    D = cache.shape[-1] // 18
    rec = cache[pages.long(), head].flatten(0, 1)
    codes = rec[:, 8 * D * which:8 * D * (which + 1)].reshape(-1, D // 2)[:n].long()
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    v = torch.stack([grid[codes & 15], grid[codes >> 4]], -1).flatten(1)
    s = rec[:, D * (16 + which):D * (17 + which)].reshape(-1, D // 16)[:n].contiguous().view(torch.float8_e4m3fn).double() * sg
    return v * s.repeat_interleave(16, 1)


class Problem:
    """Sequences of (queries, keys); `extra`: query rows before the first and behind the last sequence."""

    def __init__(self, seqs, Hq, Hkv, D, page_size, group=16, window=0, seed=0, extra=(0, 0), spread=1.0, scale=None, kv_amax=(3.0, 2.0),
                 garbage=True):
        g = torch.Generator("cuda").manual_seed(seed + 1)
        self.seqs, self.Hq, self.Hkv, self.D, self.group, self.window = seqs, Hq, Hkv, D, group, window
        need = [-(-n // page_size) for _, n in seqs]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.cache = random_cache(pages, Hkv, page_size, D, seed)
        if garbage:  # NaN scales and whatever else, where no token is
            bad = random_cache(pages, Hkv, page_size, D, seed + 7, garbage=True)
            bad[..., 16 * D:] = 0x7F
            token = torch.zeros((pages, page_size), dtype=torch.bool, device="cuda")
        most = max(need + [1])
        self.table = torch.full((len(seqs), most + 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda")[:, :most]
        at = 0
        for i, ((_, n), k) in enumerate(zip(seqs, need)):
            self.table[i, :k] = order[at:at + k]
            if garbage and n:
                flat = token[order[at:at + k].long()].flatten()
                flat[:n] = True
                token[order[at:at + k].long()] = flat.view(k, page_size)
            at += k
        if garbage:
            t = token.view(pages, 1, page_size // 16, 16)
            keep = torch.cat([t.repeat_interleave(D // 2, -1), t.repeat_interleave(D // 2, -1), t.repeat_interleave(D // 16, -1),
                              t.repeat_interleave(D // 16, -1)], -1).expand_as(self.cache)
            self.cache = torch.where(keep, self.cache, bad)
        starts = np.cumsum([extra[0]] + [q for q, _ in seqs])
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([n for _, n in seqs], dtype=torch.int32, device="cuda")
        self.T = int(starts[-1]) + extra[1]
        self.q = (torch.randn((self.T, Hq, D), generator=g, device="cuda") * spread).to(torch.bfloat16)
        self.kv_amax = torch.tensor(kv_amax, device="cuda") * 2688 / 6  # (values of codes up to 6 and scales up to 4)
        self.scale = D ** -0.5 / 16 if scale is None else scale
        self.max_q = max([q for q, _ in seqs] + [0])

    def call(self, **kw):
        kw = {"max_q": self.max_q, "return_lse": True, **kw}
        return hq.hq_kv_attention_nvfp4(self.q, self.cache, self.table, self.kv_len, self.q_start, self.kv_amax, self.scale,
                                        group=self.group, window=self.window, **kw)

    def check(self, out, lse, sequences=None):
        D, share = self.D, self.Hq // self.Hkv
        sg = (self.kv_amax.double().cpu().numpy() / 2688).astype(np.float32).astype(np.float64)
        H = hadamard(self.group) if self.group else None
        for i, (nq, n) in enumerate(self.seqs):
            if nq == 0 or (sequences is not None and i not in sequences):
                continue
            q0 = int(self.q_start[i])
            pos = torch.arange(n - nq, n, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None]
            seen = (key <= pos) & ((key > pos - self.window) if self.window else True)
            some = seen.any(1)
            for h in range(self.Hkv):
                k, v = (values(self.cache, self.table[i, :-(-n // (16 * self.cache.shape[2]))], h, n, w, sg[w]) for w in (0, 1))
                for head in range(h * share, (h + 1) * share):
                    q = self.q[q0:q0 + nq, head].double()
                    z = (q @ k.t() * self.scale).masked_fill(~seen, -math.inf)
                    e = ((D / 16 + 8) * 2.0 ** -22 * abs(self.scale) * (q.abs() @ k.abs().t())).masked_fill(~seen, 0)
                    e = e.amax(1) if n else torch.zeros(nq, device="cuda", dtype=torch.float64)
                    got, got_lse = out[q0:q0 + nq, head].double(), lse[q0:q0 + nq, head].double()
                    assert (got[~some] == 0).all() and (got_lse[~some] == -math.inf).all()
                    if not some.any():
                        continue
                    z, e, got, got_lse = z[some], e[some], got[some], got_lse[some]
                    want_lse = torch.logsumexp(z, 1)
                    sums = (n / 16 + 64) * 2.0 ** -23
                    assert ((got_lse - want_lse).abs() <= e + 2.0 ** -21 + sums + 2.0 ** -22 * want_lse.abs()).all()
                    w = torch.softmax(z, 1)
                    want = w @ v
                    tol = (2.0 ** -11 + 2 * (e[:, None] + 2.0 ** -21 + sums)) * (w @ v.abs()) * 1.01 + n * 2.0 ** -32 * v.abs().max()
                    if H is not None:
                        want = (want.unflatten(1, (-1, self.group)) @ H).flatten(1)
                        tol = (tol.unflatten(1, (-1, self.group)).sum(-1, keepdim=True) / math.sqrt(self.group)).expand(
                            -1, -1, self.group).flatten(1)
                    tol = tol + 2.0 ** -8 * want.abs()
                    off = (got - want).abs()
                    assert (off <= tol).all(), (i, head, (off > tol).nonzero()[:4].tolist(), float((off / tol).max()))

    def run(self, **kw):
        self.check(*self.call(**kw))


DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 33), (1, 100), (0, 40), (1, 250), (1, 1000), (0, 0), (1, 3)]


@pytest.mark.parametrize("Hq,Hkv,D,group", [(8, 1, 128, 16), (8, 2, 128, 0), (3, 3, 64, 16), (16, 1, 64, 16), (4, 2, 256, 256),
                                            (12, 1, 256, 16), (7, 1, 128, 16), (9, 1, 128, 16), (32, 1, 128, 16), (48, 2, 64, 0),
                                            (20, 1, 256, 0)])
@pytest.mark.parametrize("page_size", [16, 48, 64])
def test_one_token_each(Hq, Hkv, D, group, page_size):
    Problem(DECODE, Hq, Hkv, D, page_size, group=group, seed=Hq + D).run()


@pytest.mark.parametrize("D,group", [(64, 16), (128, 16), (256, 256)])
@pytest.mark.parametrize("window", [0, 1, 5, 16, 100])
def test_few_tokens_each(D, group, window):
    seqs = [(2, 2), (3, 50), (5, 200), (4, 333), (0, 10), (7, 16), (2, 129), (1, 64)]
    Problem(seqs, 4, 2, D, 32, group=group, window=window, seed=window).run()


@pytest.mark.parametrize("D,group", [(64, 0), (128, 16), (256, 16)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 1)])
def test_prompts(D, group, Hq, Hkv):
    seqs = [(1, 1), (17, 17), (130, 130), (64, 300), (257, 513), (40, 41), (0, 0)]
    Problem(seqs, Hq, Hkv, D, 16, group=group, seed=D + Hq).run()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 63, 128, 200])
def test_prompts_with_a_window(D, window):
    Problem([(200, 200), (100, 700), (3, 500), (1, 90)], 4, 2, D, 48, window=window, seed=window).run()


@pytest.mark.parametrize("D,group", [(64, 16), (128, 16), (128, 0)])
@pytest.mark.parametrize("Hq,Hkv,q", [(4, 1, 32), (2, 2, 128), (8, 1, 9), (6, 2, 42)])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_of_one_tile(D, group, Hq, Hkv, q, window):
    """33 to 128 rows of a sequence have a form of their own; sequences with more go through it in several tiles."""
    p = Problem([(q, q), (1, 700), (q - 3, 1500), (0, 9), (q, 260), (2 * q, 2 * q + 5)], Hq, Hkv, D, 32, group, window, seed=13)
    for max_q in (q, 2 * q, 10 ** 6):
        p.run(max_q=max_q)


def test_more_queries_than_keys():
    """The first queries stand before the first key: nothing to see."""
    p = Problem([(5, 3), (4, 0), (1, 0), (20, 7)], 4, 2, 64, 16, seed=3)
    p.run()
    p = Problem([(300, 170), (200, 0), (20, 7)], 4, 2, 128, 16, seed=3)
    p.run()


def test_rows_of_no_sequence_are_left():
    p = Problem([(2, 30), (1, 20)], 4, 2, 64, 16, extra=(3, 4), seed=4)
    out = torch.full((p.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = p.call(out=out)
    assert got.data_ptr() == out.data_ptr()
    p.check(out, lse)
    assert (out[:3] == 7).all() and (out[-4:] == 7).all()
    p = Problem([(150, 300), (1, 20)], 4, 2, 128, 16, extra=(3, 4), seed=4)
    out = torch.full((p.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    p.check(*p.call(out=out))
    assert (out[:3] == 7).all() and (out[-4:] == 7).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (2, 1, 256)])
def test_long_contexts(Hq, Hkv, D):
    """Items cut between many CTAs, several of them through one CTA's share."""
    Problem([(1, 20000), (1, 50), (2, 7000), (1, 1)], Hq, Hkv, D, 64, seed=8).run()


def test_many_sequences():
    rng = np.random.default_rng(0)
    seqs = [(int(q), int(q + n)) for q, n in zip(rng.integers(0, 3, 300), rng.integers(0, 90, 300))]
    Problem(seqs, 4, 2, 64, 16, seed=9).run()
    Problem([(1, 5)] * 1000, 2, 1, 64, 16, seed=10).run()


@pytest.mark.parametrize("page_size", [272, 4096])
def test_large_pages(page_size):
    Problem([(1, 1), (1, 300), (2, 5000)], 4, 2, 64, page_size).run()
    Problem([(100, 100), (40, 600)], 4, 2, 128, page_size).run()


def test_prompts_of_many_sequences():
    """More than the plan's sums hold at a time, most of them short or idle."""
    seqs = [(i % 3 if i % 7 else 0, i % 40 + 3) for i in range(1100)]
    seqs[0], seqs[600], seqs[1099] = (70, 70), (40, 300), (50, 51)
    Problem(seqs, 2, 1, 64, 16).run()


@pytest.mark.parametrize("seqs", [[(1, 100), (1, 900)], [(90, 300)]])
def test_a_cache_past_4_gigabytes(seqs):
    p = Problem(seqs, 4, 2, 128, 64)
    want = p.call()
    each = p.cache[0].numel()
    big = torch.empty((2 ** 32 // each + 50 + len(p.cache), *p.cache.shape[1:]), dtype=torch.uint8, device="cuda")
    big[-len(p.cache):] = p.cache
    for i, (_, n) in enumerate(seqs):
        p.table[i, :-(-n // 64)] += len(big) - len(p.cache)
    p.cache = big
    assert all(torch.equal(a, b) for a, b in zip(p.call(), want))


@pytest.mark.parametrize("max_q", [0, 1, 4, 1000, 10 ** 12])
def test_max_q_only_chooses(max_q):
    Problem([(9, 80), (1, 200), (70, 150)], 4, 2, 128, 16, seed=11).run(max_q=max_q)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 30.0, 300.0])
def test_flat_and_peaked_weights(spread):
    Problem([(1, 500), (3, 700), (130, 400)], 8, 2, 128, 16, spread=spread, seed=12).run()


def test_small_and_large_queries():
    for spread, scale in ((1e-30, 1e29), (1e25, 1e-27), (1e-37, 1e36)):
        Problem([(1, 300), (2, 90)], 4, 2, 64, 16, spread=spread, scale=scale, seed=13).run()
        Problem([(150, 300)], 4, 2, 64, 16, spread=spread, scale=scale, seed=13).run()


def test_negative_and_zero_scale():
    Problem([(1, 300), (2, 90), (140, 140)], 4, 2, 128, 16, scale=-0.01, seed=14).run()
    Problem([(1, 300), (2, 90), (140, 140)], 4, 2, 128, 16, scale=0.0, seed=14).run()


@pytest.mark.parametrize("D,group", [(64, 0), (64, 16), (128, 16), (256, 0), (256, 256)])
@pytest.mark.parametrize("seqs,Hq,Hkv", [([(1, 50), (1, 900)], 4, 2), ([(4, 70), (2, 1500), (3, 3)], 4, 1), ([(200, 200), (300, 900), (40, 41)], 4, 2),
                                         ([(1500, 4000)], 2, 1)])
@pytest.mark.parametrize("window", [0, 24])
def test_nan_reaches_the_rows_that_see_it(D, group, seqs, Hq, Hkv, window):
    """A NaN among the stored values: its channels (rotated back, its group's) of the rows that see its token, and nothing
    else, to the bit.  A NaN among the keys: all channels of the rows that see it, and no other row."""
    p = Problem(seqs, Hq, Hkv, D, 32, group, window, seed=11)
    clean, clean_lse = p.call()
    spoiled, base = p.cache.clone(), p.cache.clone()
    rng = np.random.default_rng(5)
    width = group or 16
    hit = torch.zeros_like(clean, dtype=torch.bool)
    blind = torch.zeros(p.T, Hq, dtype=torch.bool, device="cuda")  # rows that see a NaN key

    def rows(i, token):  # of the sequence, that see the token
        nq, n = seqs[i]
        pos = np.arange(n - nq, n)
        return int(p.q_start[i]) + np.nonzero((token <= pos) & ((token > pos - window) if window else True))[0]

    for i, (nq, n) in enumerate(seqs):
        for token in {n - 1, n // 2, max(0, n - nq), max(0, n - nq // 2 - 1), *rng.integers(0, n, 3).tolist()}:
            h, block = int(rng.integers(0, Hkv)), int(rng.integers(0, D // 16))
            page = int(p.table[i, token // 32])
            at = (page, h, token % 32 // 16, 17 * D + token % 16 * (D // 16) + block)
            spoiled[at] = 0x7F if token % 2 else 0xFF
            base[at] = 0  # (the rest of the row's sums, if they could be seen, are those of a zero)
            heads = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
            first = block * 16 // width * width
            for r in rows(i, token):
                hit[r, heads, first:first + width] = True
    p.cache = base
    want, want_lse = p.call()
    p.cache = spoiled
    got, lse = p.call()
    assert hit.any() and got[hit].isnan().all()
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse, want_lse)
    p.cache = base.clone()
    i = len(seqs) - 1
    token = seqs[i][1] - 1 - seqs[i][0] // 3
    p.cache[int(p.table[i, token // 32]), 0, token % 32 // 16, 16 * D + token % 16 * (D // 16)] = 0x7F
    for r in rows(i, token):
        blind[r, :Hq // Hkv] = True
    got, lse = p.call()
    assert blind.any() and got[blind].isnan().all() and lse[blind].isnan().all()
    assert not got[~blind].isnan().any()
    # (references move with other rows' scores: the sums differ by their rounding)
    assert ((got - want)[~blind].abs() <= 2 ** -7 * want[~blind].abs() + 2 ** -9 * want.abs().amax()).all()


def test_lengths_and_offsets_outside_are_clamped():
    p = Problem([(2, 30), (1, 64)], 4, 2, 64, 16, seed=15)
    want = p.call()
    p.kv_len[1] = 10 ** 9  # (its row of the table names 4 pages)
    for a, b in zip(p.call(), want):
        assert torch.equal(a, b)
    p.q_start[2] = 100
    for a, b in zip(p.call(), want):
        assert torch.equal(a, b)
    p.kv_len[:] = -5
    out, lse = p.call()
    assert not out.any() and (lse == -math.inf).all()


def test_strided_queries():
    p = Problem([(2, 30), (1, 64), (200, 250)], 4, 2, 64, 16, seed=16)
    want = p.call()
    wide = torch.randn((p.T, 7, 64), device="cuda").to(torch.bfloat16)
    wide[:, 2:6] = p.q
    p.q = wide[:, 2:6]
    for a, b in zip(p.call(), want):
        assert torch.equal(a, b)


def test_repeats_streams_and_graphs():
    p = Problem([(1, 3000), (1, 77), (2, 500)], 8, 2, 128, 16, seed=17)
    big = Problem([(300, 500), (2, 500)], 8, 2, 128, 16, seed=17)
    for r in (p, big):
        want = r.call()
        for _ in range(3):
            for a, b in zip(r.call(), want):
                assert torch.equal(a, b)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = r.call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = r.call()
        r.kv_len -= 20
        graph.replay()
        torch.cuda.synchronize()
        r.seqs = [(q, n - 20) for q, n in r.seqs]
        r.check(*got)


def test_nothing_to_do():
    p = Problem([(1, 20)], 4, 2, 64, 16)
    out = hq.hq_kv_attention_nvfp4(p.q[:0], p.cache, p.table, p.kv_len, torch.zeros(2, dtype=torch.int32, device="cuda"), p.kv_amax, 1.0)
    assert out.shape == (0, 4, 64)
    none = hq.hq_kv_attention_nvfp4(p.q, p.cache, p.table[:0], p.kv_len[:0], p.q_start[:1], p.kv_amax, 1.0,
                                    out=torch.full_like(p.q, 3.0))
    assert (none == 3).all()
    # a table without pages: sequences without keys
    out, lse = hq.hq_kv_attention_nvfp4(p.q, p.cache, p.table[:, :0], p.kv_len, p.q_start, p.kv_amax, 1.0, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()


def test_the_binding_refuses():
    p = Problem([(1, 20)], 4, 2, 64, 16)
    good = dict(q=p.q, cache=p.cache, page_table=p.table, kv_len=p.kv_len, q_start=p.q_start, kv_amax=p.kv_amax, scale=1.0)
    hq.hq_kv_attention_nvfp4(**good)
    for bad in (dict(q=p.q.float()), dict(q=p.q[:, :, :32]), dict(q=p.q[0]), dict(cache=p.cache.float()), dict(page_table=p.table.long()),
                dict(page_table=p.table[0]), dict(kv_len=p.kv_len.long()), dict(q_start=p.q_start[:1]), dict(kv_amax=p.kv_amax[:1]),
                dict(window=-1), dict(out=p.q.float()), dict(q=p.q.cpu())):
        with pytest.raises(ValueError):
            hq.hq_kv_attention_nvfp4(**{**good, **bad})
    for bad in (dict(group=32), dict(group=256), dict(q=torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises((hq.HQError, ValueError)):
            hq.hq_kv_attention_nvfp4(**{**good, **bad})
