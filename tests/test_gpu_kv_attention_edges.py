"""Attention over the paged cache where its plan, its hand-overs and its numbers are at their ends.  What is not said
here (the problems, the definition in 64 bits, the tolerances and their derivation) is in test_gpu_kv_attention.py.
"""
import math

import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_kv_attention import GRID, Problem, built, values  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,Hq,Hkv,D", [
    ([(1, 2000)] * 40 + [(1, 0)] * 24, 32, 8, 128),
    ([(1, 1500)] * 60 + [(1, 0)] * 2 + [(1, 1500)] * 40, 8, 8, 64),
    ([(1, 1200)] * 60 + [(1, 0)] * 60, 32, 8, 256),
    ([(5, 2500), (5, 0), (5, 0)] * 20, 8, 8, 64),
    ([(2, 1500)] * 60 + [(2, 0)] * 40, 40, 4, 256),
])
def test_queries_without_keys_among_others(seqs, Hq, Hkv, D):
    """Runs of items without records in a share that has others: more of them than the other warps are told of ahead."""
    p = Problem(seqs, Hq, Hkv, D, 64, seed=21)
    out, lse = p.call(out=torch.full_like(p.q, float("nan")))
    assert hq.hq_read_fault() == 0
    assert torch.isfinite(out).all()  # (all rows are written; a third of them are compared)
    p.check(out, lse, range(1, len(seqs), 3))


@pytest.mark.parametrize("D,group", [(64, 16), (128, 16)])
@pytest.mark.parametrize("seqs", [[(30, 500), (1, 100)], [(200, 500), (40, 128)]])  # one tile of rows at a time, two
@pytest.mark.parametrize("window", [0, 60, 400])
def test_scores_that_rise_within_a_tile_of_keys(D, group, seqs, window):
    """Keys 0..63 of each 128 small, the others large: references move between the halves of a tile, the first one's too;
    with a window rows see nothing of a first half."""
    p = Problem(seqs, 4, 1, D, 64, group=group, window=window, seed=22, scale=8 * D ** -0.5)
    for i, (_, n) in enumerate(seqs):
        p.cache[p.table[i, :-(-n // 64)][::2].long(), ..., 16 * D:17 * D] = 0x08  # K's scales: 2^-6
    p.run()


@pytest.mark.parametrize("seqs", [[(1400, 100), (1, 40)], [(3000, 2000)], [(2, 30), (1, 700)]])
@pytest.mark.parametrize("max_q", [1, 3000])  # the kernel for few rows, that for many
def test_windows_that_nothing_leaves(seqs, max_q):
    """Also behind queries that far outnumber the keys: the first of them stand 1000 places and more before key 0."""
    p = Problem(seqs, 2, 1, 64, 16, seed=23)
    want = p.call(max_q=max_q)
    p.check(*want)
    for window in (max(n for _, n in seqs), 2 ** 25, 2 ** 31 - 1500, 2 ** 31 - 1026, 2 ** 31 - 1025, 2 ** 31 - 1, 2 ** 62):
        p.window = window
        for a, b in zip(p.call(max_q=max_q), want):
            assert torch.equal(a, b), window


@pytest.mark.parametrize("D,group", [(64, 16), (128, 0), (256, 256)])
@pytest.mark.parametrize("seqs", [[(2, 1), (1, 0), (1, 300), (3, 40)], [(200, 150), (40, 0), (30, 700)]])  # few rows, many
@pytest.mark.parametrize("window", [0, 20])
def test_amax_and_scale_that_are_none(D, group, seqs, window):
    """A NaN amax of the keys or scale: NaN for all rows that see keys, whichever kernel takes them; of the values: the same,
    with the sums of weights as they are.  Rows without keys stay zeros."""
    p = Problem(seqs, 4, 2, D, 32, group=group, window=window, seed=24)
    want, want_lse = p.call()
    blind = want_lse == -math.inf
    assert blind.any() and not blind.all()
    amax, scale = p.kv_amax.clone(), p.scale
    for which in ("K", "V", "scale"):
        p.kv_amax, p.scale = amax.clone(), scale
        if which == "scale":
            p.scale = math.nan
        else:
            p.kv_amax["KV".index(which)] = math.nan
        out, lse = p.call()
        assert out[~blind].isnan().all() and not out[blind].any(), which
        assert (lse[blind] == -math.inf).all(), which
        assert torch.equal(lse, want_lse) if which == "V" else lse[~blind].isnan().all(), which


@pytest.mark.parametrize("size", [1e3, 3e7, 2e8, 5e9, 1e20, 2e30, 3e36])
@pytest.mark.parametrize("D,q", [(64, 1), (128, 4), (256, 1), (64, 30), (128, 30), (128, 200), (256, 200)])
def test_scores_of_any_magnitude(D, q, size):
    """Scores of `size` times one of E2M1's numbers and no two largest alike: the weights are 1 and 0.  The keys' first channel has
    the number, the queries' is the only one that is not zero, so a score is rounded as a product and not as a sum; the largest comes
    late or early, and is positive or negative.  out is the value itself (group 0, one rounding), lse the score to 2^-20."""
    n = 700
    for best, low, mid, high in ((650, 15, 3, 6), (5, 15, 3, 6), (300, 1, 3, 6), (100, 0, 3, 6), (650, 15, 14, 9), (3, 15, 14, 9)):
        p = Problem([(q, n)], 4, 2, D, 32, group=0, seed=25, scale=1.0, kv_amax=(6.0, 6.0), garbage=False)
        rec = p.cache[p.table[0, :-(-n // 32)].long()]  # [pages, heads, units, 18 D]
        rec[..., :8 * D] = 0
        rec[..., 16 * D:17 * D] = 0x38  # 1
        k = rec[..., :8 * D].unflatten(-1, (16, D // 2))  # (a view)
        number = torch.full((len(rec) * 32,), low, dtype=torch.uint8, device="cuda")
        number[64:90], number[best] = mid, high
        k[..., 0] = number.view(len(rec), 1, 2, 16)
        p.cache[p.table[0, :-(-n // 32)].long()] = rec
        p.q.zero_()
        p.q[..., 0] = torch.linspace(0.5, 1, p.T, device="cuda")[:, None].to(torch.bfloat16)
        p.scale = size
        out, lse = p.call()
        seen = torch.arange(n - q, n, device="cuda") >= best
        rows = seen.nonzero()[:, 0]
        assert len(rows)
        top = size * GRID[high] * p.q[rows, :, 0].double()
        assert ((lse[rows].double() - top).abs() <= 2.0 ** -20 * top.abs()).all(), (best, low)
        v = torch.stack([values(p.cache, p.table[0, :-(-n // 32)], h, n, 1, 1.0)[best] for h in (0, 0, 1, 1)])
        assert torch.equal(out[rows].double(), v.to(torch.bfloat16).double().expand(len(rows), -1, -1)), (best, low)


@pytest.mark.parametrize("D,q", [(64, 1), (128, 4), (256, 1), (64, 30), (128, 30), (128, 200), (256, 200)])
def test_scores_a_step_of_fp32_apart(D, q):
    """Scores of 2^10 to 2^33 that differ by fp32's step there, by a few of them or not at all, with one value behind every
    key: whatever its weights are, they add up to one, so out is that value (a weight's 2^-11 does not reach the rounding of a
    number of 5 bits to bf16's 8)."""
    n = 700
    p = Problem([(q, n)], 4, 2, D, 32, group=0, seed=26, scale=1.0, kv_amax=(6.0, 6.0), garbage=False)
    rec = p.cache[p.table[0, :-(-n // 32)].long()]
    rec[..., :8 * D] = 0
    rec[..., 16 * D:] = 0x38  # 1
    k, v = (rec[..., 8 * D * i:8 * D * (i + 1)].unflatten(-1, (16, D // 2)) for i in range(2))
    g = torch.Generator("cuda").manual_seed(27)
    # channel 0: 4, 2^10 as it is multiplied; channel 1: 0 to 6 times 2^-14, half of fp32's step there
    k[..., 0] = 6 | torch.randint(0, 8, k.shape[:-1], generator=g, device="cuda", dtype=torch.uint8) << 4
    v[:] = torch.randint(0, 256, (D // 2,), generator=g, device="cuda", dtype=torch.uint8)
    p.cache[p.table[0, :-(-n // 32)].long()] = rec
    want = values(p.cache, p.table[0, :-(-n // 32)], 0, n, 1, 1.0)[0].to(torch.bfloat16).expand(p.T, 4, D)
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.q[..., 1] = 2.0 ** -22  # (2^-14 where the first is 2^8: a number of f16)
    for e in range(10, 34):
        for m in (1.0, 1.37, 1.9):
            p.scale = m * 2.0 ** (e - 2)
            out, lse = p.call()
            assert torch.equal(out, want) and torch.isfinite(lse).all(), (e, m)


@pytest.mark.parametrize("seqs", [[(1, 900), (2, 70), (1, 0), (1, 300)], [(90, 200), (1, 30), (200, 700), (3, 3)]])
@pytest.mark.parametrize("D", [64, 256])
def test_the_most_sequences(seqs, D):
    """2^20 sequences, four of them with queries: the same shares and so the same bits as without the others."""
    p = Problem(seqs, 2, 1, D, 16, seed=28)
    want = p.call()
    S, at = 2 ** 20, [0, 5, 2 ** 19 + 3, 2 ** 20 - 1]
    table, kv_len = (torch.zeros((S, *t.shape[1:]), dtype=torch.int32, device="cuda") for t in (p.table, p.kv_len))
    counts = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
    for i, s in enumerate(at):
        table[s], kv_len[s], counts[s + 1] = p.table[i], p.kv_len[i], seqs[i][0]
    p.table, p.kv_len, p.q_start = table, kv_len, counts.cumsum(0).int()
    for a, b in zip(p.call(), want):
        assert torch.equal(a, b)
    assert hq.hq_read_fault() == 0


@pytest.mark.parametrize("D,group", [(64, 0), (64, 16), (128, 16), (256, 0), (256, 256)])
@pytest.mark.parametrize("window", [0, 24, 700])
@pytest.mark.parametrize("density", [0.04, 0.0003])  # of the blocks of 16 values
def test_many_nan_values(D, group, window, density):
    """NaN in any number of the values: the channels of the rows that see one, and nothing else, to the bit."""
    seqs, page = [(200, 3000), (700, 1530), (40, 41), (1, 600)], 48
    p = Problem(seqs, 2, 2, D, page, group, window, seed=29)
    base, spoiled, width = p.cache.clone(), p.cache.clone(), group or 16
    hit = torch.zeros((p.T, 2, D), dtype=torch.bool, device="cuda")
    g = torch.Generator("cuda").manual_seed(30)
    for i, (nq, n) in enumerate(seqs):
        bad = torch.rand((n, 2, D // 16), generator=g, device="cuda") < density
        bad[n // 2, 1, 0] = True
        t, h, b = bad.nonzero(as_tuple=True)
        at = (p.table[i, t // page].long(), h, t % page // 16, 17 * D + t % 16 * (D // 16) + b)
        base[at], spoiled[at] = 0, 0x7F
        pos, key = torch.arange(n - nq, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        seen = (key <= pos) & ((key > pos - window) if window else True)
        some = (seen.float() @ bad.flatten(1).float()).view(nq, 2, D // 16).repeat_interleave(16, -1) > 0
        hit[int(p.q_start[i]):int(p.q_start[i + 1])] = some.unflatten(-1, (-1, width)).any(-1, keepdim=True).expand(-1, -1, -1, width).flatten(2)
    p.cache = base
    want, want_lse = p.call()
    p.cache = spoiled
    got, lse = p.call()
    assert hit.any() and got[hit].isnan().all()
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("D,share,S,nq", [(256, 32, 1, 608), (64, 4, 152, 32)])
def test_a_nan_in_the_longest_context(D, share, S, nq):
    """2^25 keys, whole items of them: looking for the NaN ends before the other roles' waits do."""
    n, page = 2 ** 25, 4096
    cache = torch.randint(0, 256, (n // page, 1, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    cache[..., 16 * D:] = 0x38
    table = torch.arange(n // page, device="cuda").int().repeat(S, 1)
    q = torch.randn((S * nq, share, D), device="cuda").to(torch.bfloat16)
    kv_len = torch.full((S,), n, dtype=torch.int32, device="cuda")
    q_start = torch.arange(S + 1, device="cuda").int() * nq
    amax = torch.full((2,), 6.0, device="cuda")
    out = []
    for scale in (0, 0x7F):
        cache[0, 0, 0, 17 * D] = cache[-1, 0, -1, 18 * D - 1] = scale  # the first token's first block, the last one's last
        out.append(hq.hq_kv_attention_nvfp4(q, cache, table, kv_len, q_start, amax, D ** -0.5 / 16, group=0, max_q=nq))
    assert hq.hq_read_fault() == 0
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[..., :16] = True
    hit[nq - 1::nq, :, -16:] = True
    want, got = out
    assert got[hit].isnan().all() and torch.isfinite(want).all()
    assert torch.equal(got[~hit], want[~hit])
