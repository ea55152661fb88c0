"""Infinities and NaN in the adapters: they reach the rows and channels that the definition gives them, with its kind
and sign, and leave every other element the bits that it has without them -- in every form of the kernel: single CTAs, a
cluster that shares the sum, pairs of CTAs."""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_lora import call, problem

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


SHAPES = [
    (40, 64, 128, 3, 16),          # one short tile
    (32, 257, 1024, 24, 24),       # rows of many adapters, channels past the last lane tile
    (200, 384, 2048, 12, 64),      # several chunks of one accumulator
    (64, 256, 4096, 30, 40),       # a cluster shares the sum and the chunks
    (17, 136, 8224, 9, 128),
    (1100, 2304, 4128, 6, 64),     # pairs of CTAs
    (1100, 2310, 4128, 40, 16),    # and output rows that are not copied as tiles
]


def expected(p, rows, a):
    """What adapter a's term is made of, in 64 bits, by row and channel: [rows, N, R]."""
    t = p["s"][a].double() * (p["x"][rows].double() @ p["a"][a].double().t())
    return t[:, None, :] * p["b"][a].double()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,n,R", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_special_values_of_b(fmt, M, N, K, n, R, out_dtype):
    rng = np.random.default_rng(M + R)
    p = problem(fmt, M, N, K, n, R, rng.integers(-1, n, M), M * R)
    clean = call(fmt, p, out_dtype=out_dtype)
    # adapter 0: each kind alone; 1: two in one channel; the last: in its last channel and rank
    for a, c, r, v in ((0, 3, 1, INF), (0, 5, R - 1, -INF), (0, N - 1, 0, NAN), (1, 0, 0, INF), (1, 0, R - 2, INF),
                       (1, N // 2, 2, INF), (1, N // 2, 5, -INF), (n - 1, N - 1, R - 1, -INF)):
        p["b"][a, c, r] = v
    got = call(fmt, p, out_dtype=out_dtype)
    want = clean.clone()
    for a in {0, 1, n - 1}:
        rows = (p["ids"] == a).nonzero()[:, 0]
        hit = ~torch.isfinite(p["b"][a].float()).all(-1)
        term = expected(p, rows, a)[:, hit].sum(-1).to(out_dtype)
        assert not torch.isfinite(term.float()).any()
        want[rows[:, None], hit.nonzero()[:, 0]] = term
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0, INF, -INF), want.nan_to_num(7.0, INF, -INF))


@pytest.mark.parametrize("M,N,K,n,R", SHAPES)
def test_special_values_of_everything_else(M, N, K, n, R):
    """NaN and infinities in x, in A and in the scaling: the rows that use them, whole; no other row."""
    rng = np.random.default_rng(M)
    ids = rng.integers(-1, n, M)
    ids[:6] = [0, 1, -1, n - 1, 0, 1]
    p = problem("nvfp4", M, N, K, n, R, ids, M)
    clean = call("nvfp4", p)
    p["x"][0, 0], p["x"][2, K - 1] = NAN, NAN     # adapter 0's first row; a row without an adapter
    p["a"][1, R - 1, K - 1] = NAN
    p["s"][n - 1] = NAN
    got = call("nvfp4", p)
    hit = (p["ids"] == 1) | (p["ids"] == n - 1)
    hit[0] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert got[hit].isnan().all()
