"""The adapters' first product where its CTAs share an SM's tensor memory: ranks whose columns round up to a quarter of
it, several passes over the adapters, several launches at once.  Tolerance: that of test_gpu_lora.py."""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_grouped import offsets_of, operand
from test_gpu_lora import call, check, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


SHAPES = [  # M, N, K, adapters, R
    (24, 256, 1024, 24, 72),    # 128 columns in 44 KB: five CTAs would fit on an SM by their shared memory
    (1, 128, 128, 1, 80),
    (24, 256, 4096, 24, 80),    # two adapters per CTA, two passes
    (128, 200, 2048, 100, 32),  # seven per CTA
    (128, 136, 96, 128, 128),   # a pass per adapter, a short sum
    (300, 300, 4096, 40, 64),   # rows of three tiles
]


def some(fmt, M, N, K, n, R, seed):
    return problem(fmt, M, N, K, n, R, np.random.default_rng(seed).integers(-1, n, M), seed)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,n,R", SHAPES)
def test_several_passes(fmt, M, N, K, n, R):
    p = some(fmt, M, N, K, n, R, M + R)
    check(fmt, p, call(fmt, p, out_dtype=torch.float32))


def test_launches_side_by_side():
    """Calls of different ranks on three streams, with large grouped products (all 512 columns) between them: every
    result is the one that the call gives alone, bit for bit."""
    ps = [some("nvfp4", *s, seed) for seed, s in enumerate(SHAPES[:4] + [(24, 256, 1024, 24, 8)])]
    rng = np.random.default_rng(1)
    M, N, K = 1100, 2304, 4096  # taken by pairs of CTAs
    xq, xs = operand((M, K), "nvfp4", rng)
    wq, ws = operand((2, N, K), "nvfp4", rng)
    one = torch.ones(1, device="cuda")
    wide = (xq, xs, one, wq, hq.hq_swizzle_scales(ws), one.repeat(2), offsets_of([500, 600]))
    want = [call("nvfp4", p) for p in ps]
    want_wide = hq.hq_grouped_gemm_nvfp4(*wide)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got, got_wide = [], []
        for i in range(20):
            with torch.cuda.stream(streams[i % 3]):
                got.append((i % len(ps), call("nvfp4", ps[i % len(ps)])))
                if i % 4 == 0:
                    got_wide.append(hq.hq_grouped_gemm_nvfp4(*wide))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[k]) for k, g in got)
        assert all(torch.equal(g, want_wide) for g in got_wide)
