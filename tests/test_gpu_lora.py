"""A shared projection with the adapters of many requests against the definition in 64 bits: ranks, row
orders, rows without an adapter, sizes that divide nothing.

Tolerance.  The projection's term as in test_gpu_grouped.py: (K / 64 + 4) 2^-22 of the sum of its products'
magnitudes.  The adapters': t = x A^T is summed in fp32 over K terms in chunks of 16 (K / 16 roundings, 2^-22
allowed for each), carried in two bf16 terms (2^-16 of it), and multiplied into the accumulator by R exact
products per term; with U = |s| (|x| |A|^T) |B|^T that is under (K / 16 2^-22 + 2^-16 + 2^-20) U, taken once more
for the accumulator's own additions.  A bf16 output adds 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_grouped import operand, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def problem(fmt, M, N, K, n, R, ids, seed):
    rng = np.random.default_rng(seed)
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((N, K), fmt, rng)
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return dict(xq=xq, xs=xs, sx=torch.tensor([0.013], device="cuda"), wq=wq, ws=ws,
                sw=torch.tensor([0.7], device="cuda"), x=r(M, K).to(torch.bfloat16), a=r(n, R, K).to(torch.bfloat16),
                b=r(n, N, R).to(torch.bfloat16), s=0.5 + r(n).abs(),
                ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))


def call(fmt, p, **kw):
    tiles = hq.hq_swizzle_scales(p["ws"])
    if fmt == "nvfp4":
        return hq.hq_lora_gemm_nvfp4(p["xq"], p["xs"], p["sx"], p["wq"], tiles, p["sw"], p["x"], p["a"], p["b"], p["s"],
                                     p["ids"], **kw)
    return hq.hq_lora_gemm_mxfp4(p["xq"], p["xs"], p["wq"], tiles, p["x"], p["a"], p["b"], p["s"], p["ids"], **kw)


def check(fmt, p, got):
    K, n = p["x"].shape[1], p["a"].shape[0]
    xv = torch.from_numpy(values(p["xq"], p["xs"], float(p["sx"]), fmt)).cuda()
    wv = torch.from_numpy(values(p["wq"], p["ws"], float(p["sw"]), fmt)).cuda()
    want = xv @ wv.t()
    tol = (K / 64 + 4) * 2.0 ** -22 * (xv.abs() @ wv.abs().t())
    for k in range(n):
        rows = (p["ids"] == k).nonzero()[:, 0]
        x, a, b, s = p["x"][rows].double(), p["a"][k].double(), p["b"][k].double(), p["s"][k].double()
        want[rows] += s * (x @ a.t()) @ b.t()
        tol[rows] += 2 * (K / 16 * 2.0 ** -22 + 2.0 ** -16 + 2.0 ** -20) * s * (x.abs() @ a.abs().t()) @ b.abs().t()
    if got.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * want.abs()
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), (off > tol).nonzero()[:4].tolist(), float((off / tol).max()))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,n,R,order", [
    (1, 8, 32, 1, 8, "one"),             # the smallest
    (1, 300, 544, 3, 16, "one"),
    (32, 257, 1024, 24, 16, "mixed"),    # every row its own
    (17, 136, 8224, 9, 40, "mixed"),     # few tiles: sum and adapters shared by a cluster of 4
    (64, 256, 4096, 64, 16, "mixed"),    # of 2, every row its own
    (33, 128, 96, 40, 8, "mixed"),       # one row past the narrow row tile of the first product
    (64, 130, 512, 5, 24, "mixed"),      # a rank that is not a multiple of 16
    (65, 100, 1056, 2, 64, "runs"),      # past the narrow tile of the projection
    (200, 384, 2048, 64, 16, "mixed"),   # many adapters in a wide tile
    (500, 200, 4128, 6, 128, "runs"),    # two rank blocks
    (391, 128, 64, 3, 40, "sorted"),     # a short sum beside many chunks
    (130, 136, 256, 4, 72, "none"),      # no row has one
    (1100, 2304, 4128, 6, 64, "runs"),   # pairs of CTAs
    (1030, 4104, 2048, 64, 24, "mixed"),  # as many adapters as chunks hold, several times over
    (1300, 3336, 2080, 3, 128, "none"),
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_against_64_bits(fmt, M, N, K, n, R, order, out_dtype):
    rng = np.random.default_rng(M + N)
    ids = {"one": np.full(M, n - 1), "mixed": rng.integers(-1, n, M), "sorted": np.sort(rng.integers(-1, n, M)),
           "runs": np.repeat(rng.integers(-1, n, M), 37)[:M], "none": np.full(M, -1)}[order]
    p = problem(fmt, M, N, K, n, R, ids, M * N)
    check(fmt, p, call(fmt, p, out_dtype=out_dtype))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_no_adapters_is_the_projection(fmt):
    """Ids outside the adapters, or no adapters at all: the bits of the product without them."""
    M, N, K = 70, 200, 288
    p = problem(fmt, M, N, K, 2, 16, [-1, 2, 99, -7, 2 ** 31 - 1] * 14, 4)
    p["b"].fill_(float("nan"))  # never read
    off = torch.tensor([0, M], dtype=torch.int32).cuda()
    tiles = hq.hq_swizzle_scales(p["ws"])[None]
    want = hq.hq_grouped_gemm_nvfp4(p["xq"], p["xs"], p["sx"], p["wq"][None], tiles, p["sw"], off) if fmt == "nvfp4" \
        else hq.hq_grouped_gemm_mxfp4(p["xq"], p["xs"], p["wq"][None], tiles, off)
    assert torch.equal(call(fmt, p), want)
    p["a"], p["b"], p["s"] = (p[k][:0].contiguous() for k in "abs")
    assert torch.equal(call(fmt, p), want)


def test_another_rows_infinity_stays_there():
    """Infinities and NaN in x, and in an adapter, reach the rows that use them and no other."""
    M, N, K = 40, 64, 128
    p = problem("nvfp4", M, N, K, 3, 16, [0, 1, -1, 2] * 10, 6)
    clean = call("nvfp4", p)
    p["x"][2] = float("nan")       # no adapter: x itself is not read into the result
    p["x"][4] = float("inf")       # adapter 0
    p["a"][2] = float("nan")       # adapter 2: rows 3, 7, ..
    got = call("nvfp4", p)
    hit = torch.zeros(M, dtype=torch.bool, device="cuda")
    hit[4], hit[3::4] = True, True
    assert torch.equal(got[~hit], clean[~hit])
    assert not torch.isfinite(got[hit].float()).any()


def test_strided_x_streams_and_repeats():
    M, N, K = 150, 320, 512
    p = problem("nvfp4", M, N, K, 9, 32, np.random.default_rng(0).integers(-1, 9, M), 8)
    want = call("nvfp4", p)
    wide = torch.full((M, K + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = p["x"]
    assert torch.equal(call("nvfp4", dict(p, x=wide[:, 8:8 + K])), want)
    ps = [p, problem("nvfp4", M, N, K, 9, 32, np.random.default_rng(1).integers(-1, 9, M), 9)]
    wants = [want, call("nvfp4", ps[1])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(3):
        got = []
        for q, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(call("nvfp4", q))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, wants))


def test_on_the_librarys_quantized_rotated_operands():
    """x and w rotated and quantized by the library, the adapters on x itself: near the product in full
    precision, nearer than without the adapters by what they add."""
    g = torch.Generator("cuda").manual_seed(0)
    M, N, K, R = 96, 256, 512, 16
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5
    a = (torch.randn(2, R, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    b = torch.randn(2, N, R, generator=g, device="cuda").to(torch.bfloat16)
    ids = (torch.arange(M, device="cuda", dtype=torch.int32) // 20) % 2
    xq, xs, xg, _ = hq.hq_quantize_nvfp4(x, 256)
    wq, ws, wg, _ = hq.hq_quantize_nvfp4(w, 256)
    y = hq.hq_lora_gemm_nvfp4(xq, xs, xg, wq, hq.hq_swizzle_scales(ws), wg, x, a, b, torch.ones(2, device="cuda"), ids,
                              out_dtype=torch.float32)
    extra = torch.stack([(x[m].float() @ a[ids[m]].float().t()) @ b[ids[m]].float().t() for m in range(M)])
    true = x.float() @ w.t() + extra
    assert float((y - true).norm() / true.norm()) < 0.1
    assert float(extra.norm() / true.norm()) > 0.5
