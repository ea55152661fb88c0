"""The product of INT8 codes against the definition: sums of integers, two fp32 products, one rounding.

Tolerance.  While the sum of the products' magnitudes is below 2^24, every partial sum is exact in any order, and the
result is compared bit for bit.  Otherwise the fp32 sums round: with S the sum of the magnitudes, an element is off by
at most (K / 16 + 4) 2^-22 S (the tensor core adds 16 products at a time into the sum; 2^-22 allows for truncation and
for what is lost inside), and the two scales and the rounding add 2^-22 and (bf16) 2^-8 of the result.
"""
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def problem(M, N, K, seed, most=127):
    g = torch.Generator("cuda").manual_seed(seed)
    x, w = (torch.randint(-most, most + 1, (r, K), generator=g, device="cuda", dtype=torch.int8) for r in (M, N))
    xs, ws = (0.01 + torch.rand(r, generator=g, device="cuda") for r in (M, N))
    return x, xs, w, ws


def check(x, xs, w, ws, got):
    K = x.shape[1]
    sums = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    exact = ((sums.float() * xs[:, None]) * ws).to(got.dtype)
    want = sums * xs.double()[:, None] * ws.double()
    tol = (K / 16 + 4) * 2.0 ** -22 * size * xs.double()[:, None] * ws.double() + want.abs() * 2.0 ** -22
    if got.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8
    same = (got == exact) | (size >= 2 ** 24)
    assert same.all(), (int((~same).sum()), (~same).nonzero()[:4].tolist())
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off > tol).nonzero()[:4].tolist()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 4096, 4096), (2, 17, 32), (3, 130, 48), (16, 128, 64), (17, 129, 80), (31, 1100, 1056), (33, 257, 2064),
    (64, 300, 8192), (65, 100, 112), (128, 128, 128), (129, 256, 144), (200, 511, 4112), (255, 513, 1040), (256, 64, 16),
    (257, 640, 1024), (500, 1000, 528), (777, 1100, 1056), (1500, 264, 272), (4100, 96, 64), (1024, 2050, 512),
])
def test_sizes(M, N, K, out):
    x, xs, w, ws = problem(M, N, K, M + N + K)
    check(x, xs, w, ws, hq.hq_gemm_int8(x, xs, w, ws, out_dtype=out))


@pytest.mark.parametrize("M,N,K", [(48, 28672, 8192), (300, 40000, 4096), (4096, 4096, 8192), (1000, 9000, 2048), (40, 4096, 16384)])
def test_long_sums_over_more_tiles_than_places(M, N, K):
    """Stages go round the rings many times under a loaded memory, whose copies land in any order; again and again."""
    x, xs, w, ws = problem(M, N, K, 3, most=20)  # (400 * K < 2^24: exact)
    sums = torch.cat([x.double() @ v.double().t() for v in w.split(4096)], 1)
    want = ((sums.float() * xs[:, None]) * ws).to(torch.bfloat16)
    for _ in range(5):
        assert torch.equal(hq.hq_gemm_int8(x, xs, w, ws), want)


def test_every_code():
    """All pairs of codes, -128 among them (which the quantizer does not write)."""
    v = torch.arange(-128, 128, device="cuda", dtype=torch.int8)
    x = torch.zeros((256, 16), device="cuda", dtype=torch.int8)
    x[:, 5] = v
    one = torch.ones(256, device="cuda")
    got = hq.hq_gemm_int8(x, one, x, one, out_dtype=torch.float32)
    assert torch.equal(got, v.float()[:, None] * v.float())


@pytest.mark.parametrize("M", [3, 300])
def test_large_sums(M):
    """Codes of one sign: the sums leave 2^24."""
    K = 16384
    x, xs, w, ws = problem(M, 200, K, 5)
    x, w = x.abs().clamp(min=100), w.abs().clamp(min=100)
    check(x, xs, w, ws, hq.hq_gemm_int8(x, xs, w, ws, out_dtype=torch.float32))


def test_the_longest_sum():
    K = 2 ** 17 - 16
    x, xs, w, ws = problem(5, 40, K, 6, most=10)
    check(x, xs, w, ws, hq.hq_gemm_int8(x, xs, w, ws))


def test_small_codes_over_many_terms_are_exact():
    x, xs, w, ws = problem(300, 300, 65536, 7, most=15)  # (225 * 65536 < 2^24)
    got = hq.hq_gemm_int8(x, xs, w, ws, out_dtype=torch.float32)
    assert torch.equal(got, ((x.double() @ w.double().t()).float() * xs[:, None]) * ws)


def test_special_scales_stay_in_their_rows_and_columns():
    x, xs, w, ws = problem(70, 90, 256, 8)
    xs[3], xs[4], ws[5], ws[6] = float("inf"), float("nan"), float("-inf"), 0.0
    got = hq.hq_gemm_int8(x, xs, w, ws, out_dtype=torch.float32)
    want = ((x.double() @ w.double().t()).float() * xs[:, None]) * ws
    assert torch.equal(torch.nan_to_num(got, 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))


def test_empty():
    x, xs, w, ws = problem(0, 5, 32, 9)
    assert hq.hq_gemm_int8(x, xs, w, ws).shape == (0, 5)
    x, xs, w, ws = problem(4, 0, 32, 9)
    assert hq.hq_gemm_int8(x, xs, w, ws).shape == (4, 0)
    x, xs, w, ws = problem(4, 5, 0, 9)
    assert not hq.hq_gemm_int8(x, xs, w, ws).any()


def test_behind_the_quantizer():
    """x and weights rotated alike: the product of the codes is the product of the values, to the quantization."""
    g = torch.Generator("cuda").manual_seed(1)
    x, w = (torch.randn((r, 1024), generator=g, device="cuda") for r in (100, 300))
    got = hq.hq_gemm_int8(*hq.hq_rotate_quant_int8(x, 256), *hq.hq_rotate_quant_int8(w, 256), out_dtype=torch.float32)
    want = x @ w.t()
    # a code is off by half a step of amax / 127, amax below 6: 1024 products of errors of deviation 0.5 / sqrt(3) steps
    assert float((got - want).abs().max()) < 8 * 1024 ** 0.5 * (2 * 6 / 127) * 0.3


def test_misaligned_output_and_repeats():
    x, xs, w, ws = problem(40, 90, 512, 10)
    want = hq.hq_gemm_int8(x, xs, w, ws)
    room = torch.full((40 * 90 + 3,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = room[1:-2].view(40, 90)
    assert hq.hq_gemm_int8(x, xs, w, ws, out=out) is not None
    assert torch.equal(out, want) and room[0] == 7 and (room[-2:] == 7).all()
    for _ in range(3):
        assert torch.equal(hq.hq_gemm_int8(x, xs, w, ws), want)


def test_output_past_2_31_elements():
    M, N, K = 50000, 43008, 16
    x, xs, w, ws = problem(M, N, K, 11)
    got = hq.hq_gemm_int8(x, xs, w, ws)
    for r in (0, 1, 25000, M - 2, M - 1):
        assert torch.equal(got[r], (((x[r].double() @ w.double().t()).float() * xs[r]) * ws).to(torch.bfloat16))


def test_streams_and_graphs():
    x, xs, w, ws = problem(100, 260, 1024, 12)
    want = hq.hq_gemm_int8(x, xs, w, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hq.hq_gemm_int8(x, xs, w, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        hq.hq_gemm_int8(x, xs, w, ws, out=out)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, hq.hq_gemm_int8(x, xs, w, ws)) and torch.equal(out, -want)


def test_the_binding_refuses():
    x, xs, w, ws = problem(4, 6, 32, 13)
    for bad in ((x.int(), xs, w, ws), (x, xs[:3], w, ws), (x, xs, w[:, :16], ws), (x, xs, w, ws.double()), (x.cpu(), xs, w, ws),
                (x[0], xs, w, ws), (x, xs, w.t(), ws)):
        with pytest.raises(ValueError):
            hq.hq_gemm_int8(*bad)
    with pytest.raises(ValueError):
        hq.hq_gemm_int8(x, xs, w, ws, out_dtype=torch.half)
    with pytest.raises(hq.HQError):
        hq.hq_gemm_int8(x[:, :24].contiguous(), xs, w[:, :24].contiguous(), ws)
