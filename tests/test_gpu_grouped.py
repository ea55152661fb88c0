"""The products grouped by expert against the definition in 64 bits: ragged and empty groups, sizes that
divide nothing, both formats, both output types, the library's own quantizers in front.

Tolerance.  Products of codes and scales are exact and summed in fp32, one accumulation per 64 summed
elements: with S = sum |x w|, an element is off by at most (K / 64 + 4) 2^-22 S (each of the K / 64 partial
sums and the sum inside one step rounds, or truncates, to 24 bits of at most S; twice that is allowed), the
multiplication by the per-tensor scales adds 2^-23 of the result, and a bf16 output 2^-8 of it at most.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def values(q, s, sg, fmt):
    """float64 values of codes uint8 [.., K/2] and row-major scale bytes."""
    q = q.cpu().numpy()
    v = np.stack([GRID[q & 15], GRID[q >> 4]], -1).reshape(*q.shape[:-1], -1)
    if fmt == "nvfp4":
        s = s.view(torch.float8_e4m3fn).double().cpu().numpy() * sg
        return v * np.repeat(s, 16, -1)
    return v * np.repeat(2.0 ** (s.cpu().numpy().astype(np.float64) - 127), 32, -1)


def operand(shape, fmt, rng):
    """Random codes of every kind and scales over eight binades; row-major."""
    *lead, K = shape
    q = torch.from_numpy(rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)).cuda()
    if fmt == "nvfp4":
        s = torch.from_numpy(rng.uniform(2.0 ** -5, 8.0, (*lead, K // 16)).astype(np.float32)).cuda()
        return q, s.to(torch.float8_e4m3fn).view(torch.uint8)
    return q, torch.from_numpy(rng.integers(122, 131, (*lead, K // 32), dtype=np.uint8)).cuda()


def check(got, want, size, steps):
    """|got - want| within the bound above; `size` is the sum of the products' magnitudes."""
    out = got.double().cpu().numpy()
    tol = (steps + 4) * 2.0 ** -22 * size + np.abs(want) * (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23)
    bad = np.abs(out - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(out - want).max()))


def gemm(fmt, xq, xs, sx, wq, ws, sw, off, **kw):
    ws = hq.hq_swizzle_scales(ws)
    if fmt == "nvfp4":
        return hq.hq_grouped_gemm_nvfp4(xq, xs, sx, wq, ws, sw, off, **kw)
    return hq.hq_grouped_gemm_mxfp4(xq, xs, wq, ws, off, **kw)


def offsets_of(sizes):
    return torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32).cuda()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 1, 32),                        # one of everything
    ([1], 128, 256),                     # a single token
    ([0, 0, 5, 0], 130, 64),             # one expert of four, a lane tile of two
    ([16, 17, 15, 33], 96, 544),         # around the instruction's step of 16 columns, a partial K block
    ([64, 65, 1, 0, 200], 257, 1056),    # around the narrow tile, 66-byte (NVFP4) and 33-byte scale rows
    ([191, 192, 193, 385], 128, 512),    # around the wide tile
    ([700, 3, 0, 449], 384, 4128),       # several wide tiles per expert, 17 stages
    ([2] * 40 + [0] * 30 + [1] * 30, 72, 96),   # more groups than lanes of a warp
    ([5], 300, 8192),                    # few tiles: the summed axis shared by a cluster of 4
    ([0, 3, 64, 1], 130, 4640),          # of 2, uneven parts
    ([40], 200, 16416),                  # of 8, a last part with a partial block
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_grouped_gemm(fmt, sizes, N, K, out_dtype):
    rng = np.random.default_rng(hash((len(sizes), N, K)) % 2 ** 32)
    E, M = len(sizes), sum(sizes)
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((E, N, K), fmt, rng)
    sx = torch.tensor([0.37], device="cuda")
    sw = torch.linspace(0.5, 1.7, E, device="cuda")
    got = gemm(fmt, xq, xs, sx, wq, ws, sw, offsets_of(sizes), out_dtype=out_dtype)
    x = values(xq, xs, float(sx), fmt)
    at = 0
    want, size = np.zeros((M, N)), np.zeros((M, N))
    for e, n in enumerate(sizes):
        w = values(wq[e], ws[e], float(sw[e]), fmt)
        want[at:at + n] = x[at:at + n] @ w.T
        size[at:at + n] = np.abs(x[at:at + n]) @ np.abs(w).T
        at += n
    check(got, want, size, K / 64)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("sizes,N,K", [
    ([700, 3, 0, 449], 2100, 4128),            # several tiles per expert, a pair of lane tiles half empty
    ([191, 192, 193, 385, 64, 65], 1290, 4640),  # around the tile's width and its steps, no 16-byte rows of out
    ([40] * 64 + [0] * 5 + [1], 1000, 2048),   # many experts of one short tile each
    ([1300], 4104, 1056),                      # one group, a partial block, 66- and 33-byte scale rows
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_grouped_gemm_large(fmt, sizes, N, K, out_dtype):
    """Sizes that the pairs of CTAs take, whose scales are laid out in the workspace first."""
    assert hq.hq_grouped_gemm_workspace_bytes(sum(sizes), N, K, len(sizes)) > 0
    test_grouped_gemm(fmt, sizes, N, K, out_dtype)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_of_no_group_and_offsets_outside_the_tensor(fmt):
    """Rows past the last offset keep what they held; offsets beyond M are clamped to it."""
    rng = np.random.default_rng(3)
    M, N, K = 40, 64, 128
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((3, N, K), fmt, rng)
    one, ones = torch.ones(1, device="cuda"), torch.ones(3, device="cuda")
    out = torch.full((M, N), 7.0, device="cuda")
    gemm(fmt, xq, xs, one, wq, ws, ones, torch.tensor([0, 10, 10, 30], dtype=torch.int32).cuda(), out=out)
    assert (out[30:] == 7).all() and not (out[:30] == 7).all(1).any()
    x = values(xq, xs, 1.0, fmt)
    want = np.concatenate([x[:10] @ values(wq[0], ws[0], 1.0, fmt).T, x[10:30] @ values(wq[2], ws[2], 1.0, fmt).T])
    check(out[:30], want, np.abs(x[:30]) @ np.abs(values(wq, ws, 1.0, fmt)).max(0).T, K / 64)
    wild = gemm(fmt, xq, xs, one, wq, ws, ones, torch.tensor([-5, 10, 10, 9999], dtype=torch.int32).cuda(), out=out)
    assert torch.equal(wild[:30].cpu(), out[:30].cpu()) and (out != 7).any(1).all()
    check(wild[30:], x[30:] @ values(wq[2], ws[2], 1.0, fmt).T,
          np.abs(x[30:]) @ np.abs(values(wq[2], ws[2], 1.0, fmt)).T, K / 64)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_unaligned_scale_rows(fmt):
    """Scale rows at every alignment give the same bits as aligned ones."""
    rng = np.random.default_rng(5)
    M, N, K, E = 37, 70, 512, 2
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((E, N, K), fmt, rng)
    one, ones, off = torch.ones(1, device="cuda"), torch.ones(E, device="cuda"), offsets_of([20, 17])
    want = gemm(fmt, xq, xs, one, wq, ws, ones, off)
    for shift in (1, 2, 4, 8):
        buf = torch.empty(xs.numel() + 32, dtype=torch.uint8, device="cuda")
        moved = buf[shift:shift + xs.numel()].view_as(xs)
        moved.copy_(xs)
        assert torch.equal(gemm(fmt, xq, moved, one, wq, ws, ones, off), want)
    M, N, K = 1100, 2304, 4096  # and where they are laid out in a workspace
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((E, N, K), fmt, rng)
    off = offsets_of([500, 600])
    assert hq.hq_grouped_gemm_workspace_bytes(M, N, K, E) > 0
    want = gemm(fmt, xq, xs, one, wq, ws, ones, off)
    buf = torch.empty(xs.numel() + 32, dtype=torch.uint8, device="cuda")
    moved = buf[1:1 + xs.numel()].view_as(xs)
    moved.copy_(xs)
    assert torch.equal(gemm(fmt, xq, moved, one, wq, ws, ones, off), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_large_and_small_calls_give_the_same_bits(fmt):
    """The sum over K is made in the same steps by single CTAs and by pairs: a row's result does not depend on
    the rows beside it."""
    rng = np.random.default_rng(6)
    M, N, K = 1100, 2304, 4096
    xq, xs = operand((M, K), fmt, rng)
    wq, ws = operand((1, N, K), fmt, rng)
    one = torch.ones(1, device="cuda")
    large = gemm(fmt, xq, xs, one, wq, ws, one, offsets_of([M]), out_dtype=torch.float32)
    assert hq.hq_grouped_gemm_workspace_bytes(M, N, K, 1) > 0 == hq.hq_grouped_gemm_workspace_bytes(300, N, K, 1)
    small = gemm(fmt, xq[:300], xs[:300], one, wq, ws, one, offsets_of([300]), out_dtype=torch.float32)
    assert torch.equal(large[:300], small)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("units,N,K", [
    ([1], 1, 1),
    ([1, 0, 2], 100, 130),          # an expert without tokens: zeros
    ([3, 1, 4], 400, 520),          # several tiles of both operands, the second 64 rows into a scale tile
    ([0, 0], 64, 64),               # no tokens at all
    ([9], 192, 128),
])
def test_grouped_wgrad(fmt, out_dtype, units, N, K):
    rng = np.random.default_rng(N * 1000 + K)
    T = 128 * sum(units)
    gq, gs = operand((N, T), fmt, rng)
    xq, xs = operand((K, T), fmt, rng)
    sg, sx = torch.tensor([0.11], device="cuda"), torch.tensor([1.9], device="cuda")
    off = 128 * offsets_of(units)
    out = torch.full((len(units), N, K), float("nan"), dtype=out_dtype, device="cuda")
    gt, xt = hq.hq_swizzle_scales(gs), hq.hq_swizzle_scales(xs)
    if fmt == "nvfp4":
        got = hq.hq_grouped_wgrad_nvfp4(gq, gt, sg, xq, xt, sx, off, out=out)
    else:
        got = hq.hq_grouped_wgrad_mxfp4(gq, gt, xq, xt, off, out=out)
    assert got is out
    g, x = values(gq, gs, float(sg), fmt), values(xq, xs, float(sx), fmt)
    at = 0
    for e, u in enumerate(units):
        part = slice(at, at + 128 * u)
        check(got[e], g[:, part] @ x[:, part].T, np.abs(g[:, part]) @ np.abs(x[:, part]).T, 2 * u)
        at += 128 * u


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_swizzle_scales(fmt):
    import oracle

    rng = np.random.default_rng(8)
    s = rng.integers(0, 256, (3, 200, 22), dtype=np.uint8)
    got = hq.hq_swizzle_scales(torch.from_numpy(s).cuda()).cpu().numpy()
    for e in range(3):
        assert np.array_equal(got[e], oracle.swizzle_scales(s[e]).reshape(-1))


def test_offsets_past_32_bits_of_output():
    """Rows whose output lies past 2^32 elements."""
    rng = np.random.default_rng(9)
    M, N, K = 40_000, 110_000, 32
    xq, xs = operand((M, K), "nvfp4", rng)
    wq, ws = operand((1, N, K), "nvfp4", rng)
    one = torch.ones(1, device="cuda")
    got = gemm("nvfp4", xq, xs, one, wq, ws, one, offsets_of([M]))
    rows = [0, 39_000, 39_044, 39_999]  # 2^32 / 110000 = 39045.2
    x, w = values(xq[rows], xs[rows], 1.0, "nvfp4"), values(wq[0], ws[0], 1.0, "nvfp4")
    check(got[rows], x @ w.T, np.abs(x) @ np.abs(w).T, 1)


def test_training_step_of_an_expert_layer():
    """The three products of a step on the library's own operands, rotated along each summed axis:
    y = x w^T, dx = dy w, dw = dy^T x.  Each equals the product of the dequantized operands."""
    g = torch.Generator("cuda").manual_seed(1)
    sizes, N, K = [100, 0, 156], 160, 256
    M, E = sum(sizes), len(sizes)
    x = torch.randn(M, K, generator=g, device="cuda")
    w = torch.randn(E, N, K, generator=g, device="cuda")
    dy = torch.randn(M, N, generator=g, device="cuda")
    off = offsets_of(sizes)

    def quant(t):  # -> codes, row-major scales, per-tensor scale, float64 values of the rotated tensor
        q, s, sg, _ = hq.hq_quantize_nvfp4(t.contiguous(), 16)
        return q, s, sg, values(q, s, float(sg), "nvfp4")

    xq, xs, xg, xv = quant(x)
    parts = [quant(w[e]) for e in range(E)]
    y = hq.hq_grouped_gemm_nvfp4(xq, xs, xg, torch.stack([p[0] for p in parts]),
                                 hq.hq_swizzle_scales(torch.stack([p[1] for p in parts])),
                                 torch.cat([p[2] for p in parts]), off, out_dtype=torch.float32)
    yq, ys, yg, yv = quant(dy)
    back = [quant(w[e].t()) for e in range(E)]
    dx = hq.hq_grouped_gemm_nvfp4(yq, ys, yg, torch.stack([p[0] for p in back]),
                                  hq.hq_swizzle_scales(torch.stack([p[1] for p in back])),
                                  torch.cat([p[2] for p in back]), off, out_dtype=torch.float32)
    # tokens padded to 128 per expert, transposed
    pad = [(n + 127) // 128 * 128 for n in sizes]
    poff = offsets_of(pad)
    where = torch.cat([torch.arange(n) + int(poff[e]) for e, n in enumerate(sizes)]).cuda()
    xt, gt = torch.zeros(K, sum(pad), device="cuda"), torch.zeros(N, sum(pad), device="cuda")
    xt[:, where], gt[:, where] = x.t(), dy.t()
    (xq, xs, xg, xtv), (gq, gs, gg, gtv) = quant(xt), quant(gt)
    dw = hq.hq_grouped_wgrad_nvfp4(gq, hq.hq_swizzle_scales(gs), gg, xq, hq.hq_swizzle_scales(xs), xg, poff,
                                   out_dtype=torch.float32)
    at = 0
    for e, n in enumerate(sizes):
        r, p = slice(at, at + n), slice(int(poff[e]), int(poff[e + 1]))
        check(y[r], xv[r] @ parts[e][3].T, np.abs(xv[r]) @ np.abs(parts[e][3]).T, K / 64)
        check(dx[r], yv[r] @ back[e][3].T, np.abs(yv[r]) @ np.abs(back[e][3]).T, N / 64)
        check(dw[e], gtv[:, p] @ xtv[:, p].T, np.abs(gtv[:, p]) @ np.abs(xtv[:, p]).T, pad[e] / 64)
        at += n
        if n:  # and the products of the unquantized tensors, to what 4 bits can keep
            for got, true in ((y[r], x[r] @ w[e].t()), (dx[r], dy[r] @ w[e]), (dw[e], dy[r].t() @ x[r])):
                assert float((got - true).norm() / true.norm()) < 0.25


def test_streams_and_repeats():
    """The same call on two streams at once, each on its own inputs, gives what one stream gives, bit for bit."""
    rng = np.random.default_rng(12)
    sizes, N, K = [33, 100, 7], 500, 1024
    ops = []
    for _ in range(2):
        xq, xs = operand((140, K), "nvfp4", rng)
        wq, ws = operand((3, N, K), "nvfp4", rng)
        ops.append((xq, xs, torch.ones(1, device="cuda"), wq, hq.hq_swizzle_scales(ws), torch.ones(3, device="cuda")))
    off = offsets_of(sizes)
    want = [hq.hq_grouped_gemm_nvfp4(*o, off) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(3):
        got = []
        for o, s in zip(ops, streams):
            with torch.cuda.stream(s):
                got.append(hq.hq_grouped_gemm_nvfp4(*o, off))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
