"""Appending to the paged cache: bytes against the oracle's quantizer on position-rotated values, q against the same
butterfly, reading back, slots, pages, strides.

Everything is compared bit for bit: the position rotation is two products and a sum, each rounded to fp32, which numpy
does alike, and the rest is the oracle's.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built(oracle_lib):
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def tables(rows, rotary, seed=0):
    angle = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rotary // 2) / max(1, rotary // 2))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def turned(x, cos, sin, positions, rotary, interleaved):
    """The position rotation of x [T, heads, D] in fp32, numpy."""
    x = x.astype(np.float32)
    if not rotary:
        return x
    at = np.clip(positions, 0, len(cos) - 1)
    c, s = cos[at][:, None], sin[at][:, None]
    y = x.copy()
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2), slice(rotary // 2, rotary))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def to_bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16)


def place(cache, slot, head, page_size, D):
    """K codes, V codes, K scales, V scales of a token in a cache (numpy)."""
    rec = cache[slot // page_size, head, slot % page_size // 16]
    t = slot % 16
    kc, vc, ks, vs = np.split(rec, [8 * D, 16 * D, 17 * D])
    return kc.reshape(16, -1)[t], vc.reshape(16, -1)[t], ks.reshape(16, -1)[t], vs.reshape(16, -1)[t]


def check(oracle, T, Hq, Hkv, D, page_size, rotary, interleaved, group, dtype, slots=None, pages=None, fused=True, rows=5000, seed=0,
          scale=1.0, kv_amax=None, positions=None):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * scale).astype(np.float32)).to(dtype).cuda()
    if fused:
        q, k, v = (t.unflatten(1, (-1, D)) if t.shape[1] else None for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (t.unflatten(1, (-1, D)).contiguous() if t.shape[1] else None for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    pages = pages or (T + page_size - 1) // page_size + 1
    if slots is None:
        slots = rng.permutation(pages * page_size)[:T]
    slots = np.asarray(slots, np.int64)
    if positions is None:
        positions = rng.integers(0, rows, T).astype(np.int32)
    cos, sin = tables(rows, rotary)
    if kv_amax is None:
        kv_amax = [float(k.float().abs().max()) * 1.5, float(v.float().abs().max()) * 0.7]
    before = torch.from_numpy(rng.integers(0, 256, (pages, Hkv, page_size // 16, 18 * D), dtype=np.uint8))
    cache = before.cuda()
    args = [torch.from_numpy(t).cuda() for t in (cos, sin, positions)] if rotary else [None] * 3
    amax = torch.tensor(kv_amax, dtype=torch.float32, device="cuda")
    out = hq.hq_kv_append_nvfp4(q, k, v, *args, torch.from_numpy(slots).cuda(), amax, cache, group=group, interleaved=interleaved)
    got = cache.cpu().numpy()
    want = before.numpy().copy()

    def rows_of(t):
        return t.float().cpu().numpy()

    if Hq:
        y = turned(rows_of(q), cos, sin, positions, rotary, interleaved).reshape(T * Hq, D)
        if group:
            y = oracle.rot_amax(y, group, want_y=True)[1]
        assert torch.equal(out.cpu().view(torch.int16), to_bf16(y.reshape(T, Hq, D)).view(torch.int16))
    else:
        assert out is None
    kv = [turned(rows_of(k), cos, sin, positions, rotary, interleaved), rows_of(v)]
    parts = [oracle.quantize(np.ascontiguousarray(t.reshape(T * Hkv, D)), group, amax=a)[:2]
             for t, a in zip(kv, amax.cpu().numpy())]
    for t in range(T):
        if not 0 <= slots[t] < pages * page_size:
            continue
        for h in range(Hkv):
            dst = place(want, int(slots[t]), h, page_size, D)
            for to, src in zip(dst, (parts[0][0], parts[1][0], parts[0][1], parts[1][1])):
                to[:] = src[t * Hkv + h]
    assert np.array_equal(got, want)
    # and back
    sg = [oracle.global_scale(float(a)) for a in amax.cpu().numpy()]
    for g, dt in ((0, torch.float32), (0, torch.bfloat16), (group, torch.float32)):
        back = hq.hq_kv_read_nvfp4(cache, torch.from_numpy(slots).cuda(), amax, group=g, out_dtype=dt)
        live = ((slots >= 0) & (slots < pages * page_size))[:, None, None]
        for b, (codes, scales), s in zip(back, parts, sg):
            val = np.where(live, oracle.dequant(codes, scales, s, g or 16, bool(g)).reshape(T, Hkv, D), np.float32(0))
            same = torch.from_numpy(val).to(dt)
            assert torch.equal(b.cpu().float(), same.float())


@pytest.mark.parametrize("D,group", [(64, 0), (64, 16), (128, 0), (128, 16), (256, 0), (256, 16), (256, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes_and_types(oracle_lib, D, group, dtype, interleaved):
    check(oracle_lib, 37, 6, 3, D, 32, D, interleaved, group, dtype)
    check(oracle_lib, 5, 4, 1, D, 16, 48, interleaved, group, dtype, seed=1)   # (an odd count of 8-channel pieces in a half)
    check(oracle_lib, 3, 2, 2, D, 48, 16, interleaved, group, dtype, seed=2)


@pytest.mark.parametrize("T,Hq,Hkv,page_size", [(1, 1, 1, 16), (1, 32, 8, 64), (200, 0, 5, 80), (63, 7, 7, 256), (700, 3, 1, 128)])
def test_tokens_and_heads(oracle_lib, T, Hq, Hkv, page_size):
    check(oracle_lib, T, Hq, Hkv, 128, page_size, 128, False, 16, torch.bfloat16, fused=T % 2 == 0)


def test_no_position_rotation(oracle_lib):
    check(oracle_lib, 20, 4, 2, 64, 16, 0, False, 16, torch.bfloat16)


def test_slots_that_are_none_and_positions_past_the_tables(oracle_lib):
    slots = [-1, 5, 40, -(2 ** 40), 2 ** 40, 80, 79, 81, -1, 0]  # (five pages of 16)
    positions = np.array([0, -3, 99, 100, 2 ** 31 - 1, -(2 ** 31), 7, 8, 9, 10], np.int32)
    check(oracle_lib, 10, 2, 2, 64, 16, 64, False, 16, torch.bfloat16, slots=slots, pages=5, rows=100, positions=positions)


def test_values_that_saturate_vanish_and_are_zero(oracle_lib):
    check(oracle_lib, 30, 2, 2, 64, 16, 64, False, 16, torch.float32, scale=100.0, kv_amax=[1.0, 2.0], seed=3)
    check(oracle_lib, 30, 2, 2, 64, 16, 64, False, 16, torch.float32, scale=1e-6, kv_amax=[1.0, 2.0], seed=4)
    check(oracle_lib, 30, 2, 2, 64, 16, 64, False, 0, torch.bfloat16, scale=0.0, kv_amax=[0.0, 0.0], seed=5)
    check(oracle_lib, 30, 2, 2, 64, 16, 64, False, 16, torch.float32, scale=1e-30, kv_amax=[1e-30, 1e-35], seed=6)
    check(oracle_lib, 30, 2, 2, 64, 16, 64, False, 16, torch.float32, scale=1e30, kv_amax=[3e30, 3e30], seed=7)


@pytest.mark.parametrize("scale", [1e-38, 1e-22, 1e-3, 1e17, 1e20, 1e33])
@pytest.mark.parametrize("amax", [1e-38, 1e-16, 1e-13, 1.0, 1e17, 1e24, 3e38])
def test_magnitudes(oracle_lib, scale, amax):
    """Where corrected quotients would leave fp32's range the divided ones stand in: bytes as the oracle's everywhere."""
    check(oracle_lib, 9, 2, 2, 64, 16, 0, False, 16, torch.float32, scale=scale, kv_amax=[amax, 7 * amax if amax < 1 else amax / 7], seed=8)


def test_values_that_are_none():
    """NaN and infinities stay in their rotation group: the other groups' bytes are those of clean inputs."""
    D, T = 64, 16
    torch.manual_seed(0)
    x = torch.randn((T, 2, D), device="cuda")
    bad = x.clone()
    bad[3, 0, 20], bad[5, 1, 40], bad[7, 0, 0] = float("nan"), float("inf"), -float("inf")
    slots, amax = torch.arange(T, device="cuda"), torch.full((2,), 6.0, device="cuda")
    got = []
    for t in (x, bad):
        cache = torch.zeros((1, 2, 1, 18 * D), dtype=torch.uint8, device="cuda")
        q = hq.hq_kv_append_nvfp4(t, t, t, None, None, None, slots, amax, cache, group=16)
        got.append((q, *hq.hq_kv_read_nvfp4(cache, slots, amax)))
    hit = torch.zeros((T, 2, D), dtype=torch.bool, device="cuda")
    hit[3, 0, 16:32] = hit[5, 1, 32:48] = hit[7, 0, :16] = True
    for clean, other in zip(*got):
        assert torch.equal(clean[~hit], other[~hit])
    assert not torch.isfinite(got[1][0][hit]).any()
    assert got[1][1][3, 0, 16:32].isnan().all() and got[1][2][3, 0, 16:32].isnan().all()  # (an infinite block saturates)


def test_nothing_to_do():
    cache = torch.zeros((2, 1, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    amax = torch.ones(2, device="cuda")
    out = hq.hq_kv_append_nvfp4(e, e, e, None, None, None, none, amax, cache)
    assert out.shape == (0, 1, 64)
    k, v = hq.hq_kv_read_nvfp4(cache, none, amax)
    assert k.shape == v.shape == (0, 1, 64)
    # a cache without pages: no slot is one
    x = torch.randn((3, 1, 64), device="cuda")
    empty = torch.empty((0, 1, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    slots = torch.arange(3, device="cuda")
    out = hq.hq_kv_append_nvfp4(x, x, x, None, None, None, slots, amax, empty)
    assert torch.isfinite(out).all()
    k, v = hq.hq_kv_read_nvfp4(empty, slots, amax)
    assert not k.any() and not v.any()


def test_a_cache_past_4_gigabytes(oracle_lib):
    """Slots whose bytes lie behind 2^32: 1152 bytes per token and head."""
    D, page = 64, 64
    pages = (2 ** 32 // (18 * D * 4)) + 100
    cache = torch.zeros((pages, 1, 4, 18 * D), dtype=torch.uint8, device="cuda")
    x = torch.randn((4, 1, D), device="cuda")
    slots = torch.tensor([0, pages * page - 1, pages * page - 70, pages * page // 2], device="cuda")
    amax = torch.full((2,), 6.0, device="cuda")
    hq.hq_kv_append_nvfp4(None, x, x, None, None, None, slots, amax, cache, group=0)
    small = torch.zeros((1, 1, 1, 18 * D), dtype=torch.uint8, device="cuda")
    hq.hq_kv_append_nvfp4(None, x, x, None, None, None, torch.arange(4, device="cuda"), amax, small, group=0)
    for a, b in zip(hq.hq_kv_read_nvfp4(cache, slots, amax), hq.hq_kv_read_nvfp4(small, torch.arange(4, device="cuda"), amax)):
        assert torch.equal(a, b) and a.any()
    assert int((cache.view(-1, 18 * D).any(1)).sum()) == 4


def test_the_binding_refuses():
    D = 64
    cache = torch.zeros((2, 2, 1, 18 * D), dtype=torch.uint8, device="cuda")
    x = torch.zeros((3, 2, D), dtype=torch.bfloat16, device="cuda")
    slots, amax = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(2, device="cuda")
    cos = torch.ones((4, 32), device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    good = dict(q=x, k=x, v=x, cos=cos, sin=cos, positions=pos, slots=slots, kv_amax=amax, cache=cache)
    hq.hq_kv_append_nvfp4(**good)
    for bad in (dict(q=x.float()), dict(v=x.float()), dict(k=x[:, :1]), dict(v=x[:2]), dict(q=x.transpose(1, 2)), dict(k=x.cpu()),
                dict(cos=None), dict(sin=cos[:2]), dict(positions=pos.long()), dict(slots=slots.int()), dict(slots=slots[:2]),
                dict(kv_amax=amax[:1]), dict(cache=cache[0]), dict(cache=cache.int()), dict(q=None, q_out=x),
                dict(q_out=x.float()), dict(cos=cos[:, :20]), dict(k=x.half())):
        with pytest.raises(ValueError):
            hq.hq_kv_append_nvfp4(**{**good, **bad})
    for bad in (dict(group=8), dict(group=256), dict(cos=cos[:, :4].contiguous(), sin=cos[:, :4].contiguous())):
        with pytest.raises(hq.HQError):
            hq.hq_kv_append_nvfp4(**{**good, **bad})
    for bad in (dict(slots=slots.int()), dict(out_dtype=torch.half), dict(k=x.float(), v=x)):
        with pytest.raises(ValueError):
            hq.hq_kv_read_nvfp4(**{**dict(cache=cache, slots=slots, kv_amax=amax), **bad})
