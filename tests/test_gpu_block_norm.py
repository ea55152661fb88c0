"""The norms before and after a block, forward and backward, against their formulas in 64 bits and against
differences, over types, gates, widths (one CTA, several rows per step, clusters), strides and edge rows.

Tolerances.  Each output element is a handful of fp32 operations on exact inputs and row statistics; a
row statistic over D terms, added in at most ~16 + D / 512 sequential steps per thread and a tree, is off by
under 64 * 2^-24 of the sum of its terms' magnitudes.  So an fp32 output is held to 2^-16 of the magnitudes
that were added to make it (256 roundings, an order above the count), a bf16 output to 2^-8 of its value on
top (one rounding to 8 bits), a column sum over M rows to 2^-24 * (64 + M) of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def make(M, D, dt, gate, post=True, pre=True, y=True, params=F32, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + M * 7 + D)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    shape = {"none": None, "channel": (D,), "token": (M, 1), "full": (M, D)}[gate]
    s = dict(h=(3 * r(M, D)).to(dt), y=r(M, D).to(dt) if y else None,
             w_post=(1 + 0.2 * r(D)).to(params) if post and y else None, w_pre=(1 + 0.2 * r(D)).to(params) if pre else None,
             gate=None if shape is None or not y else r(*shape).to(dt if gate == "full" else params))
    return s, dict(alpha=0.8, post_norm=post, pre_norm=pre)


def d64(t):
    return None if t is None else t.double()


def forward64(s, alpha, post_norm, pre_norm, eps=1e-6):
    """(h_out, n, r_post, r_pre), and the magnitudes added for h_out."""
    h, y, wp, wq, g = (d64(s[k]) for k in ("h", "y", "w_post", "w_pre", "gate"))
    rp = rq = n = None
    size = h.abs()
    if y is not None:
        u = y
        if post_norm:
            rp = (y.square().mean(1) + eps).rsqrt()
            u = y * rp[:, None] * (1 if wp is None else wp)
        u = u if g is None else g * u
        size = (alpha * h).abs() + u.abs()
        h = alpha * h + u
    if pre_norm:
        rq = (h.square().mean(1) + eps).rsqrt()
        n = h * rq[:, None] * (1 if wq is None else wq)
    return h, n, rp, rq, size


def close(got, want, size, name):
    tol = 2.0 ** -16 * size + (2.0 ** -8 * want.abs() if got.dtype == BF else 0)
    bad = ~((got.double() - want).abs() <= tol + 1e-30)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(), float((got.double() - want).abs().max()))


SHAPES = [(1, 16), (1, 4096), (3, 48), (37, 416), (5, 8192), (2, 8208), (3, 16384), (2, 32768), (700, 256), (301, 1360), (640, 4096), (1500, 2064),
          (650, 8192), (1500, 8208), (700, 16400)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("gate,post,pre,y", [("channel", True, True, True), ("token", True, True, True),
                                             ("full", False, True, True), ("none", True, False, True),
                                             ("none", False, True, False)])
def test_forward(dt, M, D, gate, post, pre, y):
    s, kw = make(M, D, dt, gate, post, pre, y, params=BF if M % 2 else F32)
    h_out, n, rp, rq = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], **kw)
    wh, wn, wrp, wrq, size = forward64(s, **kw)
    assert (rp is None) == (wrp is None) and (n is None) == (wn is None)
    if y:
        close(h_out, wh, size, "h_out")
    else:
        assert h_out is s["h"]
    if post and y:
        close(rp, wrp, wrp, "r_post")
    if pre:
        close(rq, wrq, wrq, "r_pre")
        # an element of n is off by what h_out's rounding gives and by its row's statistic
        w = 1 if s["w_pre"] is None else s["w_pre"].double().abs()
        close(n, wn, size * wrq[:, None] * w + wn.abs(), "n")


@pytest.mark.parametrize("group", [0, 16, 256])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,D", [(1, 256), (9, 768), (40, 5120), (3, 16384), (130, 256)])
def test_amax_is_the_quantizers(group, dt, M, D):
    """The amax that the call reduces is hq_rot_amax's of n, bit for bit, so that one pass quantizes n."""
    s, kw = make(M, D, dt, "channel")
    _, n, _, _, amax = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], amax_group=group, **kw)
    assert torch.equal(amax, hq.hq_rot_amax(n, group))


@pytest.mark.parametrize("dt", [BF, F32])
def test_strided_rows_and_in_place(dt):
    M, D = 33, 320
    s, kw = make(M, D, dt, "full")
    want = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], **kw)
    wide = {}
    for k in ("h", "y", "gate"):
        wide[k] = torch.full((M, D + 64), float("nan"), dtype=dt, device="cuda")[:, 32:32 + D]
        wide[k].copy_(s[k])
    got = hq.hq_block_norm(wide["h"], wide["y"], s["w_post"], wide["gate"], s["w_pre"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    h = s["h"].clone()
    got = hq.hq_block_norm(h, s["y"], s["w_post"], s["gate"], s["w_pre"], h_out=h, **kw)
    assert got[0] is h and all(torch.equal(a, b) for a, b in zip(got, want))
    g = [torch.randn(M, D, device="cuda").to(dt) for _ in range(2)]
    a = (s["w_post"], s["gate"], s["w_pre"], want[2], want[3])
    ref = hq.hq_block_norm_bwd(*g, want[0], s["y"], *a, **kw)
    gw = []
    for t in (*g, want[0]):
        v = torch.full((M, D + 64), float("nan"), dtype=dt, device="cuda")[:, 32:32 + D]
        v.copy_(t)
        gw.append(v)
    got = hq.hq_block_norm_bwd(*gw, wide["y"], a[0], wide["gate"], *a[2:], **kw)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_zero_rows_and_extremes():
    """Rows of zeros, of tiny and of huge values: no infinity, no NaN, statistics as defined."""
    M, D = 6, 512
    for dt in (BF, F32):
        h, y = torch.zeros(M, D, device="cuda", dtype=dt), torch.zeros(M, D, device="cuda", dtype=dt)
        h[2], h[3], y[4], y[5] = 1e-20, 1e15, 1e-20, -1e15
        s = dict(h=h, y=y, w_post=torch.ones(D, device="cuda"), w_pre=torch.ones(D, device="cuda"), gate=None)
        kw = dict(alpha=1.0, post_norm=True, pre_norm=True)
        h_out, n, rp, rq = hq.hq_block_norm(h, y, s["w_post"], None, s["w_pre"])
        wh, wn, wrp, wrq, size = forward64(s, **kw)
        close(h_out, wh, size, "h_out"), close(n, wn, size * wrq[:, None] + wn.abs(), "n")
        close(rp, wrp, wrp, "r_post"), close(rq, wrq, wrq, "r_pre")
        assert not n[0].any() and not n[1].any()
        dh, dy, dwp, _, dwq = hq.hq_block_norm_bwd(torch.ones_like(h), torch.ones_like(h), h_out, y, s["w_post"], None,
                                                   s["w_pre"], rp, rq)
        assert all(torch.isfinite(t).all() for t in (dh, dy, dwp, dwq))


def test_no_rows():
    D = 64
    e = torch.empty(0, D, device="cuda")
    w = torch.ones(D, device="cuda")
    h_out, n, rp, rq, amax = hq.hq_block_norm(e, e, w, w, w, amax_group=16)
    assert n.shape == (0, D) and float(amax) == 0
    got = hq.hq_block_norm_bwd(e, e, h_out, e, w, w, w, rp, rq)
    assert all(not t.any() and t.shape == (D,) for t in got[2:])


def backward64(s, dh_out, dn, h_out, rp, rq, alpha, post_norm, pre_norm):
    """Gradients by the formulas, with the magnitudes added for each."""
    y, wp, wq, g = (d64(s[k]) for k in ("y", "w_post", "w_pre", "gate"))
    D = s["h"].shape[1]
    d = dh_out.double() if dh_out is not None else torch.zeros_like(h_out.double())
    ds = d.abs()
    out, size = {}, {}
    if pre_norm:
        h, n, r = h_out.double(), dn.double(), rq.double()[:, None]
        gn = n * (1 if wq is None else wq)
        d = d + r * gn - h * r ** 3 / D * (gn * h).sum(1, keepdim=True)
        ds = ds + (r * gn).abs() + h.abs() * r ** 3 / D * (gn * h).abs().sum(1, keepdim=True)
        out["dw_pre"], size["dw_pre"] = (n * h * r).sum(0), (n * h * r).abs().sum(0)
    out["dh"], size["dh"] = alpha * d if y is not None else d, ds
    if y is None:
        return out, size
    x = y * rp.double()[:, None] if post_norm else y
    u = x if wp is None else x * wp
    if g is not None:
        dim = 0 if g.dim() == 1 else 1 if g.shape[1] == 1 else None
        out["dgate"], size["dgate"] = d * u, ds * u.abs()
        if dim is not None:
            out["dgate"] = out["dgate"].sum(dim, keepdim=dim == 1)
            size["dgate"] = size["dgate"].sum(dim, keepdim=dim == 1)
    du, dus = (d, ds) if g is None else (d * g, ds * g.abs())
    if post_norm:
        out["dw_post"], size["dw_post"] = (du * x).sum(0), (dus * x.abs()).sum(0)
        w = 1 if wp is None else wp
        r = rp.double()[:, None]
        dy = r * du * w - y * r ** 3 / D * (du * w * y).sum(1, keepdim=True)
        dys = r * dus * abs(w) + y.abs() * r ** 3 / D * (dus * abs(w) * y.abs()).sum(1, keepdim=True)
    else:
        dy, dys = du, dus
    out["dy"], size["dy"] = dy, dys
    return out, size


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("gate,post,pre,y,skip", [
    ("channel", True, True, True, True), ("token", True, True, True, True), ("full", True, True, True, True),
    ("full", False, True, True, False), ("token", False, False, True, True), ("none", True, False, True, True),
    ("channel", False, True, True, True), ("none", False, True, False, True), ("none", False, True, False, False)])
def test_backward(dt, M, D, gate, post, pre, y, skip):
    s, kw = make(M, D, dt, gate, post, pre, y, params=F32 if M % 2 else BF, seed=3)
    h_out, n, rp, rq = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], **kw)
    g = torch.Generator("cuda").manual_seed(9)
    dh_out = torch.randn(M, D, generator=g, device="cuda").to(dt) if skip or not pre else None
    dn = torch.randn(M, D, generator=g, device="cuda").to(dt) if pre else None
    got = dict(zip(("dh", "dy", "dw_post", "dgate", "dw_pre"), hq.hq_block_norm_bwd(
        dh_out, dn, h_out, s["y"], s["w_post"], s["gate"], s["w_pre"], rp, rq, **kw)))
    want, size = backward64(s, dh_out, dn, h_out, rp, rq, **kw)
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, w in want.items():
        assert got[k].shape == w.shape, k
        if k.startswith("dw") or (k == "dgate" and gate == "channel"):
            bad = (got[k].double() - w).abs() > (2.0 ** -16 + 2.0 ** -24 * M) * size[k] + 1e-30
            assert not bad.any(), (k, float((got[k].double() - w).abs().max()))
        else:
            close(got[k], w, size[k], k)
    again = hq.hq_block_norm_bwd(dh_out, dn, h_out, s["y"], s["w_post"], s["gate"], s["w_pre"], rp, rq, **kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(again, got.values()))  # a fixed order of sums


@pytest.mark.parametrize("gate", ["channel", "token", "full", "none"])
def test_backward_against_differences(gate):
    """Directional derivatives of the forward call in 64 bits (central differences, checked to 1e-5 of the
    sum of magnitudes: step 1e-4 leaves 1e-8 of the third derivative) against the fp32 call's gradients."""
    M, D = 4, 64
    s, kw = make(M, D, F32, gate, seed=5)
    h_out, n, rp, rq = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], **kw)
    g = torch.Generator("cuda").manual_seed(2)
    a, b = (torch.randn(M, D, generator=g, device="cuda") for _ in range(2))
    grads = dict(zip(("h", "y", "w_post", "gate", "w_pre"), hq.hq_block_norm_bwd(
        a, b, h_out, s["y"], s["w_post"], s["gate"], s["w_pre"], rp, rq, **kw)))
    for k, grad in grads.items():
        if grad is None:
            continue
        way = torch.randn(s[k].shape, generator=g, device="cuda", dtype=torch.float64)
        ends = []
        for e in (1e-4, -1e-4):
            t = dict(s, **{k: s[k].double() + e * way})
            h2, n2 = forward64(t, **kw)[:2]
            ends.append((h2 * a).sum() + (n2 * b).sum())
        diff, dot = (ends[0] - ends[1]) / 2e-4, (grad.double() * way).sum()
        assert abs(float(diff - dot)) <= 1e-5 * float((grad.double() * way).abs().sum()), (k, float(diff), float(dot))


def test_long_tensor_and_streams():
    """More than 2^32 elements, rows at both ends; and two streams at once."""
    M, D = 140_000, 32768  # 4.6e9 elements
    h = torch.empty(M, D, dtype=BF, device="cuda").fill_(1.0)
    h[M - 1] = 3.0
    _, n, _, rq = hq.hq_block_norm(h)
    assert float(n[0].float().mean()) == 1.0 and float(n[M - 1].float().mean()) == 1.0
    assert abs(float(rq[0]) - 1) < 1e-6 and abs(float(rq[M - 1]) * 3 - 1) < 1e-6
    del h, n
    torch.cuda.empty_cache()
    sets = [make(257, 2048, BF, "channel", seed=k) for k in range(2)]
    call = lambda s, kw, **m: hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], **kw, **m)
    want = [call(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [call(*s, stream=t) for s, t in zip(sets, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
