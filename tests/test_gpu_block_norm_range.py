"""Gradients of the block norms for rows of very large and very small magnitude, against the formulas in 64 bits.
Tolerance: that of test_gpu_block_norm.py, relative to the magnitudes that are added in each row."""
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_block_norm import BF, F32, backward64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,D", [(14, 512), (700, 256), (650, 4096), (14, 8448)])
@pytest.mark.parametrize("gate,post,pre,y", [("channel", True, True, True), ("token", True, True, True), ("full", True, True, True),
                                             ("none", True, False, True), ("none", False, True, False)])
@pytest.mark.parametrize("large", [True, False])
def test_rows_of_every_magnitude(dt, M, D, gate, post, pre, y, large):
    """Large rows with the usual eps; small ones without, whose reciprocal norms are large."""
    s, kw = make(M, D, dt, gate, post, pre, y, seed=11)
    scales = torch.tensor([1.0, 1e12, 1e13, 1e15, 1e16] if large else [1.0, 1e-6, 1e-12, 1e-13, 1e-15], device="cuda")
    at = torch.arange(M, device="cuda")
    s["h"] = (s["h"].float() * scales[at % 5][:, None]).to(dt)
    if y:
        s["y"] = (s["y"].float() * scales[at // 5 % 5][:, None]).to(dt)
    h_out, n, rp, rq = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], eps=1e-6 if large else 0.0, **kw)
    g = torch.Generator("cuda").manual_seed(4)
    dh_out = torch.randn(M, D, generator=g, device="cuda").to(dt)
    dn = torch.randn(M, D, generator=g, device="cuda").to(dt) if pre else None
    if large:  # a row's two gradients of one size at h
        r = 1 if rq is None else rq[:, None]
        dh_out = (dh_out.float() * r).to(dt)
    got = dict(zip(("dh", "dy", "dw_post", "dgate", "dw_pre"), hq.hq_block_norm_bwd(
        dh_out, dn, h_out, s["y"], s["w_post"], s["gate"], s["w_pre"], rp, rq, **kw)))
    want, size = backward64(s, dh_out, dn, h_out, rp, rq, **kw)
    for k, w in want.items():
        if k.startswith("dw") or (k == "dgate" and gate == "channel"):
            bad = ~((got[k].double() - w).abs() <= (2.0 ** -16 + 2.0 ** -24 * M) * size[k])
            assert not bad.any(), (k, int(bad.sum()), float((got[k].double() - w).abs().max()))
            continue
        # (an fp32 or bf16 result below the normal numbers is off by at most the smallest of them)
        least = 2.0 ** -126
        tol = 2.0 ** -16 * size[k] + (2.0 ** -8 * w.abs() if got[k].dtype == BF else 0) + least
        bad = ~((got[k].double() - w).abs() <= tol)
        assert not bad.any(), (k, int(bad.sum()), bad.nonzero()[:3].tolist(), float(((got[k].double() - w).abs() / tol).max()))
