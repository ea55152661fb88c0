"""The amax that hq_block_norm reduces is hq_rot_amax of its n, bit for bit: where a step of the kernel holds several rows
and the last one is not full, with and without an eps, in every form of the call."""
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_block_norm import BF, F32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("group", [0, 16, 256])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,D", [
    (777, 256), (768, 256), (305, 256),   # several rows per step, the last step full or not
    (1500, 2304), (641, 4096), (2, 256),
    (20000, 256),                         # many steps
    (700, 8448), (3, 16640),              # rows over a cluster, whose last CTA has fewer columns
])
def test_bits_of_the_quantizers_pass(M, D, dt, group, eps):
    s, kw = make(M, D, dt, "channel")
    for y in (s["y"], None):
        a = (s["w_post"], s["gate"]) if y is not None else (None, None)
        _, n, _, _, amax = hq.hq_block_norm(s["h"], y, *a, s["w_pre"], amax_group=group, eps=eps,
                                            **(kw if y is not None else {}))
        assert torch.equal(amax, hq.hq_rot_amax(n, group))
        assert torch.isfinite(amax).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group", [0, 16])
def test_narrow_rows_without_an_eps(dt, group):
    """Rows that leave lanes of a warp idle, and rows past M beside them."""
    for M, D in ((305, 64), (1001, 48), (160, 16), (4000, 112)):
        s, kw = make(M, D, dt, "token")
        _, n, _, _, amax = hq.hq_block_norm(s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], amax_group=group, eps=0.0, **kw)
        assert torch.isfinite(amax).all() and torch.equal(amax, hq.hq_rot_amax(n, group))


def test_rows_that_are_not_finite():
    """A row of zeros without an eps is 0 / 0 in n, and the amax says so like the quantizer's; tiny rows whose squares
    vanish are infinite."""
    s, _ = make(777, 256, F32, "none")
    s["h"][100] = 0.0
    _, n, _, _, amax = hq.hq_block_norm(s["h"], amax_group=16, eps=0.0)
    assert n[100].isnan().all() and amax.isnan().all() and hq.hq_rot_amax(n, 16).isnan().all()
    s["h"][100] = 1e-30
    _, n, _, _, amax = hq.hq_block_norm(s["h"], amax_group=0, eps=0.0)
    assert n[100].isinf().all() and torch.equal(amax, hq.hq_rot_amax(n, 0))
