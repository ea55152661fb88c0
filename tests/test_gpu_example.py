"""The example's block against the same block in plain fp32 tensors: its output and every gradient to what four
bits keep, its training, its serving step.

Tolerance.  A value of four bits (E2M1) is off by at most 1/8 of its block's scale step pattern; over normally
distributed operands the rotated NVFP4 codes have a relative rms error near 0.095, so a product of two such operands
is off by about 0.095 sqrt(2) = 0.135 of its norm.  0.2 is allowed for one product.  Gradients behind two products
(of operands that carry the first one's error) add in squares: 0.28 is allowed there.
"""
import os
import sys

import pytest
import torch

import hadamard_rotation_gb300 as hq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    import expert_block

    yield expert_block
    assert hq.hq_read_fault() == 0


def norm(x, w, eps=1e-6):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def plain(h, y, p, expert):
    h = h + p["gate"] * norm(y, p["w_post"])
    n = norm(h, p["w_pre"])
    return h, torch.einsum("mk,mnk->mn", n, p["w"][expert])


def off(got, want):
    return float((got.detach().float() - want.detach()).norm() / want.detach().norm())


def test_training_step(example):
    g = torch.Generator("cuda").manual_seed(5)
    M, D, E = 300, 256, 5
    expert = torch.randint(0, E - 1, (M,), generator=g, device="cuda").sort().values  # the last one is idle
    order, *route = example.routing(expert, E)
    assert torch.equal(order, torch.arange(M, device="cuda"))
    p = example.parameters(D, E)
    ins = {"h": torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16),
           "y": torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16), **p}
    dh, do = (torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    a = {k: v.clone().requires_grad_() for k, v in ins.items()}
    b = {k: v.float().requires_grad_() for k, v in ins.items()}
    got = example.block(a["h"], a["y"], a, route)
    want = plain(b["h"], b["y"], b, expert)
    assert off(got[0], want[0]) < 2 ** -7
    assert off(got[1], want[1]) < 0.2
    ga = torch.autograd.grad(got, list(a.values()), (dh, do))
    gb = torch.autograd.grad(want, list(b.values()), (dh.float(), do.float()))
    for (k, _), x, y in zip(a.items(), ga, gb):
        assert x.shape == y.shape
        assert off(x, y) < 0.28, (k, off(x, y))
    assert not ga[-1][E - 1].any()  # the idle expert's weights have a gradient of zero


def test_training_fits(example):
    losses = example.train()
    assert losses[-1] < 0.5 * losses[0] and all(v == v for v in losses)


@pytest.mark.parametrize("M", [1, 33])
def test_serving(example, M):
    g = torch.Generator("cuda").manual_seed(M)
    D, E, R = 256, 6, 16

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    p, shared = example.parameters(D, E), draw(D, D, scale=D ** -0.5)
    A, B, scaling = draw(3, R, D, scale=D ** -0.5), draw(3, D, R, scale=0.5), torch.ones(3, device="cuda")
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 4 - 1
    expert = torch.randint(0, E, (M,), generator=g, device="cuda")
    h, y = draw(M, D), draw(M, D)
    got = example.serve(h, y, p, shared, (A, B, scaling), ids, expert)
    f = {k: v.float() for k, v in p.items()}
    h = h.float() + f["gate"] * norm(y.float(), f["w_post"])
    n = norm(h, f["w_pre"])
    z = n @ shared.float().t()
    for m in range(M):
        if ids[m] >= 0:
            z[m] += B[ids[m]].float() @ (A[ids[m]].float() @ n[m])
    want = torch.einsum("mk,mnk->mn", z, f["w"][expert])
    assert off(got[0], h) < 2 ** -7
    assert off(got[1], want) < 0.28


def test_main_runs(example, capsys):
    example.main()
    text = capsys.readouterr().out
    assert "training" in text and "serving: (33, 256) (33, 256)" in text
