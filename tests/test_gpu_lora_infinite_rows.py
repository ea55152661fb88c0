"""Infinities in x: a row's thin product is then infinite, and its term has the sign and kind of the definition (infinite
where all of the channel's ranks agree in sign, NaN where they do not)."""
import numpy as np
import pytest
import torch

import hadamard_rotation_gb300 as hq
from test_gpu_lora import call, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,R", [(40, 64, 128, 16), (64, 256, 4096, 24), (1100, 2304, 4128, 64)])
def test_infinite_rows(fmt, M, N, K, R):
    p = problem(fmt, M, N, K, 2, R, np.arange(M) % 3 - 1, M + K)
    p["a"][:, :, :8] = p["a"][:, :, :8].abs() + 1
    p["b"][:, ::2] = p["b"][:, ::2].abs() + 1   # every second channel's ranks agree
    p["b"][:, ::4] *= -1
    clean = call(fmt, p)
    rows = torch.tensor([1, 2, M - 3, M - 2], device="cuda")
    rows = rows[p["ids"][rows] >= 0]
    p["x"][rows, :8] = float("inf")
    got = call(fmt, p)
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert torch.equal(got[others], clean[others])
    inf = torch.full((len(rows), N), float("inf"), device="cuda")
    inf[:, ::4] *= -1
    mixed = (p["b"][p["ids"][rows].long()] > 0).any(-1) & (p["b"][p["ids"][rows].long()] < 0).any(-1)
    assert not mixed[:, ::2].any()
    want = torch.where(mixed, torch.full_like(inf, float("nan")), inf)
    sure = mixed.clone()
    sure[:, ::2] = True                          # (a channel whose ranks happen to agree: either sign)
    got = got[rows].float()
    assert torch.equal(got.isnan()[sure], want.isnan()[sure])
    assert torch.equal(got.nan_to_num(7.0)[sure], want.nan_to_num(7.0)[sure])
    assert not torch.isfinite(got).any()
