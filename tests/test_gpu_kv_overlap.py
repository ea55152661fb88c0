"""Outputs of the paged cache's calls that lie in their inputs: the binding refuses them, for other threads still read there.
Neighbours in one storage are fine.
"""
import pytest
import torch

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu
T, Hq, Hkv, D = 6, 4, 2, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build

    build.build()
    hq.load()
    yield
    assert hq.hq_read_fault() == 0


def tensors():
    torch.manual_seed(0)
    cache = torch.zeros((2, Hkv, 1, 18 * D), dtype=torch.uint8, device="cuda")
    return cache, torch.arange(T, device="cuda"), torch.full((2,), 5.0, device="cuda")


def test_append():
    cache, slots, amax = tensors()
    store = torch.randn(4 * T * Hq * D, device="cuda").to(torch.bfloat16)
    n = T * Hq * D
    at = {name: store[i * n:i * n + T * h * D].view(T, h, D) for i, (name, h) in enumerate((("q", Hq), ("k", Hkv), ("v", Hkv)))}
    q, k, v = (at[x].clone() for x in "qkv")

    def call(q_out):
        return hq.hq_kv_append_nvfp4(at["q"], at["k"], at["v"], None, None, None, slots, amax, cache, q_out=q_out)

    half = T * Hkv * D  # elements of k and of v
    for begin in (0, 64, n - 64, n, n + half - 8, 2 * n - 64, 2 * n + half - 8):
        with pytest.raises(ValueError, match="overlap"):
            call(store[begin:begin + n].view(T, Hq, D))
    with pytest.raises(ValueError, match="overlap"):
        call(at["q"])
    for x, y in zip((q, k, v), (at[x] for x in "qkv")):
        assert torch.equal(x, y)
    want = call(None)
    assert torch.equal(call(store[3 * n:].view(T, Hq, D)), want)
    assert torch.equal(call(store[2 * n + half:3 * n + half].view(T, Hq, D)), want)
    # parts of one projection, and q_out behind it
    y = torch.cat([t.flatten(1) for t in (q, k, v)], 1)
    both = torch.cat([y.flatten(), torch.zeros(n, dtype=torch.bfloat16, device="cuda")])
    y, out = both[:y.numel()].view(T, -1), both[y.numel():].view(T, Hq, D)
    parts = [t.unflatten(1, (-1, D)) for t in y.split([Hq * D, Hkv * D, Hkv * D], 1)]
    assert torch.equal(hq.hq_kv_append_nvfp4(*parts, None, None, None, slots, amax, cache, q_out=out), want)
    with pytest.raises(ValueError, match="overlap"):
        hq.hq_kv_append_nvfp4(*parts, None, None, None, slots, amax, cache, q_out=both[y.numel() - 8:-8].view(T, Hq, D))


def test_attention():
    cache, slots, amax = tensors()
    x = torch.randn((T, Hkv, D), device="cuda")
    hq.hq_kv_append_nvfp4(None, x, x, None, None, None, slots, amax, cache)
    n = T * Hq * D
    store = torch.randn(2 * n, device="cuda").to(torch.bfloat16)
    table = torch.arange(2, device="cuda").int()[None]
    kv_len, q_start = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([T], [0, T]))

    def call(out):
        return hq.hq_kv_attention_nvfp4(store[:n].view(T, Hq, D), cache, table, kv_len, q_start, amax, 0.1, out=out)

    for begin in (0, 8, n - 8):
        with pytest.raises(ValueError, match="overlap"):
            call(store[begin:begin + n].view(T, Hq, D))
    want = call(None)
    assert torch.equal(call(store[n:].view(T, Hq, D)), want)
