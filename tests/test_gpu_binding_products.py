"""The binding of the products and norms on a GPU: what it refuses (before any launch), and that memory it
allocates for a call on a given stream is not still in use elsewhere."""
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


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def f32(*shape):
    return torch.ones(shape, device="cuda")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def refused(call, args, changes):
    call(*args)
    for at, value in changes:
        wrong = list(args)
        wrong[at] = value
        with pytest.raises(ValueError):
            call(*wrong)
    torch.cuda.synchronize()


def test_grouped_gemm():
    args = (u8(5, 32), u8(5, 4), f32(1), u8(2, 40, 32), u8(2, 512), f32(2), i32(0, 2, 5))
    refused(hq.hq_grouped_gemm_nvfp4, args, [
        (0, u8(5, 16)), (0, u8(4, 32)), (0, bf16(5, 32)), (0, u8(5, 64)[:, ::2]), (0, None), (1, u8(5, 2)),
        (1, u8(5, 4).cpu()), (2, f32(2)), (2, None), (3, u8(40, 32)), (3, u8(3, 40, 32)), (4, u8(1024)), (5, f32(1)),
        (6, i32(0, 5)), (6, i32(0, 2, 5).long()), (6, i32(0, 2, 5).cpu())])
    for kw in (dict(out=f32(5, 41)), dict(out=u8(5, 40)), dict(out=f32(40, 5).t()), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            hq.hq_grouped_gemm_nvfp4(*args, **kw)
    refused(hq.hq_grouped_gemm_mxfp4, (u8(5, 32), u8(5, 2), u8(2, 40, 32), u8(2, 512), i32(0, 2, 5)),
            [(1, u8(5, 4)), (3, u8(2, 1024)), (4, i32(0))])
    with pytest.raises(ValueError):  # K that is no multiple of 32
        hq.hq_grouped_gemm_nvfp4(u8(5, 24), u8(5, 3), f32(1), u8(2, 40, 24), u8(2, 512), f32(2), i32(0, 2, 5))


def test_grouped_wgrad():
    args = (u8(40, 128), u8(4 * 512), f32(1), u8(32, 128), u8(4 * 512), f32(1), i32(0, 128, 256))
    refused(hq.hq_grouped_wgrad_nvfp4, args, [
        (0, u8(40, 64)), (1, u8(512)), (2, f32(2)), (3, u8(32, 64)), (3, u8(2, 32, 128)), (4, u8(5, 512)),
        (6, i32()), (6, i32(0, 128, 256).long()), (6, None)])
    with pytest.raises(hq.HQError):  # tokens not padded to 128: the library's own refusal
        hq.hq_grouped_wgrad_nvfp4(u8(40, 32), u8(512), f32(1), u8(32, 32), u8(512), f32(1), i32(0, 64))


def test_lora_gemm():
    args = (u8(5, 32), u8(5, 4), f32(1), u8(40, 32), u8(512), f32(1), bf16(5, 64), bf16(3, 8, 64), bf16(3, 40, 8), f32(3),
            i32(0, 1, 2, -1, 0))
    refused(hq.hq_lora_gemm_nvfp4, args, [
        (6, f32(5, 64)), (6, bf16(5, 32)), (6, bf16(64, 5).t()), (6, bf16(5, 64).cpu()), (7, bf16(3, 12, 64)), (7, bf16(8, 64)),
        (7, bf16(3, 8, 32)), (8, bf16(3, 8, 40)), (8, bf16(2, 40, 8)), (9, f32(2)), (10, i32(0, 1)),
        (10, i32(0, 1, 2, -1, 0).long())])


@pytest.mark.parametrize("where,value", [
    (1, "bf16(5, 64)"), (1, "f32(4, 64)"), (2, "f32(32)"), (2, "f32(64).double()"), (3, "f32(5)"), (3, "f32(5, 32)"),
    (3, "f32(1, 64)"), (4, "bf16(64)"), (0, "f32(5, 24)"), (0, "f32(64)"), (0, "f32(64, 5).t()"), (0, "f32(5, 64).half()")])
def test_block_norm(where, value):
    args = [f32(5, 64), f32(5, 64), f32(64), f32(64), f32(64)]
    hq.hq_block_norm(*args)
    args[where] = eval(value)
    with pytest.raises(ValueError):
        hq.hq_block_norm(*args)


def test_block_norm_options():
    h, y, w = f32(5, 64), f32(5, 64), f32(64)
    for kw in (dict(y=None, gate=w), dict(y=y, w_post=w, post_norm=False), dict(y=y, w_pre=w, pre_norm=False),
               dict(y=y, h_out=f32(5, 32)), dict(y=y, n=bf16(5, 64))):
        with pytest.raises(ValueError):
            hq.hq_block_norm(h, **kw)
    for group in (32, -16, 2 ** 32 + 16):
        with pytest.raises(hq.HQError):
            hq.hq_block_norm(h, y, amax_group=group)
    h_out, n, r_post, r_pre = hq.hq_block_norm(h, y, w, None, w)
    for kw in (dict(dn=None), dict(r_pre=None), dict(r_post=None), dict(dn=bf16(5, 64)), dict(h_out=f32(4, 64)),
               dict(r_pre=f32(4)), dict(w_post=bf16(64)), dict(pre_norm=False)):
        args = dict(dh_out=h, dn=n, h_out=h_out, y=y, w_post=w, w_pre=w, r_post=r_post, r_pre=r_pre)
        hq.hq_block_norm_bwd(**args)
        with pytest.raises(ValueError):
            hq.hq_block_norm_bwd(**{**args, **kw})


def test_memory_of_a_call_is_its_streams():
    """Calls in turn on the current stream and, without any order between them, on another: a call's new memory
    (results, workspace) must not be what the other stream's last call is still using."""
    g = torch.Generator("cuda").manual_seed(0)
    M, D = 20000, 256
    side = torch.cuda.Stream()
    ins = [[torch.randn(M, D, generator=g, device="cuda") for _ in range(3)] for _ in range(2)]
    w = torch.randn(D, generator=g, device="cuda")

    def run(i, stream):
        h, y, dn = ins[i]
        _, n, r_post, r_pre = hq.hq_block_norm(h, y, w, None, w, h_out=outs[i], stream=stream)
        return hq.hq_block_norm_bwd(None, dn, outs[i], y, w, None, w, r_post, r_pre, stream=stream)[2::2]

    outs = [torch.empty(M, D, device="cuda") for _ in range(2)]
    want = [[t.clone() for t in run(i, None)] for i in range(2)]
    torch.cuda.synchronize()
    got = [[run(0, None), run(1, side)] for _ in range(50)]
    torch.cuda.synchronize()
    for pair in got:
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(pair[i], want[i]))
