"""Host-side checks of the products of codes and of the block norms (no GPU needed): every call refuses
bad arguments synchronously, before any CUDA call, with the status that include/hq.h names; the workspace
sizes; the binding's refusals.
"""
import ctypes

import pytest
import torch

OK, NULL, SHAPE, ALIGN, DTYPE, GROUP, CUDA = 0, 1, 2, 3, 4, 5, 6
F32, BF16 = 0, 1
P = 0x10000  # never dereferenced: every call below ends before its launch


@pytest.fixture(scope="module")
def lib():
    from hadamard_rotation_gb300 import build
    import hadamard_rotation_gb300 as hq

    build.build()
    return hq.load()


def test_the_status_codes_are_the_headers():
    from hadamard_rotation_gb300 import _lib

    assert [getattr(_lib, "HQ_" + n) for n in ("OK", "F32", "BF16")] == [OK, F32, BF16]


GEMM = dict(xq=P, xs=P, x_sg=P, wq=P, ws=P, w_sg=P, offsets=P, M=8, N=128, K=256, E=2, out=P, dt=BF16, work=P)
WGRAD = dict(gq=P, gs=P, g_sg=P, xq=P, xs=P, x_sg=P, offsets=P, T=256, N=128, K=256, E=2, out=P, dt=BF16)
LORA = dict(xq=P, xs=P, x_sg=P, wq=P, ws=P, w_sg=P, x=P, ldx=256, a=P, b=P, scaling=P, ids=P, M=8, N=128, K=256,
            n=2, R=16, out=P, dt=BF16, work=P)
ONLY_NVFP4 = {"x_sg", "w_sg", "g_sg"}
NORM = dict(h=P, ld_h=256, y=P, ld_y=256, dt=BF16, M=4, D=256, w_post=P, w_pre=P, pdt=BF16, kind=1, gate=P, ld_gate=0,
            norms=3, alpha=1.0, eps=1e-6, h_out=P, n=P, r_post=P, r_pre=P, group=16, amax=P)
NORM_BWD = dict(dh_out=P, ld_dh=256, dn=P, ld_dn=256, h_out=P, ld_h=256, y=P, ld_y=256, dt=BF16, M=4, D=256, w_post=P,
                w_pre=P, pdt=BF16, kind=1, gate=P, ld_gate=0, norms=3, r_post=P, r_pre=P, alpha=1.0, dh=P, dy=P,
                dw_post=P, dgate=P, dw_pre=P, work=P)


def call(lib, name, base, **change):
    args = {**base, **change}
    if name.endswith("mxfp4"):
        args = {k: v for k, v in args.items() if k not in ONLY_NVFP4}
    return getattr(lib, name)(*args.values(), None)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_grouped_gemm(lib, fmt):
    def st(**c):
        return call(lib, "hq_grouped_gemm_" + fmt, GEMM, **c)

    assert st(dt=2) == DTYPE and st(dt=-1) == DTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K=-32), dict(E=-1), dict(K=48), dict(E=513), dict(M=1 << 31),
                dict(N=1 << 31), dict(K=1 << 31), dict(N=(1 << 31) - 2048, M=1 << 30)):
        assert st(**bad) == SHAPE, bad
    assert st(M=0) == OK and st(N=0) == OK and st(E=0) == OK       # nothing to do
    assert st(M=0, xq=None, out=None, offsets=None) == OK
    nulls = ["xq", "xs", "wq", "ws", "offsets", "out"] + (["x_sg", "w_sg"] if fmt == "nvfp4" else [])
    for k in nulls:
        assert st(**{k: None}) == NULL, k
    for k, off in (("xq", 8), ("wq", 8), ("ws", 16), ("out", 1), ("offsets", 2)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(out=P + 2, dt=F32) == ALIGN
    if fmt == "nvfp4":
        assert st(x_sg=P + 2) == ALIGN and st(w_sg=P + 2) == ALIGN
    large = dict(M=65536, N=4096, K=4096, E=4)                     # needs its workspace
    assert lib.hq_grouped_gemm_workspace_bytes(65536, 4096, 4096, 4) > 0
    if not torch.cuda.is_available():                              # (the statuses after the sizes' own checks)
        assert st() == CUDA                                        # valid: fails for want of a device
    assert st(**large, wq=None) == NULL


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_grouped_wgrad(lib, fmt):
    def st(**c):
        return call(lib, "hq_grouped_wgrad_" + fmt, WGRAD, **c)

    assert st(dt=2) == DTYPE
    for bad in (dict(T=-128), dict(T=100), dict(N=-1), dict(K=-1), dict(E=-1), dict(E=513), dict(T=1 << 31),
                dict(N=(1 << 31) - 2048, K=(1 << 31) - 2048)):
        assert st(**bad) == SHAPE, bad
    assert st(N=0) == OK and st(K=0) == OK and st(E=0) == OK
    nulls = ["gq", "gs", "xq", "xs", "offsets", "out"] + (["x_sg", "g_sg"] if fmt == "nvfp4" else [])
    for k in nulls:
        assert st(**{k: None}) == NULL, k
    for k, off in (("gq", 8), ("xq", 8), ("gs", 16), ("xs", 16), ("out", 1), ("offsets", 2)):
        assert st(**{k: P + off}) == ALIGN, k
    if not torch.cuda.is_available():
        assert st() == CUDA


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_lora_gemm(lib, fmt):
    def st(**c):
        return call(lib, "hq_lora_gemm_" + fmt, LORA, **c)

    assert st(dt=2) == DTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=48, ldx=48), dict(n=-1), dict(R=0), dict(R=12), dict(R=136),
                dict(ldx=255), dict(M=1 << 31), dict(N=1 << 31), dict(n=1 << 31), dict(ldx=1 << 62)):
        assert st(**bad) == SHAPE, bad
    assert st(M=0) == OK and st(N=0) == OK
    nulls = ["xq", "xs", "wq", "ws", "x", "a", "b", "scaling", "ids", "out", "work"]
    for k in nulls + (["x_sg", "w_sg"] if fmt == "nvfp4" else []):
        assert st(**{k: None}) == NULL, k
    for k, off in (("xq", 8), ("wq", 8), ("ws", 16), ("x", 8), ("a", 8), ("b", 8), ("out", 1), ("ids", 2), ("work", 16),
                   ("scaling", 2)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(ldx=260) == ALIGN                                    # rows of x off their 16 bytes
    if not torch.cuda.is_available():
        assert st() == CUDA


def test_swizzle_scales(lib):
    def st(scales=P, groups=2, rows=100, cols=6, out=P):
        return lib.hq_swizzle_scales(scales, groups, rows, cols, out, None)

    for bad in (dict(groups=-1), dict(rows=-1), dict(cols=-1), dict(rows=(1 << 63) - 1), dict(cols=1 << 62),
                dict(groups=1 << 50, rows=1 << 20)):
        assert st(**bad) == SHAPE, bad
    assert st(groups=0) == OK and st(rows=0) == OK and st(cols=0, scales=None) == OK
    assert st(scales=None) == NULL and st(out=None) == NULL
    assert st(out=P + 16) == ALIGN


def test_workspace_sizes(lib):
    gemm, lora, norm = (lib.hq_grouped_gemm_workspace_bytes, lib.hq_lora_gemm_workspace_bytes,
                        lib.hq_block_norm_bwd_workspace_bytes)
    for bad in ((-1, 128, 256, 2), (8, -1, 256, 2), (8, 128, 48, 2), (8, 128, -32, 2), (8, 128, 256, -1),
                (8, 128, 256, 513), (1 << 31, 128, 256, 2)):
        assert gemm(*bad) == -1, bad
    assert gemm(1, 128, 256, 1) == 0 and gemm(0, 128, 256, 8) == 0 and gemm(8, 128, 256, 0) == 0
    for bad in ((-1, 128, 256, 16), (8, -1, 256, 16), (8, 128, 48, 16), (8, 128, 256, 0), (8, 128, 256, 12),
                (8, 128, 256, 136)):
        assert lora(*bad) == -1, bad
    assert lora(8, 128, 256, 16) >= 8 * 16 * 4                     # the thin product of every row
    for bad in ((-1, 256), (4, 0), (4, 24), (4, 32784)):
        assert norm(*bad) == -1, bad
    assert norm(0, 256) >= 0
    sizes = [norm(m, 256) for m in (1, 10, 100, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] >= 2 * 256 * 4


def test_block_norm(lib):
    def st(**c):
        return call(lib, "hq_block_norm", NORM, **c)

    assert st(dt=2) == DTYPE and st(pdt=2) == DTYPE
    for bad in (dict(M=-1), dict(D=0), dict(D=-16), dict(D=24), dict(D=32784, ld_h=32784, ld_y=32784),
                dict(M=1 << 62), dict(kind=4), dict(kind=-1), dict(norms=4), dict(norms=-1), dict(ld_h=255),
                dict(ld_y=255), dict(kind=3, ld_gate=255), dict(group=256, D=272, ld_h=272, ld_y=272)):
        assert st(**bad) == SHAPE, bad
    assert st(group=32) == GROUP and st(group=-1) == GROUP
    for k in ("h", "y", "gate", "h_out", "n", "r_post", "r_pre"):
        assert st(**{k: None}) == NULL, k
    assert st(norms=1) == NULL                                     # an amax without the norm it is of
    assert st(y=None, kind=0, gate=None, norms=0, amax=None) == NULL   # nothing to compute
    for k, off in (("h", 8), ("y", 8), ("h_out", 8), ("n", 8), ("gate", 1), ("w_post", 1), ("w_pre", 1), ("amax", 2),
                   ("r_post", 2), ("r_pre", 2)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(ld_h=260) == ALIGN and st(ld_y=260) == ALIGN and st(kind=3, ld_gate=260) == ALIGN
    assert st(M=0, amax=None, h=None, y=None) == OK
    if not torch.cuda.is_available():
        assert st() == CUDA
        assert st(M=1, ld_h=260) == CUDA                           # one row has no stride


def test_block_norm_bwd(lib):
    def st(**c):
        return call(lib, "hq_block_norm_bwd", NORM_BWD, **c)

    assert st(dt=2) == DTYPE and st(pdt=2) == DTYPE
    for bad in (dict(M=-1), dict(D=0), dict(D=24), dict(M=1 << 62), dict(kind=4), dict(norms=4), dict(ld_dh=255),
                dict(ld_dn=255), dict(ld_h=255), dict(ld_y=255)):
        assert st(**bad) == SHAPE, bad
    for k in ("dn", "h_out", "y", "gate", "r_post", "r_pre", "dh", "dy", "dgate", "work"):
        assert st(**{k: None}) == NULL, k
    assert st(dh_out=None, norms=1) == NULL                        # no gradient at all
    for k, off in (("dh_out", 8), ("dn", 8), ("h_out", 8), ("y", 8), ("dh", 8), ("dy", 8), ("work", 8), ("dgate", 2),
                   ("dw_post", 2), ("dw_pre", 2), ("r_post", 2), ("r_pre", 2), ("gate", 1)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(M=0, dw_post=None, dw_pre=None, dgate=None) == OK
    if not torch.cuda.is_available():
        assert st() == CUDA
        assert st(dw_post=None, dw_pre=None, dh_out=None) == CUDA  # what may be left out


def test_binding_refuses_host_tensors():
    import hadamard_rotation_gb300 as hq

    u8, one, off = torch.zeros(4, 16, dtype=torch.uint8), torch.ones(1), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    a, b = torch.zeros(1, 8, 32, dtype=torch.bfloat16), torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    for refused in (lambda: hq.hq_grouped_gemm_nvfp4(u8, u8, one, u8[None], u8, one, off),
                    lambda: hq.hq_grouped_gemm_mxfp4(u8, u8, u8[None], u8, off),
                    lambda: hq.hq_grouped_wgrad_nvfp4(u8, u8, one, u8, u8, one, off),
                    lambda: hq.hq_grouped_wgrad_mxfp4(u8, u8, u8, u8, off),
                    lambda: hq.hq_lora_gemm_nvfp4(u8, u8, one, u8, u8, one, x, a, b, one, off),
                    lambda: hq.hq_lora_gemm_mxfp4(u8, u8, u8, u8, x, a, b, one, off),
                    lambda: hq.hq_swizzle_scales(u8),
                    lambda: hq.hq_block_norm(x), lambda: hq.hq_block_norm_bwd(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            refused()


def test_binding_refuses_sizes_and_things_that_are_no_tensors():
    import hadamard_rotation_gb300 as hq

    with pytest.raises(ValueError):
        hq.hq_grouped_gemm_workspace_bytes(8, 128, 48, 2)
    with pytest.raises(ValueError):
        hq.hq_lora_gemm_workspace_bytes(8, 128, 256, 12)
    with pytest.raises(ValueError):
        hq.hq_block_norm_bwd_workspace_bytes(4, 24)
    for refused in (lambda: hq.hq_block_norm(None), lambda: hq.hq_block_norm(3.0),
                    lambda: hq.hq_grouped_gemm_mxfp4(1, 2, 3, 4, 5), lambda: hq.hq_swizzle_scales([1])):
        with pytest.raises((ValueError, TypeError)):
            refused()
