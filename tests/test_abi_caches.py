"""Host-side checks of the INT8 product and of the paged cache (no GPU needed): every call refuses bad arguments
synchronously, before any CUDA call, with the status that include/hq.h names; the sizes' functions.
"""
import pytest
import torch

import hadamard_rotation_gb300 as hq

OK, NULL, SHAPE, ALIGN, DTYPE, GROUP, CUDA = 0, 1, 2, 3, 4, 5, 6
F32, BF16 = 0, 1
P = 0x10000  # never dereferenced: every call below ends before its launch


@pytest.fixture(scope="module")
def lib():
    from hadamard_rotation_gb300 import build

    build.build()
    return hq.load()


INT8 = dict(xq=P, xs=P, wq=P, ws=P, M=8, N=100, K=256, out=P, dt=BF16)
APPEND = dict(q=P, ld_q=2048, k=P, ld_k=512, v=P, ld_v=512, dt=BF16, T=4, q_heads=8, kv_heads=2, D=128, cos=P, sin=P, rows=100,
              rotary=128, interleaved=0, positions=P, slots=P, group=16, amax=P, q_out=P, cache=P, pages=3, page=32)
READ = dict(cache=P, pages=3, page=32, kv_heads=2, D=128, slots=P, T=4, amax=P, group=16, k=P, v=P, dt=BF16)
ATTEND = dict(q=P, ld_q=1024, T=4, q_heads=8, cache=P, pages=3, page=32, kv_heads=2, D=128, table=P, ld_table=5, table_pages=5,
              kv_len=P, q_start=P, S=2, max_q=2, amax=P, scale=0.1, window=0, group=16, out=P, lse=P, work=P)


def caller(lib, name, base):
    return lambda **c: getattr(lib, name)(*{**base, **c}.values(), None)


def test_gemm_int8(lib):
    st = caller(lib, "hq_gemm_int8", INT8)
    assert st(dt=2) == DTYPE and st(dt=-1) == DTYPE
    for bad in (dict(M=-1), dict(N=-1), dict(K=-16), dict(K=24), dict(K=1 << 17), dict(M=1 << 31), dict(N=1 << 31)):
        assert st(**bad) == SHAPE, bad
    assert st(M=0) == OK and st(N=0, xq=None, xs=None, wq=None, ws=None, out=None) == OK
    for k in ("xq", "xs", "wq", "ws", "out"):
        assert st(**{k: None}) == NULL, k
    for k, off in (("xq", 8), ("wq", 8), ("xs", 2), ("ws", 2), ("out", 1)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(out=P + 2, dt=F32) == ALIGN


CACHE = (dict(kv_heads=0), dict(kv_heads=5000), dict(D=32), dict(D=96), dict(D=-128), dict(page=0), dict(page=24), dict(page=-16),
         dict(pages=-1), dict(pages=1 << 60))


def test_kv_append(lib):
    st = caller(lib, "hq_kv_append_nvfp4", APPEND)
    assert st(dt=2) == DTYPE
    for bad in CACHE + (dict(T=-1), dict(T=1 << 31), dict(T=1 << 30, q_heads=2, ld_q=2 * 128), dict(q_heads=-1), dict(q_heads=5000), dict(rotary=-16), dict(rotary=8), dict(rotary=144),
                        dict(rows=0), dict(ld_q=1000), dict(ld_k=255), dict(ld_v=0), dict(ld_k=1 << 62), dict(D=64, group=256)):
        assert st(**bad) in (SHAPE, GROUP), bad
    assert st(group=8) == GROUP and st(group=256) == SHAPE and st(group=-1) == GROUP
    assert st(T=0) == OK and st(T=0, k=None, cache=None, slots=None) == OK
    for k in ("q", "k", "v", "cos", "sin", "positions", "slots", "amax", "q_out", "cache"):
        assert st(**{k: None}) == NULL, k
    for k, off in (("q", 8), ("k", 8), ("v", 2), ("cos", 4), ("sin", 8), ("positions", 2), ("slots", 4), ("amax", 2), ("q_out", 8),
                   ("cache", 8), ("ld_q", 0)):
        bad = dict(ld_q=2052) if k == "ld_q" else {k: P + off}
        assert st(**bad) == ALIGN, k
    # not asked for, not needed: what is refused is only the alignment that comes last
    assert st(rotary=0, cos=None, sin=None, positions=None, rows=0, cache=P + 8) == ALIGN
    assert st(q_heads=0, q=None, q_out=None, ld_q=0, cache=P + 8) == ALIGN
    assert st(pages=0, cache=None, slots=P + 4) == ALIGN


def test_kv_read(lib):
    st = caller(lib, "hq_kv_read_nvfp4", READ)
    assert st(dt=5) == DTYPE
    for bad in CACHE + (dict(T=-1), dict(T=1 << 31), dict(T=1 << 30)):
        assert st(**bad) == SHAPE, bad
    assert st(group=64) == GROUP and st(group=256) == SHAPE
    assert st(T=0, cache=None, k=None) == OK
    for k in ("cache", "slots", "amax", "k", "v"):
        assert st(**{k: None}) == NULL, k
    for k, off in (("cache", 8), ("slots", 4), ("amax", 2), ("k", 8), ("v", 4)):
        assert st(**{k: P + off}) == ALIGN, k


def test_kv_attention(lib):
    st = caller(lib, "hq_kv_attention_nvfp4", ATTEND)
    for bad in CACHE + (dict(T=-1), dict(T=1 << 31), dict(S=-1), dict(S=1 << 31), dict(q_heads=0), dict(q_heads=7), dict(q_heads=5000),
                        dict(max_q=-1), dict(window=-1), dict(table_pages=-1), dict(ld_table=4), dict(table_pages=1 << 27, ld_table=1 << 27),
                        dict(table_pages=(1 << 20) + 1, ld_table=1 << 27),
                        dict(pages=0), dict(ld_q=1000), dict(ld_q=1 << 62), dict(ld_table=1 << 62), dict(T=1 << 29)):
        assert st(**bad) == SHAPE, bad
    assert st(group=8) == GROUP and st(group=256) == SHAPE
    assert st(T=0) == OK and st(S=0, q=None, cache=None, work=None) == OK
    for k in ("q", "out", "kv_len", "q_start", "amax", "work", "table", "cache"):
        assert st(**{k: None}) == NULL, k
    for k, off in (("q", 8), ("cache", 8), ("table", 2), ("kv_len", 2), ("q_start", 1), ("amax", 2), ("out", 8), ("lse", 2), ("work", 8)):
        assert st(**{k: P + off}) == ALIGN, k
    assert st(ld_q=1028) == ALIGN and st(table_pages=1 << 20, ld_table=1 << 20, work=P + 8) == ALIGN
    assert st(lse=None, work=P + 8) == ALIGN and st(table_pages=0, pages=0, table=None, cache=None, work=P + 8) == ALIGN


def test_sizes(lib):
    assert lib.hq_kv_page_bytes(64, 8, 128) == 64 * 8 * 144 and lib.hq_kv_page_bytes(16, 1, 64) == 18 * 64
    for bad in ((0, 1, 64), (24, 1, 64), (16, 0, 64), (16, 1, 80)):
        assert lib.hq_kv_page_bytes(*bad) == -1
        with pytest.raises(ValueError):
            hq.hq_kv_page_bytes(*bad)
    assert lib.hq_kv_attention_workspace_bytes(8, 2, 128, 100, 100) > lib.hq_kv_attention_workspace_bytes(8, 2, 128, 100, 1) > 0
    for bad in ((0, 1, 64, 1, 1), (7, 2, 64, 1, 1), (8, 2, 96, 1, 1), (8, 0, 64, 1, 1), (5000, 1, 64, 1, 1), (8, 2, 64, -1, 1), (8, 2, 64, 1, -1),
                (8, 2, 64, 1 << 31, 1)):
        assert lib.hq_kv_attention_workspace_bytes(*bad) == -1
        with pytest.raises(ValueError):
            hq.hq_kv_attention_workspace_bytes(*bad)


def test_the_binding_has_no_cpu_path():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 2, 1, 18 * 64), dtype=torch.uint8)
    i8 = torch.zeros((2, 16), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_gemm_int8(i8, torch.ones(2), i8, torch.ones(2))
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_kv_append_nvfp4(x, x, x, None, None, None, torch.zeros(2, dtype=torch.int64), torch.ones(2), cache)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_kv_read_nvfp4(cache, torch.zeros(2, dtype=torch.int64), torch.ones(2))
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_kv_attention_nvfp4(x, cache, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                                 torch.zeros(2, dtype=torch.int32), torch.ones(2), 1.0)
