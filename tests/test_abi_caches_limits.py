"""Limits of the paged cache's calls (no GPU needed): the largest sizes that pass, and the first that are refused."""
from test_abi_caches import ALIGN, ATTEND, P, SHAPE, caller, lib  # noqa: F401 (the fixture)


def test_sequences(lib):  # noqa: F811
    st = caller(lib, "hq_kv_attention_nvfp4", ATTEND)
    assert st(S=1 << 20, work=P + 8) == ALIGN  # (what comes last)
    for S in ((1 << 20) + 1, 1 << 24, (1 << 31) - 1025):
        assert st(S=S) == SHAPE, S
        assert st(S=S, T=0) == SHAPE, S
