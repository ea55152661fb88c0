"""The workspace functions of the products and of the adapters refuse what the calls refuse (no GPU needed: every call here
ends before its launch)."""
import itertools

import pytest

from test_abi_products import GEMM, LORA, SHAPE, call, lib  # noqa: F401

BIG = (1 << 31) - 2048
SIZES = (-1, 0, 1, 8, 4096, 1 << 20, BIG, 1 << 31)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_grouped_gemm(lib, fmt):  # noqa: F811
    for M, N, K, E in itertools.product(SIZES, SIZES, (-32, 0, 32, 48, 4096, BIG), (-1, 0, 1, 512, 513)):
        # (a missing operand: refused after the sizes, before anything is enqueued)
        got = call(lib, "hq_grouped_gemm_" + fmt, GEMM, M=M, N=N, K=K, E=E, **({"xq": None} if K else {"out": None}))
        assert (got == SHAPE) == (lib.hq_grouped_gemm_workspace_bytes(M, N, K, E) == -1), (M, N, K, E, got)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_lora_gemm(lib, fmt):  # noqa: F811
    for M, N, K, R in itertools.product(SIZES, SIZES, (-32, 0, 32, 48, 4096, BIG), (0, 8, 12, 128, 136)):
        got = call(lib, "hq_lora_gemm_" + fmt, LORA, M=M, N=N, K=K, R=R, ldx=max(K, 256), xq=None)
        assert (got == SHAPE) == (lib.hq_lora_gemm_workspace_bytes(M, N, K, R) == -1), (M, N, K, R, got)
