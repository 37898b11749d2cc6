"""Sizes past what the operators of include/bqmm_groups.h count in 32 bits are refused before anything is launched (no
GPU; the stand-in pointers are never dereferenced)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
A, B, C, D, E, F = (P(i << 20) for i in range(1, 7))
NUL = P(0)
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    import block_quantized_matmul_02_amd as bqm

    if not os.path.exists(bqm.LIB_PATH):
        from block_quantized_matmul_02_amd import build

        build.build()
    return bqm.lib()


def test_lora_add_rows_and_widths_past_the_grid(L):
    def f(m, k=64, n=8, adapters=1):
        return L.bqm_lora_add(A, k, 0, B, C, 2, NUL, D, E, NUL, n, F, n, A, m, k, n, 8, adapters, NUL)

    assert f(2_097_088) == 2 and f(MOST) == 2               # a tile of 32 rows each, and two more: 65535 at most
    assert f(1_000_000, n=80_000) == 2 and f(1, n=MOST) == 2   # tiles times columns
    assert f(1023, n=2 ** 21, adapters=1024) == 2           # every adapter may have a tile of its own
    assert f(1, k=(1 << 21) + 8) == 2


def test_limits_that_the_header_names(L):
    """The first size past each."""
    def route(m):
        return L.bqm_route(A, 8, 0, 2, 1, B, C, m, 8, NUL)

    def combine(m, n, t):
        return L.bqm_combine(A, t, B, NUL, C, t, m, 1, n, NUL)

    def gemm(slots, groups, n, k=32, glu=0):
        return L.bqm_mxfp4_grouped_gemm(A, B, C, D, E, F, A, 0, glu, 1, slots, groups, k, n, NUL)

    assert route(2 ** 25 - 3) == 2 and route(MOST) == 2
    assert combine(MOST - 254, 4, 0) == 2 and combine(MOST - 254, 8, 2) == 2     # pieces of 16 bytes of y
    assert combine(2 ** 20, 2 ** 13 + 1, 0) == 2 and combine(2 ** 20, 2 ** 14 + 1, 1) == 2
    for glu in (0, 1):
        assert gemm(256 * 4094, 1, 256 * 1024, glu=glu) == 2                      # 4094 + 2 tiles of rows
        assert gemm(1024, 1023, 256 * 4080 + 2, glu=glu) == 2                     # 4 + 1024, of 4081 of columns
        assert gemm(1, 1, 32, k=(1 << 22) + 32, glu=glu) == 2
