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


@pytest.mark.parametrize("rows,slots", [(1, 1), (4, 4), (16, 64)])
def test_expert_gemv_rows_that_round_up_past_31_bits(L, rows, slots):
    """Rounded up to units of 32 rows their count wraps; the last 512 also end a workgroup's loop over a row past it."""
    for n in (MOST, MOST - 15, MOST - 30, MOST - 31, MOST - 511, MOST - 1023):
        assert L.bqm_mxfp4_expert_gemv(A, B, C, D, E, 0, rows, slots, 3, 32, n, NUL) == 2


def test_lora_add_rows_and_widths_past_the_grid(L):
    def f(m, k=64, n=8, adapters=1):
        return L.bqm_lora_add(A, k, 0, B, C, 2, NUL, D, E, NUL, n, F, n, A, m, k, n, 8, adapters, NUL)

    assert f(2_097_088) == 2 and f(MOST) == 2               # a tile of 32 rows each, and two more: 65535 at most
    assert f(1_000_000, n=80_000) == 2 and f(1, n=MOST) == 2   # tiles times columns
    assert f(1023, n=2 ** 21, adapters=1024) == 2           # every adapter may have a tile of its own
    assert f(1, k=(1 << 21) + 8) == 2
