"""Sizes past what the operators of include/bqmm_layer.h count in 32 bits are refused before anything is launched (no
GPU; the stand-in pointers are never dereferenced)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
A, B, C, D, E = (P(i << 20) for i in range(1, 6))
NUL = P(0)
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    import block_quantized_matmul_02_amd as bqm

    if not os.path.exists(bqm.LIB_PATH):
        from block_quantized_matmul_02_amd import build

        build.build()
    return bqm.lib()


def test_gemv_rows_that_round_up_past_31_bits(L):
    for m in (1, 5, 6, 16):
        for n in (MOST, MOST - 15, MOST - 30):         # + 15 or + 31 for whole tiles
            assert L.bqm_mxfp4_gemv(A, B, C, D, m, 32, n, NUL) == 2


def test_logprobs_workspace_of_sizes_that_are_refused(L):
    """-1 where bqm_logprobs itself answers 2."""
    def call(m, n):
        return L.bqm_logprobs(A, n, 0, NUL, 0, NUL, B, C, D, E, 5, A, m, n, NUL)

    for m, n in ((1, 2 ** 28 + 1), (1, MOST), (2 ** 24, 100), (MOST, 100)):
        assert call(m, n) == 2
        assert L.bqm_logprobs_workspace(m, n, 5) == -1
    assert L.bqm_logprobs_workspace(1, 2 ** 28, 5) > 0 and L.bqm_logprobs_workspace(2 ** 24 - 1, 100, 5) == 0


def test_binding_names_the_reason(L):
    import block_quantized_matmul_02_amd as bqm

    for sizes, rc in (((1, 2 ** 28 + 1, 5), 2), ((2 ** 24, 100, 0), 2), ((1, 100, 33), 1), ((0, 100, 1), 1), ((1, 4, 5), 1)):
        with pytest.raises(bqm.BqmError) as e:
            bqm.bqm_logprobs_workspace(*sizes)
        assert e.value.rc == rc
