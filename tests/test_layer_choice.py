"""The rule that chooses between the kernels of the MXFP4 GEMM, on the host (no GPU)."""
import ctypes
import os

import pytest

GRID_Y = 65535     # workgroups along y that every HIP device takes


@pytest.fixture(scope="module")
def groups():
    import block_quantized_matmul_02_amd as bqm

    if not os.path.exists(bqm.LIB_PATH):
        from block_quantized_matmul_02_amd import build

        build.build()
    # int bqm::mxfp4_stream_groups(int m, int k, int n, int cus, double tile_cost): groups of 16 tokens at a time, 0 for tiles
    f = bqm.lib()._ZN3bqm19mxfp4_stream_groupsEiiiid
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_double]
    f.restype = ctypes.c_int
    return f


@pytest.mark.parametrize("k", [32, 512, 2048, 4096, 4128, 8192, 17408])
def test_chunks_of_tokens_fit_the_grid(groups, k):
    for n in (1, 16, 17, 32, 33, 320):
        for m in (65, 1_000_000, 1_048_560, 1_048_561, 2_200_000, 4_194_240, 4_194_241, 4_300_000, 2_000_000_000):
            for cost in (50.0, 1e3, 1e5, 1e12):
                g = groups(m, k, n, 256, cost)
                assert 0 <= g <= 4
                assert g == 0 or -(-m // (16 * g)) <= GRID_Y, f"{m} x {k} x {n}: chunks of {16 * g} tokens"


def test_few_tokens_and_few_tiles_still_stream(groups):
    assert groups(16, 4096, 5152, 256, 16.0) == 1
    assert groups(64, 4096, 8192, 256, 18.5) == 4
    assert groups(64, 4096, 65536, 256, 30.0) == 0
    assert groups(98, 12512, 320, 256, 47.0) > 0
    assert groups(1_000_000, 2048, 16, 256, 1e12) > 0      # 15625 chunks
