"""The gathering of the top alternatives in every order of a workgroup's waves, on the CPU.

The kernel's waves share a bound and nothing orders their steps, so a result that is right in the order that a GPU
mostly takes may be wrong in another.  ``logprobs_model.hip`` runs the kernel's own keys and gate on the host in many
orders: the ids have to be exact and the keys that wait have to fit their buffer in each."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import layer_ref

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
N = 12000          # three steps of 4096


@pytest.fixture(scope="module")
def orders(tmp_path_factory):
    from block_quantized_matmul_02_amd import build

    lib = str(tmp_path_factory.mktemp("model") / "model.so")
    subprocess.run([build.HIPCC, "--offload-host-only", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", build.INCLUDE,
                    "-I", build.CSRC, os.path.join(HERE, "logprobs_model.hip"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).logprobs_orders
    P, I = ctypes.c_void_p, ctypes.c_int
    f.argtypes = [P, I, I, I, I, I, ctypes.c_uint, P, P, P]

    def run(row, top, skip=0, vec=4, count=200):
        row = np.ascontiguousarray(row, np.float32)
        want = layer_ref.logprobs(row[None].astype(np.float64), np.zeros((1, 0), np.int32), top)[3][0].astype(np.int32)
        got, most = np.zeros(top, np.int32), ctypes.c_int()
        rc = f(row.ctypes.data, len(row), skip, vec, top, count, 7 * top + skip, want.ctypes.data, got.ctypes.data,
               ctypes.byref(most))
        assert rc != 2, f"{most.value} keys wait"
        assert rc == 0, f"ids {got} instead of {want}"

    return run


def normal(seed):
    return np.random.default_rng(seed).standard_normal(N).astype(np.float32) * 3


TOPS = [1, 2, 5, 8, 20, 32]


@pytest.mark.parametrize("top", TOPS)
def test_rows_of_values(orders, top):
    i = np.arange(N)
    for row in (normal(0), normal(1).round(), i / N * 9, -i / N * 9, np.full(N, 1.5), (i * 7919 % 11 == 3) * 1.0,
                (i // 16) % 64, np.where(normal(2) > 9, np.nan, normal(2)), np.full(N, np.nan), np.full(N, np.inf)):
        for skip, vec in ((0, 4), (3, 4), (5, 8)):
            orders(row, top, skip, vec, 60)


@pytest.mark.parametrize("top", TOPS)
def test_a_masked_row_with_one_value(orders, top):
    """A step with one finite lane under another wave's -inf bound: its -inf keys all pass that bound's column."""
    for at in (5, 1030, 5000):
        row = np.full(N, -math.inf)
        row[at] = 1.0
        orders(row, top)


@pytest.mark.parametrize("top", TOPS)
def test_masks_that_leave_fewer_than_top(orders, top):
    """The bound's own value is -inf: -inf columns before it still come first."""
    orders(np.full(N, -math.inf), top)
    for seed, left in enumerate((1, 2, top - 1, top, 3 * top, 100)):
        rng = np.random.default_rng(seed)
        row = np.full(N, -math.inf)
        at = rng.choice(N, left, replace=False)
        row[at] = rng.standard_normal(left)
        orders(row, top)
        row[rng.choice(N, 40, replace=False)] = math.nan
        orders(row, top)
    for start in (0, 1000, 1024, 4000, 4096, 11999):       # a run of finite ones
        row = np.full(N, -math.inf)
        row[start:start + 3] = 1.0
        orders(row, top)
        row[start:start + 3] = np.finfo(np.float32).min
        orders(row, top, 2, 8)


def few_zeros(count, seed):
    """Negative logits but for `count` zeros of both signs, in different waves of the same and of neighbouring steps."""
    rng = np.random.default_rng(seed)
    row = -1.0 - rng.random(N)
    row[rng.choice(N, count, replace=False)] = np.where(rng.random(count) < 0.5, 0.0, -0.0)
    return row


@pytest.mark.parametrize("top", range(1, 9))
def test_alternatives_that_tie_at_zero(orders, top):
    """A bound just below +0 admits every zero of either sign, at the columns that win the tie too."""
    for count in range(2, 9):
        for seed in range(4):
            orders(few_zeros(count, seed), top, count=100)
    for tiny in (1e-45, -1e-45, 2e-38, -2e-38):          # and the neighbours of zero
        row = few_zeros(6, top)
        row[row == 0] = np.float32(tiny)
        orders(row, top, count=100)
