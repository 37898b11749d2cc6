"""Rows whose K-th alternative ties with many columns: the lowest columns come first, exactly, whichever wave of a
workgroup holds them (``test_logprobs_model.py`` tries the waves' orders on the host)."""
import math

import numpy as np
import pytest

import layer_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def ids_are_exact(bqm, rows, top, what):
    logits = torch.from_numpy(np.stack(rows).astype(np.float32))
    want = layer_ref.logprobs(logits.double().numpy(), np.zeros((len(rows), 0), np.int32), top)[3]
    for t in (torch.float32, torch.bfloat16):
        if not torch.equal(logits.to(t).float().nan_to_num(7.0), logits.nan_to_num(7.0)):
            continue   # not values of that type
        got = bqm.bqm_logprobs(logits.to(t).to(DEV), None, top)[3].cpu().numpy()
        assert np.array_equal(got, want), f"{what} {t} top {top}"


# one workgroup a row (600 rows; up to a step of 4096) and rows split over workgroups
@pytest.mark.parametrize("m,n", [(600, 12000), (6, 4096), (3, 70000)])
@pytest.mark.parametrize("top", [1, 5, 32])
def test_fewer_finite_logits_than_alternatives(bqm, m, n, top):
    rng = np.random.default_rng(n + top)
    rows = []
    for t in range(m):
        row = np.full(n, -math.inf)
        left = rng.integers(0, top + 1)
        row[rng.choice(n, left, replace=False)] = rng.integers(-4, 4, left)
        if t % 3 == 2:
            row[rng.choice(n, 40, replace=False)] = math.nan
        rows.append(row)
    ids_are_exact(bqm, rows, top, f"{m}x{n}")


@pytest.mark.parametrize("m,n", [(600, 12000), (6, 4096), (40, 70000)])
@pytest.mark.parametrize("top", range(1, 9))
def test_ties_at_zero(bqm, m, n, top):
    """All negative but for 2..8 zeros of both signs, anywhere in the row."""
    rng = np.random.default_rng(n + top)
    rows = []
    for t in range(m):
        row = -1.0 - rng.integers(0, 64, n) / 64.0
        count = rng.integers(2, 9)
        row[rng.choice(min(n, 20000), count, replace=False)] = np.where(rng.random(count) < 0.5, 0.0, -0.0)
        rows.append(row)
    ids_are_exact(bqm, rows, top, f"{m}x{n}")
