"""bqm_group_rows where a workgroup's 2048 rows are full, the counts of 32 chunks that are read together, and groups that
fill the 512 threads of a workgroup."""
import numpy as np
import pytest

from test_gpu_route import bqm, check_groups  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [2047, 2048, 2049, 65535, 65536, 65537, 131072, 131073])
def test_group_rows_at_whole_chunks(bqm, count):  # noqa: F811
    for groups in (1, 64, 510, 511, 512, 513, 1024):
        rng = np.random.default_rng(count + groups)
        check_groups(bqm, rng.integers(-1, groups + 1, count), groups)
    check_groups(bqm, np.full(count, 510), 511)                # all in the last thread's group, and none of any
    check_groups(bqm, np.full(count, 511), 511)
    check_groups(bqm, np.arange(count) // 2048, 64)            # a group a chunk


def test_group_rows_workspace_begins_past_one_chunk(bqm):  # noqa: F811
    assert bqm.bqm_group_rows_workspace(2048, 7) == 0
    assert bqm.bqm_group_rows_workspace(2049, 7) == 2 * 8 * 4
    assert bqm.bqm_group_rows_workspace(65537, 1024) == 33 * 1025 * 4
