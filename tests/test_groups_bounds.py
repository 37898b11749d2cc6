"""Buffer loads of the kernels of bqmm_groups.h must be covered by their range checks (no GPU)."""
import re

import pytest

from test_kernel_code import assembly

SOURCES = ["grouped_gemm.hip", "grouped_stream.hip", "expert_gemv.hip", "lora.hip"]


@pytest.mark.parametrize("source", SOURCES)
def test_range_checked_loads_have_no_scalar_offset(source):
    """A buffer's range check is made for the per-lane offset and the instruction's constant; what the scalar offset
    adds is past it.  These kernels' buffers end where a tensor may end, so the scalar offset is 0."""
    loads = re.findall(r"^\s*buffer_load_\w+\s+(.*)$", assembly(source), flags=re.M)
    scalar = [re.search(r"s\[\d+:\d+\],\s*(\S+?)(?:\s|$)", load).group(1) for load in loads]
    assert scalar and set(scalar) == {"0"}, sorted(set(scalar))
