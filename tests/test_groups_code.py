"""What the compiled kernels of bqmm_groups.h must not contain, read from what the build's flags give (no GPU)."""
import re

import pytest

from test_kernel_code import assembly

SOURCES = ["route.hip", "grouped_gemm.hip", "grouped_stream.hip", "expert_gemv.hip", "combine.hip", "lora.hip"]


@pytest.mark.parametrize("source", SOURCES)
def test_no_access_claims_more_alignment_than_is_checked(source):
    """Pointers are checked to 16 bytes at most, so no access to memory may be compiled for more."""
    accesses = re.findall(r"\b(?:load|store)\b.*ptr addrspace\(1\).*\balign (\d+)", assembly(source, "-emit-llvm"))
    assert accesses and max(map(int, accesses)) <= 16


@pytest.mark.parametrize("source", SOURCES)
def test_no_kernel_spills(source):
    """Scratch memory in the loops of these kernels costs more than any of their tiles gains."""
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size (\d+)", assembly(source))
    assert sizes and set(sizes) == {"0"}
