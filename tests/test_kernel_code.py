"""What the compiled kernels must not contain, read from the assembly (or, before it, the compiler's
own form) that the build's flags give (no GPU)."""
import os
import re
import subprocess

import pytest

from block_quantized_matmul_02_amd import build


def assembly(source, *more):
    cmd = [build.HIPCC, *build.HIPFLAGS, *build.EXTRA.get(source, []), "--cuda-device-only", "-S", *more,
           os.path.join(build.CSRC, source), "-o", "-"]
    return subprocess.run(cmd, check=True, capture_output=True, text=True).stdout


@pytest.fixture(scope="module")
def logprobs():
    return assembly("logprobs.hip")


def test_the_waves_bound_is_read_from_lds(logprobs):
    """An access that has lost its address space waits for every load in flight, the next steps' logits among them."""
    assert "ds_max_u64" in logprobs                       # the bound's update
    assert not re.findall(r"\bflat_(?:load|store|atomic)\w*", logprobs)


@pytest.mark.parametrize("source", ["norm.hip", "mxfp4_quantize.hip", "logprobs.hip"])
def test_no_access_claims_more_alignment_than_is_checked(source):
    """Pointers are checked to 16 bytes at most, so no access to memory may be compiled for more."""
    accesses = re.findall(r"\b(?:load|store)\b.*ptr addrspace\(1\).*\balign (\d+)", assembly(source, "-emit-llvm"))
    assert accesses and max(map(int, accesses)) <= 16
