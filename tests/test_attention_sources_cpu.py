"""Rules that the sources of the norm, cache and attention kernels keep and no run can show."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_quantized_gemm_b200", "csrc")
FILES = ["qg_norm.cu", "qg_kv4.cu", "qg_attn_kv4_decode.cu", "qg_attn_kv4_prompt.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_waits_for_what_came_before(name):
    """A kernel that may start early sees the grids before it through griddepcontrol.wait and through nothing else:
    each executes it, in every thread."""
    text = source(name)
    kernels = len(re.findall(r"\b__global__\b", text))
    assert kernels > 0
    plain = re.findall(r"^  pdl_wait\(\);", text, re.M)      # a statement of the kernel's own block
    assert len(plain) == len(re.findall(r"\bpdl_wait\(", text)) == kernels


@pytest.mark.parametrize("name", FILES)
def test_a_wait_that_gives_up_does_so_for_the_whole_warp(name):
    """A bounded wait ends lane by lane; what a warp does next is decided by all of its lanes."""
    assert not re.findall(r"if \(!\s*mbar_wait\(", source(name))
