"""Kernels that may start before the one ahead of them has ended (those that wait
with pdl_wait) read what another kernel may have written by plain loads.

A non-coherent load (__ldg, ld.global.nc) takes its data as constant from the
kernel's start, which lies before that wait, and a compiler may move it there.  It
is for weights and tables alone."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cache_host_gb300", "csrc")

# what these read so: norms' weights and the table of angles; an expert's scales
CONSTANTS = {"qk_norm_rope.cu": 6, "expert_decode_mxfp4.cu": 4}


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def waiting():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        if "pdl_wait();" in code(path):
            out.append(os.path.basename(path))
    return out


ATTENTION_SIDE = ["kv8_cache.cu", "kv8_few.cuh", "kv_plan.cu", "qk_norm_rope.cu", "token_logprobs.cu", "tree_attention.cuh",
                  "verify_drafts.cu"]
EXPERTS = ["control.cu", "decode_bf16.cuh", "expert_decode.cu", "expert_decode_mxfp4.cu", "merge.cu"]


def test_these_kernels_wait():
    assert set(ATTENTION_SIDE + EXPERTS) - {"decode_bf16.cuh"} == set(waiting())


@pytest.mark.parametrize("name", ATTENTION_SIDE + EXPERTS)
def test_non_coherent_loads_are_of_constants(name):
    text = code(os.path.join(CSRC, name))
    assert len(re.findall(r"__ldg\(|ld\.global\.nc", text)) == CONSTANTS.get(name, 0)
    # (the compiler makes such loads itself of a kernel's pointer that is const and restrict)
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text)
