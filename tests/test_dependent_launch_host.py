"""Kernels that may be scheduled while the one before them still runs (programmatic stream serialisation) wait
for it before they read what it wrote.  A load that the compiler knows to be invariant (__ldg, or through
a const __restrict__ pointer) is bound to no wait and may be moved in front of it, so these kernels use
ordinary loads.  (Reads the sources; no GPU needed.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_latent_kv_37_b200", "csrc")
FILES = ["attn_simt.cuh", "attn_sm100.cuh", "chunk_plan.cuh", "chunk_sm100.cuh", "epilogue.cuh", "fp8.cuh", "gemm_streamk.cuh",
         "prompt_pair_sm100.cuh", "prompt_sm100.cuh", "rows.cuh"]


@pytest.mark.parametrize("name", FILES)
def test_kernels_that_wait_for_the_grid_before_use_ordinary_loads(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernels = [k for k in text.split("__global__")[1:] if "griddep_wait" in k]
    assert kernels
    for k in kernels:
        # to the end of the kernel: a closing brace at the start of a line
        k = k[:re.search(r"^}", k, re.M).end()]
        assert "__restrict__" not in k and "__ldg" not in k, k[:200]
