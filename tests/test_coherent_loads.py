"""Kernels are launched programmatically, so one may be resident while the kernel
before it writes, and non-coherent loads promise nothing for such memory.  So there
is no __ldg, and the only const __restrict__ parameters (which the compiler may read
that way) are queries, block tables and pools in the attention kernels of pa_decode:
its plan kernel has waited for whatever wrote them before those start."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_150_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
BEHIND_A_PLAN = {"decode_mma.cuh", "decode_fma.cuh", "decode_simt.cuh", "decode_tc.cuh"}
READ_ONLY = {"q", "tables", "k_cache", "v_cache", "p"}  # p: a row of them


def code(f):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())


@pytest.mark.parametrize("f", SOURCES)
def test_no_non_coherent_loads(f):
    text = code(f)
    assert "__ldg(" not in text and "ld.global.nc" not in text
    names = set(re.findall(r"const\s+[\w:]+\s*\*\s*__restrict__\s+(\w+)", text))
    assert names <= (READ_ONLY if f in BEHIND_A_PLAN else set())
