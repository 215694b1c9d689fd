"""Kernels that are set up while the kernel before them still runs read nothing through the read-only path."""

from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_relative_attn_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_no_read_only_loads():
    found = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_dependent(" in code(f)]
    assert {"decode_q4.cu", "prefill.cu", "q4_rows.cu", "tables.cu"} <= set(found)
    for f in found + ["async.cuh", "ptx.cuh", "q4.cuh", "tc.cuh", "plan.cuh"]:
        text = code(f)
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text), f
        # every kernel of the file that is launched so waits
        assert f not in found or text.count("__global__") == text.count("await_previous_kernel()"), f
