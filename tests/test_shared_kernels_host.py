"""Kernels that two formats share in headers keep the rules of launches that overlap: they wait for the kernel before
and read nothing through the read-only path."""

from __future__ import annotations

import re

from tests.test_dependent_launches_host import code


def test_shared_headers():
    for f in ("decode_blocks.cuh", "expand.cuh", "q8.cuh"):
        text = code(f)
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text), f
        assert text.count("__global__") == text.count("await_previous_kernel()"), f
    assert code("decode_blocks.cuh").count("__global__") == 2
