"""Several things wrong in one step: each has its bit in the error word."""

from __future__ import annotations

import numpy as np
import pytest

from oracle.q4 import ref_build_tables
from tests.test_tables_gpu import compare, ops, run  # noqa: F401

pytestmark = pytest.mark.gpu


def test_stack_past_the_pool_and_too_few_slots(ops):  # noqa: F811
    # two requests give three pages back to a stack of three in a pool of four; the third asks for more than the slots
    lens, new = [32, 16, 0], [-1, -1, 5]
    pt, free = np.array([[0, 1], [2, -1], [-1, -1]]), np.array([3, 2, 1, 0])
    want = ref_build_tables(lens, new, pt, free, 3, 16, 3)
    assert want["bits"] == {"bad_page", "bad_chunk"}
    compare(*run(ops, lens, new, pt, free, 3, 16, 3), want)


def test_all_refusals_at_once(ops):  # noqa: F811
    # 0: its row is too short; 1: served; 2: no page; 3: no slots
    lens, new = [30, 16, 16, 3], [3, 1, 1, 2]
    pt, free = np.array([[0, 1], [2, -1], [3, -1], [4, -1]]), np.array([5, 0, 0, 0, 0, 0])
    want = ref_build_tables(lens, new, pt, free, 1, 16, 6)
    assert want["bits"] == {"too_long", "no_pages", "bad_chunk"} and list(want["kv_lens"]) == [30, 17, 16, 3]
    compare(*run(ops, lens, new, pt, free, 1, 16, 6), want)
