"""Compactions of a stack that an earlier one has repaired, without a GPU: the oracle by hand."""

from __future__ import annotations

import numpy as np

from oracle.pages import ref_compact


def test_a_repaired_stack_is_no_news():
    table = np.array([[3, 1]])
    free = np.array([5, 3, 5, 2, 0, 0, 0])
    c = ref_compact([32], table, np.zeros(7, dtype=int), free, 4, 16)
    assert c["bits"] == {"bad_page"} and list(c["free"][:4]) == [-1, -1, 5, 3] and list(c["table"][0]) == [2, 1]
    again = ref_compact([32], c["table"], c["refs"], c["free"], 4, 16)
    assert not again["bits"] and again["moves"] == 0
    assert np.array_equal(again["free"], c["free"]) and np.array_equal(again["table"], c["table"])
    c["free"][3] = 9  # another id that is none
    assert ref_compact([32], c["table"], c["refs"], c["free"], 4, 16)["bits"] == {"bad_page"}
