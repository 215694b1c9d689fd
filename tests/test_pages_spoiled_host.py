"""Forks that meet page ids that are none, without a GPU: the oracle refuses them."""

from __future__ import annotations

import numpy as np
import pytest

from oracle.pages import ref_fork


def fork(table, free, count, source=(-1, 0, 0), lens=(40, 0, 0)):
    return ref_fork(list(source), list(lens), np.array(table), np.zeros(10, dtype=int), np.array(free), count, 16)


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("bad", [-1, 10, 1 << 30, -(1 << 31)])
def test_a_source_with_a_page_that_is_none(at, bad):
    table = [[7, 2, 5], [0, 0, 0], [0, 0, 0]]
    table[0][at] = bad
    f = fork(table, [1, 4, 8] + [0] * 7, 3)
    assert f["bits"] == {"bad_page"} and list(f["kv_lens"]) == [40, 0, 0] and f["left"] == 3
    assert np.array_equal(f["table"], table) and not f["refs"].any()
    assert list(f["src"]) == [-1] * 3 and list(f["dst"]) == [-1] * 3


@pytest.mark.parametrize("bad", [-1, 10, 1 << 30, -(1 << 31)])
def test_a_stack_entry_that_is_none(bad):
    """The row that would get it stays empty and the entry is gone; the next row gets the page below."""
    table = [[7, 2, 5], [0, 0, 0], [0, 0, 0]]
    f = fork(table, [1, 4, bad] + [0] * 7, 3)
    assert f["bits"] == {"bad_page"} and list(f["kv_lens"]) == [40, 0, 40] and f["left"] == 1
    assert f["table"].tolist() == [[7, 2, 5], [0, 0, 0], [7, 2, 4]]
    assert f["refs"][7] == f["refs"][2] == 1 and f["refs"].sum() == 2
    assert list(f["src"]) == [-1, -1, 5] and list(f["dst"]) == [-1, -1, 4]
