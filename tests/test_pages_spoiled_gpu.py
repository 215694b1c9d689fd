"""Forks that meet page ids that are none, on the GPU against the oracle."""

from __future__ import annotations

import numpy as np
import pytest

from tests.test_pages_gpu import State, check_fork, ops  # noqa: F401 (ops: a fixture)

pytestmark = pytest.mark.gpu
BAD = [-1, 1 << 30, -(1 << 31)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", BAD + ["first past the pool"])
@pytest.mark.parametrize("tokens,at", [(40, 0), (40, 1), (40, 2), (32, 1), (3, 0), (100 * 16 + 1, 97), (100 * 16 + 1, 100)])
def test_fork_of_a_source_with_a_page_that_is_none(ops, tokens, at, bad, in_place):  # noqa: F811
    """The fork stays empty and takes nothing; a fork of another source gets the page on top."""
    s = State([tokens, 20, 0, 0, 0], 16, 101, 6, tokens + at)
    s.table[0, at] = s.n_pages if isinstance(bad, str) else bad
    want = check_fork(ops, s, [-1, -1, 0, 1, 0], in_place)
    assert want["bits"] == {"bad_page"} and list(want["kv_lens"]) == [tokens, 20, 0, 20, 0] and want["left"] == 5


def test_fork_of_a_source_whose_other_entries_are_none(ops):  # noqa: F811
    """What lies behind a source's tokens is no page of it."""
    s = State([40, 0], 16, 8, 3, 2)
    s.table[0, 3:] = -1
    want = check_fork(ops, s, [-1, 0])
    assert not want["bits"] and list(want["kv_lens"]) == [40, 40]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_fork_off_a_stack_with_entries_that_are_none(ops, bad, in_place):  # noqa: F811
    """The row that would get one stays empty, shares nothing, and the entry is gone; too few pages are told too."""
    s = State([40, 33, 48] + [0] * 7, 16, 5, 4, 8)
    s.free[[1, 3]] = bad
    source = [-1, -1, -1, 0, 2, 1, 0, 0, 2, 1]
    want = check_fork(ops, s, source, in_place)
    assert want["bits"] == {"bad_page", "no_pages"} and want["left"] == 0
    assert list(want["kv_lens"]) == [40, 33, 48, 0, 48, 33, 0, 40, 48, 0]


@pytest.mark.parametrize("B", [70, 300, 1100])
def test_forks_by_several_thread_blocks(ops, B):  # noqa: F811
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 200, B)
    kids = rng.permutation(B)[:B // 2]
    lens[kids] = 0
    s = State(list(lens), 16, 13, B // 3, B)
    source = np.full(B, -1)
    source[kids] = rng.integers(0, B, len(kids))
    held = [(b, c) for b in range(B) for c in range(-(-lens[b] // 16))]
    for i in rng.permutation(len(held))[:B // 20]:
        s.table[held[i]] = rng.choice(BAD)
    s.free[rng.permutation(B // 3)[:5]] = -1
    want = check_fork(ops, s, source)
    assert "bad_page" in want["bits"]
