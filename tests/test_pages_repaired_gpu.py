"""Stacks that a compaction has repaired, on the GPU against the oracle: compacted again, and forked from."""

from __future__ import annotations

import pytest
import torch

from tests.test_pages_gpu import State, check_compact, check_fork, ops  # noqa: F401 (ops: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,spare,spoil", [([40, 33], 9, [1]), ([16] * 70, 40, [0, 7, 39]), ([0, 0], 4, [2])])
def test_compact_a_repaired_stack_again(ops, lens, spare, spoil):  # noqa: F811
    """The places that a first compaction leaves without a page are not told again; a new fault is."""
    s = State(lens, 16, 4, spare, 21)
    pages = s.table[0, 0] if lens[0] else s.free[3]
    s.free[spoil] = pages
    assert check_compact(ops, s)["bits"] == {"bad_page"}
    assert list(s.free[:len(spoil)]) == [-1] * len(spoil)
    for _ in range(2):
        assert not check_compact(ops, s)["bits"]
    s.free[s.count - 1] = s.n_pages
    assert check_compact(ops, s)["bits"] == {"bad_page"}
    assert not check_compact(ops, s)["bits"]


def test_fork_after_a_repaired_stack(ops):  # noqa: F811
    """A stack repaired down to places without a page serves no fork."""
    s = State([40, 0, 0, 0], 16, 4, 3, 5)
    s.free[0] = s.table[0, 1]
    check_compact(ops, s)
    want = check_fork(ops, s, [-1, 0, 0, 0])
    assert want["bits"] == {"bad_page"} and list(want["kv_lens"]) == [40, 40, 40, 0] and want["left"] == 0
    assert torch.equal(torch.tensor(sorted(want["dst"][1:])), torch.tensor(sorted([-1, *s.free[1:3]])))
