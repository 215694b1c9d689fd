"""Requests whose new tokens do not all fit the slot map are refused: their lengths, rows and the stack stay whole."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.q4 import ref_build_tables
from tests.test_tables_gpu import DEV, compare, ops, run, state  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("most,kv,none", [
    (12, [20, 17, 20, 0], 0),  # all served
    (11, [20, 10, 20, 0], 6),  # the second does not fit: none of its tokens has a slot
    (5, [20, 10, 20, 0], 0),
    (4, [15, 10, 20, 0], 4),   # nor the first
    (0, [15, 10, 20, 0], 0),
])
def test_refused_for_slots(ops, in_place, most, kv, none):  # noqa: F811
    # request 0 starts on the last place of page 0, 1 on page 6, 2 asks for nothing, 3 has ended (its page 5 on top)
    lens, new = [15, 10, 20, 3], [5, 7, 0, -1]
    pt, free = np.array([[0, -1], [6, -1], [3, 4], [5, -1]]), np.array([1, 2, 7, 8, 0, 0, 0, 0, 0, 0])
    got, err = run(ops, lens, new, pt, free, 4, 16, most, in_place)
    compare(got, err, ref_build_tables(lens, new, pt, free, 4, 16, most))
    assert got["kv_lens"].tolist() == kv and err == (0 if most >= 12 else 8) and got["cu"].tolist() == [0, 5, 12, 12, 12]
    assert int(got["left"]) == 5 - (kv[0] == 20) - (kv[1] == 17)
    assert got["table"][:2].tolist() == [[0, 5 if kv[0] == 20 else -1], [6, 8 if kv[1] == 17 else -1]]
    if kv[0] == 20:
        assert got["slots"][:5].tolist() == [15, 80, 81, 82, 83]
    assert int((got["slots"] < 0).sum()) == none


def test_state_is_whole_and_the_step_can_be_taken_again(ops):  # noqa: F811
    """In place, with a map that grows: after refusals the same lengths as in one step with room for all."""
    r = np.random.default_rng(8)
    B, P = 60, 32
    lens, pt, free = state(B, P, 12, 400, 9, 6 * P)
    new = r.integers(0, 3 * P, B)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    d = dict(lens=i32(lens), pt=i32(pt), free=i32(free), count=i32([400]))
    left, total, live = new.copy(), int(new.sum()), []
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for most in (total // 3, total // 2, total):
        before = d["lens"].tolist()
        kv, cu, slots, _ = ops.build_tables(d["lens"], i32(left), d["pt"], d["free"], d["count"], page_size=P,
                                            max_tokens=most, kv_lens=d["lens"], free_left=d["count"], device_error=err)
        s, c = slots.tolist(), cu.tolist()
        for b in range(B):
            mine = s[c[b]:min(c[b + 1], most)]
            if d["lens"][b].item() == before[b] + left[b]:
                assert len(mine) == left[b] and all(x >= 0 for x in mine)
                live += mine
                left[b] = 0
            else:
                assert d["lens"][b].item() == before[b] and all(x < 0 for x in mine)
    assert not left.any() and len(set(live)) == len(live) == total
    assert d["lens"].tolist() == (lens + new).tolist() and int(err) == 8
    held = sum(-(-int(x) // P) for x in lens + new)
    assert int(d["count"]) == 400 - (held - sum(-(-int(x) // P) for x in lens))
