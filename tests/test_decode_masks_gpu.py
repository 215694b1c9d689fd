"""Decode over the bf16 cache with a bias of -inf as a mask, on the far keys (whole splits of them) or on a whole row,
however many splits there are."""

from __future__ import annotations

import dataclasses

import pytest
import torch

from tests.helpers import assert_close, oracle_prefill
from tests.test_decode_nan_gpu import LENS, inputs, ops, run  # noqa: F401 (ops: a fixture)

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("splits", [0, 1, 3, 9])
@pytest.mark.parametrize("q_len,D,window", [(1, 64, 0), (1, 128, 0), (4, 64, 0), (4, 128, 0), (1, 128, 100), (4, 128, 100)])
def test_far_keys(ops, q_len, D, window, splits):  # noqa: F811
    inp = inputs(q_len, D, window)
    rel = inp.rel_logits.clone()
    rel[..., 10:] = -INF
    out, lse = run(ops, inp, q_len, splits, rel=rel)
    ro, rl, rows = oracle_prefill(dataclasses.replace(inp, rel_logits=rel))
    assert len(rows) == len(LENS) * q_len
    assert_close(out, ro, lse, rl, what=f"splits {splits}")


@pytest.mark.parametrize("splits", [0, 1, 3, 9])
@pytest.mark.parametrize("q_len,D", [(1, 64), (1, 128), (4, 64), (4, 128)])
def test_rows_and_near_keys(ops, q_len, D, splits):  # noqa: F811
    """A row masked everywhere gets out = 0 and lse = -inf; one whose near keys are masked keeps the far ones."""
    inp = inputs(q_len, D, 0)
    rel = inp.rel_logits.clone()
    rel[0, 1] = -INF
    rel[-1, 5, :-1] = -INF
    out, lse = run(ops, inp, q_len, splits, rel=rel)
    assert not out[0, 1].any() and float(lse[0, 1]) == -INF
    some = rel.clone()
    some[0, 1] = 0.0
    ro, rl, _ = oracle_prefill(dataclasses.replace(inp, rel_logits=some))
    out, lse = out.clone(), lse.clone()
    out[0, 1] = torch.from_numpy(ro[0, 1]).to(out)
    lse[0, 1] = float(rl[0, 1])
    assert_close(out, ro, lse, rl, what=f"splits {splits}")
