"""Prefill under biases used as masks: -1e4, -1e9, -1e30 or fp32's lowest number on far keys (whole tiles before the
first that counts) or on every key of a row."""

from __future__ import annotations

import dataclasses

import pytest
import torch

import workloads as W
from tests.helpers import assert_close, oracle_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


@pytest.mark.parametrize("low", [-1e4, -1e9, -1e30, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("D", [64, 128])
def test_far_keys_and_whole_rows_masked(ops, low, D):
    cache = W.make_prefill_cache([400, 300], 1, D, 64, device="cuda", seed=3)
    inp = W.make_prefill(cache, [140, 70], [400, 300], 2, 512, 0, device="cuda", seed=4)
    rel = inp.rel_logits.clone()
    rel[:140, :, 10:] = low
    rel[140:] = low
    if low > -1e6:  # fp32 holds score + bias to 2^-10: as the oracle does
        want = dataclasses.replace(inp, rel_logits=rel)
        cut = 0
    else:           # the scores of a row masked everywhere round to one number: the mean of its values
        r2 = rel.clone()
        r2[140:] = 0.0
        q = inp.q.clone()
        q[140:] = 0.0 if low < -1e29 else q[140:]
        want = dataclasses.replace(inp, rel_logits=r2, q=q)
        cut = 0 if low < -1e29 else 70  # at -1e9 they round to steps of 64: left out below
    out, lse = ops.prefill_inputs(dataclasses.replace(inp, rel_logits=rel))
    assert bool(torch.isfinite(out.float()).all())
    ro, rl, rows = oracle_prefill(want)
    n = len(rows) - cut
    assert_close(out[:n], ro[:n], what=f"mask {low}")
    assert_close(out[:140], ro[:140], lse[:140], rl[:140], what=f"mask {low}, lse")
