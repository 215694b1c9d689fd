"""A prefill row does not depend on the other rows of its call: their scores may be of any size."""

from __future__ import annotations

import dataclasses

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [2.0 ** 21, -1e9, -3e38])
@pytest.mark.parametrize("D,P", [(64, 64), (128, 64), (128, 16)])
def test_rows_beside_one_of_huge_scores_keep_their_bits(value, D, P):
    import paged_attention_relative_attn_gb300 as ops
    cache = W.make_prefill_cache([400, 300], 1, D, P, device="cuda", seed=3)
    inp = W.make_prefill(cache, [140, 70], [400, 300], 2, 512, 0, device="cuda", seed=4)
    want, lwant = ops.prefill_inputs(inp)
    rel = inp.rel_logits.clone()
    huge = [3, 57, 130, 200]  # a row of each of some warps
    rel[huge] = value
    out, lse = ops.prefill_inputs(dataclasses.replace(inp, rel_logits=rel))
    keep = torch.ones(210, dtype=torch.bool, device="cuda")
    keep[huge] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], lwant[keep])
    assert bool(torch.isfinite(out.float()).all())
