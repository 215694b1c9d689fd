"""Decode over the bf16 cache where scores are NaN: out and lse of those rows are NaN however many splits there are (zeros
and an lse of -inf would say that the row has no keys); the others keep their bits."""

from __future__ import annotations

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
LENS = [700, 5, 1300]


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def inputs(q_len, D, window):
    cache = W.make_prefill_cache(LENS, 2, D, 64, device="cuda", seed=7)
    return W.make_prefill(cache, [q_len] * 3, LENS, 6, 32, window, device="cuda", seed=8)


def run(ops, inp, q_len, splits, **kw):
    a = dict(q=inp.q, k=inp.k_cache, rel=inp.rel_logits)
    a.update(kw)
    args = (a["q"], a["k"], inp.v_cache, inp.page_table, inp.seq_lens, a["rel"])
    kw = dict(window=inp.window, scale=inp.scale, max_seq_len=inp.max_seq_len, num_splits=splits)
    return ops.decode(*args, **kw) if q_len == 1 else ops.decode_multi(*args, q_len=q_len, **kw)


def check(ops, inp, q_len, splits, hit, **bad):
    clean, lclean = run(ops, inp, q_len, splits)
    assert bool(torch.isfinite(clean.float()).all()) and bool(torch.isfinite(lclean).all())
    out, lse = run(ops, inp, q_len, splits, **bad)
    assert bool(torch.isnan(out[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit])


@pytest.mark.parametrize("splits", [1, 3, 9])
@pytest.mark.parametrize("q_len,D,window", [(1, 64, 0), (1, 128, 0), (4, 64, 0), (4, 128, 0), (1, 128, 100), (4, 128, 100)])
def test_query(ops, q_len, D, window, splits):
    """Every score of the row is NaN, in every split."""
    inp = inputs(q_len, D, window)
    q = inp.q.clone()
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for row, h in ((0, 1), (q_len, 5), (3 * q_len - 1, 0)):
        q[row, h, 9] = float("nan")
        hit[row, h] = True
    check(ops, inp, q_len, splits, hit, q=q)


@pytest.mark.parametrize("splits", [1, 3, 9])
@pytest.mark.parametrize("q_len,D", [(1, 64), (1, 128), (4, 64), (4, 128)])
@pytest.mark.parametrize("key", [3, 400, 697])
def test_key(ops, q_len, D, splits, key):
    inp = inputs(q_len, D, 0)
    k = inp.k_cache.clone()
    k[int(inp.page_table[0, key // 64]), key % 64, 1, 0] = float("nan")
    hit = torch.zeros(inp.q.shape[:2], dtype=torch.bool, device="cuda")
    for i in range(q_len):
        hit[i, 3:] = LENS[0] - q_len + i >= key
    check(ops, inp, q_len, splits, hit, k=k)
