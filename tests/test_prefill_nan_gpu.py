"""Prefill where a score is NaN: out and lse of the rows that see it are NaN (an lse of -inf would say that the row has
no keys), and the others keep their bits."""

from __future__ import annotations

import dataclasses

import pytest
import torch

import workloads as W
from tests.q8_cases import make
from tests.test_q8_marked_rows_gpu import mark

pytestmark = pytest.mark.gpu
LENS, CHUNK, WINDOW = [300, 90], [200, 40], 60


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def inputs(kind, D, window):
    if kind == "q8":
        return make(CHUNK, LENS, 4, 2, D, 64, window, 32, seed=5, poison=False)
    cache = W.make_prefill_cache(LENS, 2, D, 64, device="cuda", seed=3)
    return W.make_prefill(cache, CHUNK, LENS, 4, 32, window, device="cuda", seed=4)


def run(ops, kind, inp):
    if kind == "bf16":
        return ops.prefill_inputs(inp)
    return ops.prefill_q8(inp.q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens,
                          inp.rel_logits, window=inp.window, scale=inp.scale, max_seq_len=inp.max_seq_len,
                          max_q_len=inp.max_q_len)


def check(ops, kind, inp, bad, hit):
    clean, lclean = run(ops, kind, inp)
    assert bool(torch.isfinite(clean.float()).all()) and bool(torch.isfinite(lclean).all())
    out, lse = run(ops, kind, bad)
    assert bool(torch.isnan(out[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit])


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, WINDOW)])
@pytest.mark.parametrize("key", [10, 90, 150, 299])
def test_key(ops, kind, D, window, key):
    inp = inputs(kind, D, window)
    if kind == "q8":
        bad = mark(inp, "k", 0, key)
    else:
        pool = inp.k_cache.clone()
        pool[int(inp.page_table[0, key // 64]), key % 64, 0, 3] = float("nan")
        bad = dataclasses.replace(inp, k_cache=pool)
    hit = torch.zeros((sum(CHUNK), 4), dtype=torch.bool, device="cuda")
    pos = torch.arange(CHUNK[0], device="cuda") + LENS[0] - CHUNK[0]
    hit[:CHUNK[0], :2] = ((pos >= key) & ((window <= 0) | (pos - key < window)))[:, None]
    check(ops, kind, inp, bad, hit)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("what", ["q", "bias"])
def test_query_or_bias(ops, kind, what):
    inp = inputs(kind, 128, 0)
    hit = torch.zeros((sum(CHUNK), 4), dtype=torch.bool, device="cuda")
    t = inp.rel_logits.clone() if what == "bias" else inp.q.clone()
    for row, h in ((0, 1), (131, 3), (239, 0)):
        t[row, h, 7] = float("nan")
        hit[row, h] = True
    check(ops, kind, inp, dataclasses.replace(inp, **{"rel_logits" if what == "bias" else "q": t}), hit)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_row_without_a_finite_score(ops, kind):
    inp = inputs(kind, 128, 0)
    rel = inp.rel_logits.clone()
    rel[7, 2] = -float("inf")
    out, lse = run(ops, kind, dataclasses.replace(inp, rel_logits=rel))
    assert not out[7, 2].any() and float(lse[7, 2]) == -float("inf")
