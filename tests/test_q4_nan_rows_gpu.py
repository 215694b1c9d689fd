"""Tokens with a NaN in the 4-bit cache: whoever sees one gets NaN, whatever bias or weight it has there, for one token
and for several; who does not keeps its bits."""

from __future__ import annotations

import dataclasses

import pytest
import torch

from tests.q4_cases import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def decode(ops, inp, q_len):
    return ops.decode_q4(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits, q_len=q_len,
                         window=inp.window, scale=inp.scale)


def with_nan(ops, inp, side, j):
    """The inputs with a NaN in every group of KV head 0 of token j of sequence 0, in K or V."""
    n, H, P, row = inp.k_cache.shape
    D = 16 * row // 9
    slot = torch.tensor([int(inp.page_table[0, j // P]) * P + j % P], device="cuda")
    kr, vr = ops.kv_read_q4(slot, inp.k_cache, inp.v_cache)
    rows = (kr if side == "k" else vr).clone()
    rows[0, 0] = float("nan")
    k, v = inp.k_cache.clone(), inp.v_cache.clone()
    ops.kv_append_q4(rows, rows, slot, k, v)
    return dataclasses.replace(inp, **({"k_cache": k} if side == "k" else {"v_cache": v}))


def check(ops, inp, bad, q_len, G, sees, lse_too):
    clean, lclean = decode(ops, inp, q_len)
    assert bool(torch.isfinite(clean.float()).all())
    out, lse = decode(ops, bad, q_len)
    for i in range(q_len):
        if sees(i):
            assert bool(torch.isnan(out[i, :G].float()).all()), i
            assert bool(torch.isnan(lse[i, :G]).all()) if lse_too else torch.equal(lse[i], lclean[i]), i
        else:
            assert torch.equal(out[i, :G], clean[i, :G]) and torch.equal(lse[i, :G], lclean[i, :G]), i


@pytest.mark.parametrize("D,q_len,G", [(64, 1, 3), (128, 1, 6), (64, 4, 2), (128, 2, 3), (128, 8, 1)])
@pytest.mark.parametrize("distance", [0, 7, 31, 32, 33, 100, 290])
def test_key_under_a_bias_of_minus_infinity(ops, D, q_len, G, distance):
    L, R = 300, 32
    inp = make([q_len], [L], 2 * G, 2, D, 16, 0, R, seed=distance)
    rel = inp.rel_logits.clone()
    rel[..., min(distance, R - 1)] = -float("inf")
    inp = dataclasses.replace(inp, rel_logits=rel)
    check(ops, inp, with_nan(ops, inp, "k", L - 1 - distance), q_len, G, lambda i: i >= q_len - 1 - distance, True)


@pytest.mark.parametrize("at", [0, 40, 100, 200, 270, 290, 299])
@pytest.mark.parametrize("D,q_len,low", [(64, 1, -1e4), (128, 1, -float("inf")), (128, 4, -1e4), (64, 4, -float("inf"))])
def test_value_whose_weight_is_nought(ops, D, q_len, low, at):
    """Before and after the key that has all of the weight."""
    L, G, R = 300, 2, 512
    inp = make([q_len], [L], 2 * G, 2, D, 64, 0, R, seed=at)
    rel = inp.rel_logits.clone()
    for i in range(q_len):
        rel[i] = low
        rel[i, :, L - q_len + i - 150] = 0.0  # key 150 alone counts
    inp = dataclasses.replace(inp, rel_logits=rel)
    check(ops, inp, with_nan(ops, inp, "v", at), q_len, G, lambda i: at <= L - q_len + i, False)
