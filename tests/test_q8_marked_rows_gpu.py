"""Marked rows (tokens with a NaN) of the 8-bit cache: what a token that sees one gets depends on neither the bias, nor
the weight, nor the order in which keys are taken, nor the other sequences of the batch."""

from __future__ import annotations

import dataclasses

import pytest
import torch

from tests.q8_cases import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def decode(ops, inp, q_len=1):
    return ops.decode_q8(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits, q_len=q_len,
                         window=inp.window, scale=inp.scale)


def mark(inp, side, b, j):
    """The inputs with token j of sequence b marked in K or V, for KV head 0."""
    pool = (inp.k_cache if side == "k" else inp.v_cache).clone()
    n, H, P, row = pool.shape
    D = row - 1
    place = j % P
    block = pool.view(n, H, P // 16, -1)[int(inp.page_table[b, j // P]), 0, place // 16]
    block[16 * D + 4 + place % 16 // 8] |= 1 << place % 8
    return dataclasses.replace(inp, **{side + "_cache": pool})


def is_nan(x):
    return bool(torch.isnan(x.float()).all())


@pytest.mark.parametrize("D,q_len,G", [(64, 1, 3), (128, 1, 6), (64, 4, 2), (128, 2, 3)])
@pytest.mark.parametrize("distance", [0, 7, 31, 32, 33, 100, 290])
def test_key_under_a_bias_of_minus_infinity(ops, D, q_len, G, distance):
    """NaN + -inf is NaN: at distances inside the bias table, at its end and past it.  Other heads keep their bits."""
    L, H, R = 300, 2, 32
    inp = make([q_len], [L], G * H, H, D, 16, 0, R, seed=distance)
    rel = inp.rel_logits.clone()
    rel[..., min(distance, R - 1)] = -float("inf")
    inp = dataclasses.replace(inp, rel_logits=rel)
    clean, lclean = decode(ops, inp, q_len)
    assert bool(torch.isfinite(clean.float()).all())
    out, lse = decode(ops, mark(inp, "k", 0, L - 1 - distance), q_len)
    sees = [i for i in range(q_len) if i >= q_len - 1 - distance]
    for i in range(q_len):
        if i in sees:
            assert is_nan(out[i, :G]) and is_nan(lse[i, :G]), i
        else:
            assert torch.equal(out[i, :G], clean[i, :G]) and torch.equal(lse[i, :G], lclean[i, :G]), i
    assert torch.equal(out[:, G:], clean[:, G:]) and torch.equal(lse[:, G:], lclean[:, G:])


@pytest.mark.parametrize("others", [[], [5000], [17, 3, 900]])
@pytest.mark.parametrize("at", [0, 40, 100, 200, 270, 290, 299])
@pytest.mark.parametrize("D,q_len,low", [(64, 1, -1e4), (128, 1, -float("inf")), (128, 4, -1e4), (64, 4, -float("inf"))])
def test_value_whose_weight_is_nought(ops, D, q_len, low, at, others):
    """0 * NaN is NaN: before and after the key that has all of the weight, whatever the rest of the batch.  lse, and
    the tokens that do not see the row, keep their bits."""
    L, H, G, R = 300, 2, 2, 512
    lens = [L] + [max(x, q_len) for x in others]
    inp = make([q_len] * len(lens), lens, G * H, H, D, 64, 0, R, seed=at + len(others))
    rel = inp.rel_logits.clone()
    for i in range(q_len):
        rel[i] = low
        rel[i, :, L - q_len + i - 150] = 0.0  # key 150 alone counts
    inp = dataclasses.replace(inp, rel_logits=rel)
    clean, lclean = decode(ops, inp, q_len)
    assert bool(torch.isfinite(clean.float()).all())
    out, lse = decode(ops, mark(inp, "v", 0, at), q_len)
    for i in range(q_len):
        if at <= L - q_len + i:
            assert is_nan(out[i, :G]), i
        else:
            assert torch.equal(out[i, :G], clean[i, :G]), i
    assert torch.equal(out[:, G:], clean[:, G:]) and torch.equal(out[q_len:], clean[q_len:])
    assert torch.equal(lse, lclean)


@pytest.mark.parametrize("L", [20, 40000])
@pytest.mark.parametrize("D,q_len", [(64, 1), (128, 1), (128, 4)])
def test_row_without_a_finite_score(ops, D, q_len, L):
    """Every visible score is -inf: out = 0 and lse = -inf beside a marked value too, whether one thread block has the
    whole row or many share it; a marked key makes it NaN."""
    inp = make([q_len], [L], 4, 2, D, 64, 0, 32, seed=L)
    rel = inp.rel_logits.clone()
    rel[:, 1] = -float("inf")
    inp = dataclasses.replace(inp, rel_logits=rel)
    out, lse = decode(ops, mark(inp, "v", 0, 3), q_len)
    assert not out[:, 1].any() and bool((lse[:, 1] == -float("inf")).all())
    assert is_nan(out[:, 0]) and bool(torch.isfinite(lse[:, 0]).all())
    out, lse = decode(ops, mark(inp, "k", 0, 3), q_len)
    assert is_nan(out[:, :2]) and is_nan(lse[:, :2])
    assert bool(torch.isfinite(out[:, 2:].float()).all())
