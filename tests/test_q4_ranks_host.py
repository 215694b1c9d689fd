"""Tensors of the wrong rank are named by the 4-bit cache's wrappers."""

from __future__ import annotations

import pytest
import torch

import paged_attention_relative_attn_gb300 as ira


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


POOL = torch.zeros((3, 2, 16, 36), dtype=torch.uint8)


@pytest.mark.parametrize("which", ["q", "page_table", "seq_lens", "rel_logits"])
def test_attention_names_the_tensor(which):
    a = dict(q=torch.zeros((2, 4, 64), dtype=torch.bfloat16), page_table=i32(2, 4), seq_lens=i32(2),
             rel_logits=torch.zeros((2, 4, 8)))
    for shape in ((), (2,), (2, 2), (2, 4, 8, 1)):
        if len(shape) == a[which].dim():
            continue
        b = dict(a, **{which: torch.zeros(shape, dtype=a[which].dtype)})
        with pytest.raises(ValueError, match=f"{which}: expected {a[which].dim()} dims"):
            ira.decode_q4(b["q"], POOL, POOL, b["page_table"], b["seq_lens"], b["rel_logits"], window=0, scale=0.1)
        with pytest.raises(ValueError, match=f"{which}: expected {a[which].dim()} dims"):
            ira.prefill_q4(b["q"], i32(3), POOL, POOL, b["page_table"], b["seq_lens"], b["rel_logits"], window=0,
                           scale=0.1, max_seq_len=8, max_q_len=1)


def test_rows_and_tables_name_the_tensor():
    rows, slots = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="slot_map: expected 1 dims"):
        ira.kv_append_q4(rows, rows, slots[0], POOL, POOL)
    with pytest.raises(ValueError, match="slot_map: expected 1 dims"):
        ira.kv_read_q4(slots[0], POOL, POOL)
    with pytest.raises(ValueError, match="k_new: expected 3 dims"):
        ira.kv_append_q4(rows[0], rows[0], slots, POOL, POOL)
    with pytest.raises(TypeError, match="uint8 pools"):
        ira.kv_read_q4(slots, POOL[0], POOL[0])
    with pytest.raises(ValueError, match="seq_lens: expected 1 dims"):
        ira.build_tables(i32(2, 1), i32(2), i32(2, 4), i32(8), i32(1), page_size=16, max_tokens=4)
    with pytest.raises(ValueError, match="page_table: expected 2 dims"):
        ira.build_tables(i32(2), i32(2), i32(8), i32(8), i32(1), page_size=16, max_tokens=4)
