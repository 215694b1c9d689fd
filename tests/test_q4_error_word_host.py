"""An error word without a word is refused by every call on the 4-bit cache and the tables."""

from __future__ import annotations

import pytest
import torch

import paged_attention_relative_attn_gb300 as ira


@pytest.mark.parametrize("word", [torch.zeros(0, dtype=torch.int32), torch.zeros((), dtype=torch.int32),
                                  torch.zeros(1, dtype=torch.int64)])
def test_error_word(word):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rows, slots = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    pool, q, rel = torch.zeros((3, 2, 16, 36), dtype=torch.uint8), rows[:2].repeat(1, 2, 1), torch.zeros((2, 4, 8))
    ws = torch.zeros(1, dtype=torch.uint8)
    for call in (lambda **k: ira.kv_append_q4(rows, rows, slots, pool, pool, **k),
                 lambda **k: ira.kv_read_q4(slots, pool, pool, **k),
                 lambda **k: ira.decode_q4(q, pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1, workspace=ws, **k),
                 lambda **k: ira.prefill_q4(q, i32(3), pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1,
                                            max_seq_len=8, max_q_len=1, workspace=ws, **k),
                 lambda **k: ira.build_tables(i32(2), i32(2), i32(2, 4), i32(8), i32(1), page_size=16, max_tokens=4, **k)):
        with pytest.raises(TypeError, match="device_error"):
            call(device_error=word)
