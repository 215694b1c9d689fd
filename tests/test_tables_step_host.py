"""The tables call with lengths of the step, without a GPU: its checks, plain and packed, and the wrapper's."""

from __future__ import annotations

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    return _lib


ARGS = dict(seq_lens=4, new_lens=4, page_table=4, page_table_stride=4, free_pages=4, free_count=4, B=2, page_size=16,
            num_pages=8, max_tokens=4, kv_lens=4, cu_seqlens_q=4, slot_map=8, free_left=4, step_lens=4, device_error=0,
            stream=0)


def test_checks_plain_and_packed(lib):
    call, pack, count = lib.PACKED["inkling_rel_attn_build_tables_step"]
    assert count == len(ARGS)
    for name, bad, code in (("step_lens", 2, -2), ("kv_lens", 6, -2), ("device_error", 2, -2), ("slot_map", 4, -2),
                            ("B", -1, -1), ("page_size", 40, -1), ("free_left", 0, -1), ("max_tokens", -1, -1)):
        a = {**ARGS, name: bad}
        assert lib.inkling_rel_attn_build_tables_step(**a) == code, name
        assert lib.inkling_rel_attn_packed(call, pack(*a.values()), count) == code, name
    # optional: the check behind it is reached without it
    assert lib.inkling_rel_attn_build_tables_step(**{**ARGS, "step_lens": 0, "device_error": 2}) == -2
    assert lib.inkling_rel_attn_build_tables_step(**{**ARGS, "B": 0}) == 0
    assert lib.inkling_rel_attn_packed(call, pack(*ARGS.values()), count + 1) == -1


def test_wrapper_names_it():
    import paged_attention_relative_attn_gb300 as ira
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    call = lambda s: ira.build_tables(i32(2), i32(2), i32(2, 4), i32(8), i32(1), page_size=16, max_tokens=4,  # noqa: E731
                                      step_lens=s)
    with pytest.raises(TypeError, match="step_lens"):
        call(i32(2).long())
    with pytest.raises(ValueError, match="step_lens"):
        call(i32(2, 1))
    with pytest.raises(ValueError, match="inconsistent"):
        call(i32(3))
    with pytest.raises(ValueError, match="CUDA"):
        call(i32(2))
