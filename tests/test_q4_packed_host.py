"""The packed form of the calls on the 4-bit cache, without a GPU: it reaches the same checks as the plain calls,
argument by argument, and refuses words that do not fit."""

from __future__ import annotations

import pytest


@pytest.fixture(scope="module")
def lib():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    return _lib


def plain_args():
    """Per call its arguments in order: (name, a value that passes, a value that is refused and its code)."""
    ok = lambda n, v: (n, v, None, None)  # noqa: E731
    a16, a4, a8 = (lambda n: (n, 16, 8, -2)), (lambda n: (n, 4, 2, -2)), (lambda n: (n, 8, 4, -2))
    rows = [("T", 4, -1, -1), ("H_kv", 2, 0, -1), ("D", 64, 32, -1), ("page_size", 16, 8, -1), ("num_pages", 8, 0, -1)]
    return {
        "inkling_rel_attn_build_tables": [
            a4("seq_lens"), a4("new_lens"), a4("page_table"), ("stride", 4, 0, -1), a4("free_pages"), a4("free_count"),
            ("B", 2, -1, -1), ("page_size", 16, 40, -1), ("num_pages", 8, 0, -1), ("max_tokens", 4, -1, -1),
            a4("kv_lens"), a4("cu"), a8("slot_map"), a4("free_left"), a4("device_error"), ok("stream", 0)],
        "inkling_rel_attn_kv_append_q4": [
            a16("k_new"), a16("v_new"), a8("slot_map"), *rows, a16("k_cache"), a16("v_cache"), a4("device_error"),
            ok("stream", 0)],
        "inkling_rel_attn_kv_read_q4": [
            a8("slot_map"), a16("k_cache"), a16("v_cache"), *rows, a16("k_rows"), a16("v_rows"), a4("device_error"),
            ok("stream", 0)],
        "inkling_rel_attn_decode_q4": [
            a16("q"), a16("k"), a16("v"), a4("page_table"), ("stride", 4, 0, -1), a4("seq_lens"), a4("rel"),
            ("B", 2, -1, -1), ("q_len", 1, 65, -1), ("H_q", 4, 3, -1), ("H_kv", 2, 0, -1), ("D", 64, 63, -1),
            ("page_size", 16, 17, -1), ("num_pages", 8, 0, -1), ("R", 8, 0, -1), ok("window", 0),
            ("scale", 0.1, float("nan"), -1), a16("out"), a4("lse"), a16("workspace"), ok("workspace_bytes", 1 << 30),
            a4("device_error"), ok("stream", 0)],
        "inkling_rel_attn_prefill_q4": [
            a16("q"), a4("cu"), a16("k"), a16("v"), a4("page_table"), ("stride", 4, 0, -1), a4("seq_lens"), a16("rel"),
            ("B", 2, -1, -1), ("T", 4, -1, -1), ("max_q_len", 2, -1, -1), ("H_q", 4, 3, -1), ("H_kv", 2, 0, -1),
            ("D", 64, 63, -1), ("page_size", 16, 17, -1), ("num_pages", 8, 0, -1), ("R", 8, 6, -1), ok("window", 0),
            ("scale", 0.1, float("nan"), -1), ("max_seq_len", 64, -1, -1), a16("out"), a4("lse"),
            ("workspace", 256, 128, -2), ok("workspace_bytes", 1 << 30), a4("device_error"), ok("stream", 0)],
    }


@pytest.mark.parametrize("name", sorted(plain_args()))
def test_packed_reaches_every_argument(lib, name):
    spec = plain_args()[name]
    call, pack, count = lib.PACKED[name]
    assert count == len(spec)
    good = [s[1] for s in spec]
    for i, (arg, value, bad, code) in enumerate(spec):
        if bad is None:
            continue
        args = good[:i] + [bad] + good[i + 1:]
        assert getattr(lib, name)(*args) == code, arg
        assert lib.inkling_rel_attn_packed(call, pack(*args), count) == code, arg
        if isinstance(value, int) and arg in ("T", "B", "H_kv", "D", "R", "stride", "page_size", "num_pages", "max_tokens"):
            wide = good[:i] + [value + (1 << 32)] + good[i + 1:]
            assert lib.inkling_rel_attn_packed(call, pack(*wide), count) == -1, arg
    assert lib.inkling_rel_attn_packed(call, pack(*good), count - 1) == -1


def test_packed_refuses_unknown_calls(lib):
    assert lib.inkling_rel_attn_packed(5, b"\0" * 256, 16) == -1
    assert lib.inkling_rel_attn_packed(-1, b"\0" * 256, 16) == -1
    assert lib.inkling_rel_attn_packed(0, None, 16) == -1
