"""The 4-bit cache and the step tables without a GPU: pins of the oracle, host-side refusals of the C ABI and of
the Python wrappers, workspace sizes."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.q4 as q4

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    return _lib


# ------------------------------------------------------------------ the oracle

def test_scale_is_smallest_with_five_bits():
    rng = np.random.default_rng(0)
    for a in np.concatenate([np.abs(rng.standard_normal(50)), 7 * 2.0 ** np.arange(-6, 7), [1e-20, 3e30]]):
        a = float(torch.tensor(a).to(BF16))
        s = q4.group_scale(a)
        m, _ = np.frexp(s)
        assert m * 32 == int(m * 32) and 7 * s >= a
        lower = s - 2.0 ** (np.floor(np.log2(s)) - 4) if m != 0.5 else s * 31 / 32
        assert 7 * lower < a
    assert q4.group_scale(2.0 ** -101) == 0.0


def test_rounding_by_hand():
    s = 0.5
    for v, x in [(0.25, 0), (0.26, 1), (0.75, 1), (0.76, 2), (-0.25, 0), (-0.75, -1), (-0.8, -2), (3.5, 7), (0.0, 0)]:
        assert q4.round_x(v, s) == x, v


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_row_order_is_a_permutation_and_rows_come_back(D, is_v):
    assert sorted(q4.nibble_of(c, D, is_v) for c in range(D)) == list(range(D))
    rng = np.random.default_rng(1)
    pool = np.zeros((3, 2, 32, 9 * D // 16), dtype=np.uint8)
    rows = torch.from_numpy(rng.standard_normal((5, 2, D))).to(BF16).double().numpy()
    slots = [0, 17, 31, 64, -1]
    out = q4.ref_append_q4(pool, rows, slots, is_v)
    vals = q4.read_pool(out, is_v)
    for t, slot in enumerate(slots[:4]):
        got = vals[slot // 32, slot % 32]
        s = np.abs(rows[t].reshape(2, -1, 32)).max(-1, keepdims=True) / 7 * (1 + 2.0 ** -4)
        assert np.all(np.abs(got - rows[t]).reshape(2, -1, 32) <= s / 2 + 1e-12)
        # every value is a bf16 number
        assert np.array_equal(torch.from_numpy(got).to(BF16).double().numpy(), got)
    assert np.count_nonzero(vals[0, 1]) == 0 or out[0, 0].any()  # untouched places keep their bytes
    assert not out[2, :, 16:].any()


def test_planted_mistakes_in_the_format_are_seen(monkeypatch):
    rng = np.random.default_rng(2)
    rows = torch.from_numpy(rng.standard_normal((1, 1, 64))).to(BF16).double().numpy()
    pool = np.zeros((1, 1, 16, 36), dtype=np.uint8)
    good = q4.ref_append_q4(pool, rows, [3], False)
    monkeypatch.setattr(q4, "nibble_of", lambda c, D, is_v: c)
    assert not np.array_equal(good, q4.ref_append_q4(pool, rows, [3], False))


def test_tables_by_hand():
    # page size 16: request 0 crosses a page, 1 ends (2 pages back), 2 stays inside its page, 3 starts
    pt = np.array([[5, 0, 0], [1, 2, 0], [7, 0, 0], [0, 0, 0]])
    free = np.array([9, 8, 0, 0, 0, 0, 0, 0, 0, 0])
    r = q4.ref_build_tables([16, 20, 3, 0], [1, -1, 2, 17], pt, free, 2, 16, 24)
    assert list(r["free"][:4]) == [9, 8, 1, 2]          # pages 1, 2 on top
    assert r["table"][0, 1] == 2                         # popped first
    assert list(r["table"][3, :2]) == [1, 8] and r["left"] == 1
    assert list(r["kv_lens"]) == [17, 0, 5, 17] and list(r["cu"]) == [0, 1, 1, 3, 20]
    assert list(r["slots"][:4]) == [2 * 16, 7 * 16 + 3, 7 * 16 + 4, 1 * 16] and r["slots"][19] == 8 * 16
    assert list(r["slots"][20:]) == [-1] * 4 and not r["bits"]


# ------------------------------------------------------------------ refusals of the C ABI

def test_append_and_read_validation(lib):
    a = dict(k_new=16, v_new=16, slot_map=8, T=2, H_kv=2, D=64, page_size=16, num_pages=8, k_cache=16, v_cache=16,
             device_error=None, stream=None)
    ap = lambda **o: lib.inkling_rel_attn_kv_append_q4(**{**a, **o})  # noqa: E731
    b = {**a, "k_rows": 16, "v_rows": 16}
    del b["k_new"], b["v_new"]
    rd = lambda **o: lib.inkling_rel_attn_kv_read_q4(**{**b, **o})  # noqa: E731
    for f in (ap, rd):
        assert f(D=96) == -1 and f(page_size=24) == -1 and f(page_size=272) == -1 and f(num_pages=0) == -1
        assert f(H_kv=0) == -1 and f(T=-1) == -1 and f(slot_map=None) == -1 and f(v_cache=None) == -1
        assert f(T=0) == 0
        assert f(k_cache=24) == -2 and f(slot_map=12) == -2 and f(device_error=2) == -2
    assert ap(k_new=24) == -2 and rd(v_rows=8) == -2


def test_tables_validation(lib):
    a = dict(seq_lens=4, new_lens=4, page_table=4, page_table_stride=4, free_pages=4, free_count=4, B=2, page_size=16,
             num_pages=8, max_tokens=4, kv_lens=4, cu_seqlens_q=4, slot_map=8, free_left=4, device_error=None,
             stream=None)
    f = lambda **o: lib.inkling_rel_attn_build_tables(**{**a, **o})  # noqa: E731
    assert f(B=-1) == -1 and f(B=8193) == -1 and f(max_tokens=-1) == -1 and f(page_size=40) == -1
    assert f(num_pages=0) == -1 and f(page_table_stride=0) == -1 and f(page_table_stride=1 << 28) == -1
    assert f(seq_lens=None) == -1 and f(slot_map=None) == -1 and f(free_left=None) == -1
    assert f(B=0) == 0
    assert f(slot_map=4) == -2 and f(kv_lens=6) == -2
    # no slots asked for: the map may be missing (the next check is reached)
    assert f(max_tokens=0, slot_map=None, kv_lens=6) == -2


def test_decode_q4_validation(lib):
    a = dict(q=16, k_cache=16, v_cache=16, page_table=4, page_table_stride=4, seq_lens=4, rel_logits=4, B=2, q_len=1,
             H_q=4, H_kv=2, D=64, page_size=16, num_pages=16, R=32, window=32, scale=0.125, out=16, lse_out=None,
             workspace=None, workspace_bytes=0, device_error=None, stream=None)
    f = lambda **o: lib.inkling_rel_attn_decode_q4(**{**a, **o})  # noqa: E731
    assert f(q_len=0) == -1 and f(q_len=65) == -1 and f(D=96) == -1 and f(H_q=5) == -1 and f(H_q=34) == -1
    assert f(page_size=24) == -1 and f(R=0) == -1 and f(B=-1) == -1 and f(q=None) == -1
    assert f(scale=float("nan")) == -1
    assert f(B=0) == 0
    assert f(q=24) == -2 and f(workspace=8) == -2 and f(seq_lens=6) == -2


def test_prefill_q4_validation_and_workspace(lib):
    a = dict(q=16, cu_seqlens_q=4, k_cache=16, v_cache=16, page_table=4, page_table_stride=4, seq_lens=4,
             rel_logits=16, B=1, T=4, max_q_len=4, H_q=4, H_kv=2, D=64, page_size=16, num_pages=4, R=32, window=0,
             scale=0.1, max_seq_len=64, out=16, lse_out=None, workspace=256, workspace_bytes=1 << 20,
             device_error=None, stream=None)
    f = lambda **o: lib.inkling_rel_attn_prefill_q4(**{**a, **o})  # noqa: E731
    assert f(R=30) == -1 and f(D=96) == -1 and f(max_q_len=-1) == -1 and f(cu_seqlens_q=None) == -1
    assert f(B=65536, max_q_len=128) == -1
    assert f(T=0) == 0 and f(B=0) == 0 and f(max_q_len=0) == 0
    assert f(rel_logits=8) == -2 and f(workspace=128) == -2
    ws = lib.inkling_rel_attn_prefill_q4_workspace_size
    pool = lambda B, pages, H, D: (B * pages * 64 * H * D * 2 + 255) // 256 * 256  # noqa: E731
    assert ws(3, 100, 2, 64, 0, 1000) == 256 + 256 + 2 * pool(3, 16, 2, 64)
    # a window bounds what a chunk sees: 512 - 1 + 100 keys from a multiple of 64 on
    assert ws(3, 100, 2, 64, 512, 100000) == 256 + 256 + 2 * pool(3, 11, 2, 64)
    assert ws(3, 100, 2, 64, 512, 200) == 256 + 256 + 2 * pool(3, 4, 2, 64)
    assert ws(0, 100, 2, 64, 0, 1000) == 0


# ------------------------------------------------------------------ refusals of the wrappers

def test_wrappers_refuse_wrong_tensors():
    import paged_attention_relative_attn_gb300 as ira
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rows = torch.zeros((4, 2, 64), dtype=BF16)
    pool = torch.zeros((3, 2, 16, 36), dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="slot_map"):
        ira.kv_append_q4(rows, rows, slots.int(), pool, pool)
    with pytest.raises(TypeError, match="k_new"):
        ira.kv_append_q4(rows.float(), rows, slots, pool, pool)
    with pytest.raises(ValueError, match="contiguous|CUDA"):
        ira.kv_append_q4(rows.transpose(0, 1), rows, slots, pool, pool)
    with pytest.raises(ValueError, match="dims"):
        ira.kv_read_q4(slots.view(2, 2), pool, pool)
    with pytest.raises(ValueError, match="rows of 40 bytes"):
        ira.kv_read_q4(slots, torch.zeros((3, 2, 16, 40), dtype=torch.uint8), torch.zeros((3, 2, 16, 40), dtype=torch.uint8))
    with pytest.raises(ValueError, match="shapes differ"):
        ira.kv_read_q4(slots, pool, pool[:2])
    with pytest.raises(ValueError, match="inconsistent"):
        ira.kv_append_q4(rows, rows, slots[:3], pool, pool)
    with pytest.raises(ValueError, match="max_tokens"):
        ira.build_tables(i32(2), i32(2), i32(2, 4), i32(8), i32(1), page_size=16)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.build_tables(i32(2), i32(3), i32(2, 4), i32(8), i32(1), page_size=16, max_tokens=4)
    with pytest.raises(TypeError, match="page_table"):
        ira.build_tables(i32(2), i32(2), i32(2, 4).long(), i32(8), i32(1), page_size=16, max_tokens=4)
    rel = torch.zeros((2, 4, 8))
    q = torch.zeros((2, 4, 64), dtype=BF16)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.decode_q4(q, pool, pool, i32(2, 4), i32(2), rel[:, :3].contiguous(), window=0, scale=0.1)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.decode_q4(q, pool, pool, i32(2, 4), i32(2), rel, q_len=2, window=0, scale=0.1)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.prefill_q4(q, i32(2), pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1, max_seq_len=8, max_q_len=1)
    # the right types and shapes, but on the CPU
    for call in (lambda: ira.kv_append_q4(rows, rows, slots, pool, pool), lambda: ira.kv_read_q4(slots, pool, pool),
                 lambda: ira.decode_q4(q, pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1),
                 lambda: ira.build_tables(i32(2), i32(2), i32(2, 4), i32(8), i32(1), page_size=16, max_tokens=4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
