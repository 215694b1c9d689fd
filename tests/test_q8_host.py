"""The 8-bit cache without a GPU: pins of the oracle, refusals of the C ABI, of its packed form and of the Python
wrappers, workspace sizes."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.q8 as q8
from tests.test_q4_packed_host import plain_args

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    return _lib


# ------------------------------------------------------------------ the oracle

def test_e4m3_numbers_by_hand():
    v = q8.VALUES
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[7] == 7 * 2.0 ** -9 and v[8] == 2.0 ** -6
    assert v[0x38] == 1.0 and v[0x39] == 1.125 and v[0x7e] == 448 and v[0xfe] == -448 and np.isnan(v[0x7f])
    for x, b in [(1.0625, 0x38), (1.1875, 0x3a), (500.0, 0x7e), (-1e30, 0xfe), (2.0 ** -10, 0), (3 * 2.0 ** -10, 2),
                 (-0.0, 0x80), (464.0, 0x7e)]:
        assert q8.e4m3_byte(x) == b, x


def test_rounding_is_that_of_the_type():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(200) * 2.0 ** rng.integers(-11, 9, 200), q8.VALUES[np.isfinite(q8.VALUES)]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [q8.e4m3_byte(float(y)) for y in x] == list(want)
    ties = np.concatenate([x.astype(np.float64), (q8.MAGS[1:] + q8.MAGS[:-1]) / 2, [1e30, -500.0, 2.0 ** -70, -0.0]])
    assert [q8.e4m3_byte(float(y)) for y in ties] == list(q8.e4m3_bytes(ties))


def test_exponent_is_the_smallest_that_fits():
    for a, e in [(0.0, -60), (448.0, 0), (449.0, 1), (1.75, -8), (1.7578125, -7), (2.0 ** -70, -60), (2.0 ** 100, 55)]:
        assert q8.exponent_for(a) == e, a


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_order_is_a_permutation_of_units(D, is_v):
    at = q8.places(D, is_v)
    assert sorted(at.flatten()) == list(range(16 * D))
    assert np.array_equal(at[:, 1::8] - at[:, 0::8], np.ones((16, D // 8)))  # 8 channels side by side
    # what a quarter warp (K, and V of 128 channels: 16 bytes a lane) or half of one (V of 64: 8 bytes) reads
    # together lies in different banks
    if is_v and D == 64:
        got = {(at[2 * t, 8 * g]) % 128 for g in range(4) for t in range(4)}
        assert len(got) == 16
    elif is_v:
        assert len({at[2 * t, 16 * g] % 128 for g in range(2) for t in range(4)}) == 8
    else:
        assert len({at[g, 16 * t] % 128 for g in range(2) for t in range(4)}) == 8


def test_rows_join_and_come_back():
    rng = np.random.default_rng(1)
    bf = lambda a: torch.from_numpy(a).to(BF16).double().numpy()  # noqa: E731
    for D, is_v in ((64, True), (128, False)):
        pool = np.zeros((2, 1, 32, D + 1), dtype=np.uint8)
        a, b = bf(rng.standard_normal((5, 1, D))), bf(1000 * rng.standard_normal((2, 1, D)))
        pool = q8.ref_append_q8(pool, a, [32, 33, 34, 35, -1], is_v)
        before = q8.read_pool(pool, is_v)
        assert np.all(np.abs(before[1, :4, 0] - a[:4, 0]) <= 2.0 ** -4 * np.abs(a[:4, 0]) + 2.0 ** -14)
        pool = q8.ref_append_q8(pool, b, [36, 37], is_v)
        after = q8.read_pool(pool, is_v)
        e = q8.tail_of(q8.block_of(pool, 32, 0))[0]
        assert e == q8.exponent_for(np.abs(b).max())
        # rounded again: exact down to the new scale's normal range
        assert np.all(np.abs(after[1, :4, 0] - before[1, :4, 0]) <= 2.0 ** (e - 10))
        big = np.abs(before[1, :4, 0]) >= 2.0 ** (e - 6)
        assert np.array_equal(after[1, :4, 0][big], before[1, :4, 0][big])
        assert np.array_equal(bf(after), after)  # every value is a bf16 number
        # begun anew: the exponent falls again
        pool = q8.ref_append_q8(pool, a[:1], [32], is_v)
        assert q8.tail_of(q8.block_of(pool, 32, 0))[0] == q8.exponent_for(np.abs(a[0]).max())


def test_nan_rows_and_infinities():
    pool = np.zeros((1, 1, 16, 65), dtype=np.uint8)
    rows = np.ones((3, 1, 64))
    rows[0, 0, 5] = np.nan
    rows[1, 0, 6] = -np.inf
    pool = q8.ref_append_q8(pool, rows, [0, 1, 2], False)
    v = q8.read_pool(pool, False)[0, :, 0]
    assert np.isnan(v[0]).all() and v[1, 6] == -448 * 2.0 ** 55 and v[1, 5] == 0 and not np.isnan(v[1:]).any()
    pool = q8.ref_append_q8(pool, np.ones((1, 1, 64)), [0], False)  # begun anew
    assert (q8.read_pool(pool, False)[0, 0, 0] == 1).all()


def test_planted_mistakes_are_seen(monkeypatch):
    rows = torch.from_numpy(np.random.default_rng(2).standard_normal((1, 1, 128))).to(BF16).double().numpy()
    pool = np.zeros((1, 1, 16, 129), dtype=np.uint8)
    good = q8.ref_append_q8(pool, rows, [3], False)
    with monkeypatch.context() as m:
        m.setattr(q8, "places", lambda D, is_v: np.arange(16 * D).reshape(16, D))
        assert not np.array_equal(good, q8.ref_append_q8(pool, rows, [3], False))
    with monkeypatch.context() as m:
        m.setattr(q8, "exponent_for", lambda a: 1 + int(np.ceil(np.log2(a / 448))))
        assert not np.array_equal(good, q8.ref_append_q8(pool, rows, [3], False))


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("name", ["kv_append", "kv_read", "decode", "prefill"])
def test_calls_and_packed_calls_check_every_argument(lib, name):
    spec = plain_args()[f"inkling_rel_attn_{name}_q4"]
    call, pack, count = lib.PACKED[f"inkling_rel_attn_{name}_q8"]
    assert count == len(spec)
    good = [s[1] for s in spec]
    for i, (arg, value, bad, code) in enumerate(spec):
        if bad is None:
            continue
        args = good[:i] + [bad] + good[i + 1:]
        assert getattr(lib, f"inkling_rel_attn_{name}_q8")(*args) == code, arg
        assert lib.inkling_rel_attn_packed(call, pack(*args), count) == code, arg
        if isinstance(value, int) and arg in ("T", "B", "H_kv", "D", "R", "stride", "page_size", "num_pages"):
            wide = good[:i] + [value + (1 << 32)] + good[i + 1:]
            assert lib.inkling_rel_attn_packed(call, pack(*wide), count) == -1, arg
    assert lib.inkling_rel_attn_packed(call, pack(*good), count - 1) == -1


def test_ranges(lib):
    a = dict(q=16, k_cache=16, v_cache=16, page_table=4, page_table_stride=4, seq_lens=4, rel_logits=4, B=2, q_len=1,
             H_q=4, H_kv=2, D=64, page_size=16, num_pages=16, R=32, window=32, scale=0.125, out=16, lse_out=None,
             workspace=None, workspace_bytes=0, device_error=None, stream=None)
    f = lambda **o: lib.inkling_rel_attn_decode_q8(**{**a, **o})  # noqa: E731
    assert f(scale=2.0 ** 55) == -1 and f(scale=-2.0 ** 55) == -1 and f(q_len=65) == -1 and f(H_q=34) == -1
    assert f(B=0) == 0
    assert lib.inkling_rel_attn_kv_append_q8(16, 16, 8, 2, 65536, 64, 16, 8, 16, 16, None, None) == -1
    assert (lib.inkling_rel_attn_decode_q8_workspace_size(3, 2, 6, 2, 128, 152)
            == lib.inkling_rel_attn_decode_q4_workspace_size(3, 2, 6, 2, 128, 152) > 0)
    assert (lib.inkling_rel_attn_prefill_q8_workspace_size(3, 100, 2, 64, 0, 1000)
            == lib.inkling_rel_attn_prefill_q4_workspace_size(3, 100, 2, 64, 0, 1000) > 0)


def test_wrappers_refuse_wrong_tensors():
    import paged_attention_relative_attn_gb300 as ira
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rows = torch.zeros((4, 2, 64), dtype=BF16)
    pool = torch.zeros((3, 2, 16, 65), dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="slot_map"):
        ira.kv_append_q8(rows, rows, slots.int(), pool, pool)
    with pytest.raises(TypeError, match="v_new"):
        ira.kv_append_q8(rows, rows.float(), slots, pool, pool)
    with pytest.raises(TypeError, match=r"D \+ 1"):
        ira.kv_append_q8(rows, rows, slots, pool.view(torch.float8_e4m3fn), pool)
    with pytest.raises(ValueError, match="contiguous|CUDA"):
        ira.kv_append_q8(rows.transpose(0, 1), rows, slots, pool, pool)
    with pytest.raises(ValueError, match="dims"):
        ira.kv_read_q8(slots.view(2, 2), pool, pool)
    four = torch.zeros((3, 2, 16, 36), dtype=torch.uint8)
    with pytest.raises(ValueError, match=r"rows of 36 bytes; 65 \(D = 64\) or 129 \(D = 128\)"):
        ira.kv_read_q8(slots, four, four)  # a 4-bit pool
    with pytest.raises(ValueError, match="shapes differ"):
        ira.kv_read_q8(slots, pool, pool[:2])
    with pytest.raises(ValueError, match="inconsistent"):
        ira.kv_append_q8(rows, rows, slots[:3], pool, pool)
    rel = torch.zeros((2, 4, 8))
    q = torch.zeros((2, 4, 64), dtype=BF16)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.decode_q8(q, pool, pool, i32(2, 4), i32(2), rel[:, :3].contiguous(), window=0, scale=0.1)
    with pytest.raises(ValueError, match="seq_lens"):
        ira.decode_q8(q, pool, pool, i32(2, 4), i32(2, 1), rel, window=0, scale=0.1)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.prefill_q8(q, i32(2), pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1, max_seq_len=8, max_q_len=1)
    # the right types and shapes, but on the CPU
    for call in (lambda: ira.kv_append_q8(rows, rows, slots, pool, pool), lambda: ira.kv_read_q8(slots, pool, pool),
                 lambda: ira.decode_q8(q, pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1),
                 lambda: ira.prefill_q8(q, i32(3), pool, pool, i32(2, 4), i32(2), rel, window=0, scale=0.1,
                                        max_seq_len=8, max_q_len=1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
