"""The 8-bit cache on the GPU: append and read-back bit for bit against the oracle, decode and prefill against
float64 attention over the values the cache stands for, at the shapes and contents where they can go wrong."""

from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

import oracle.q8 as q8
import workloads as W
from tests.helpers import bits, f64
from tests.q8_cases import BF16 as P_BF16
from tests.q8_cases import check, largest, make, random_pool, reference, score_error

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


# ------------------------------------------------------------------ append and read

def special_rows(T, H, D, seed):
    """Rows at the format's borders: e4m3 ties, magnitudes on and past 448 * 2^e, zeros, tiny, huge, infinite, NaN, a
    single outlier, values under e4m3's normal range."""
    g = torch.Generator().manual_seed(seed)
    r = torch.randn((T, H, D), generator=g)
    s = 2.0 ** torch.randint(-8, 8, (T, H, 1), generator=g)
    r[..., :16] = (torch.randint(-256, 257, (T, H, 16), generator=g) + 0.5) / 16 * s   # many of them ties
    r[..., 16:20] = 448.0 * s
    kind = torch.arange(T) % 11
    r[kind == 1] = 0.0
    r[kind == 2] *= 2.0 ** -64
    r[kind == 3] *= 2.0 ** -50
    r[kind == 4] *= 2.0 ** 58
    r[kind == 5, :, -1] = float("inf")
    r[kind == 6, :, -7] = float("nan")
    r[kind == 7, :, -5] = -2.0e4
    r[kind == 8, :, -32:] = 2.0 ** -133  # bf16 subnormals
    r[kind == 9] *= torch.exp2(-torch.arange(D) / 4)
    return r.to(BF16)


def runs(counts, starts, P, g, extra=2):
    """Slots of runs of tokens, each from a place of its own first page on, in a shuffled pool."""
    need = [(a + n + P - 1) // P for n, a in zip(counts, starts)]
    n_pages = sum(need) + extra
    pages = torch.randperm(n_pages, generator=g)
    out, base = [], 0
    for n, a, m in zip(counts, starts, need):
        at = a + torch.arange(n)
        out.append(pages[base + at // P] * P + at % P)
        base += m
    return torch.cat(out), n_pages


def check_append(ops, k, v, slots, kd, vd, k_want, v_want):
    """One append on pools kd, vd, and on the oracle's; every byte has to be the same."""
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.kv_append_q8(k.to(DEV), v.to(DEV), slots.to(DEV), kd, vd, device_error=err)
    k_want = q8.ref_append_q8(k_want, f64(k), slots.numpy(), False)
    v_want = q8.ref_append_q8(v_want, f64(v), slots.numpy(), True)
    assert np.array_equal(kd.cpu().numpy(), k_want) and np.array_equal(vd.cpu().numpy(), v_want)
    kr, vr = ops.kv_read_q8(slots.to(DEV), kd, vd, device_error=err)
    live = slots.numpy() >= 0
    at = slots.numpy()[live]
    P = kd.shape[2]
    for got, pool, is_v in ((kr, k_want, False), (vr, v_want, True)):
        want = np.zeros(tuple(got.shape))
        want[live] = q8.read_pool(pool, is_v)[at // P, at % P]
        assert np.array_equal(f64(got), want, equal_nan=True)
    assert int(err) == 0
    return k_want, v_want


# counts and first places of runs of tokens, H, D, page size; the last two have enough rows for windows of 16 tokens
APPEND = [
    ([1], [0], 1, 64, 16),
    ([1, 1, 1], [5, 0, 31], 3, 64, 32),
    ([17, 2, 40], [15, 46, 3], 2, 128, 48),
    ([16, 15, 33, 1], [0, 1, 250, 16], 5, 128, 256),
    ([1] * 40, [3 * i % 64 for i in range(40)], 2, 128, 64),
    ([700, 1, 30, 333], [7, 16, 0, 13], 16, 64, 16),
    ([500, 600, 3], [9, 32, 30], 16, 128, 64),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_and_read_bit_exact(ops, case):
    counts, starts, H, D, P = APPEND[case]
    g = torch.Generator().manual_seed(case)
    slots, n = runs(counts, starts, P, g)
    T = slots.numel()
    pools = [random_pool(n, H, P, D, 7 + i, "cpu") for i in range(2)]
    blocks = pools[0].view(-1, 16 * (D + 1))
    blocks[::3, 16 * D:] = 255              # tails that are none: the block counts as not begun
    blocks[1::3, 16 * D + 4] = 0x5a         # some NaN rows
    kd, vd = (x.to(DEV) for x in pools)
    k_want, v_want = (x.numpy() for x in pools)
    keep = slots.clone()
    if T > 4:
        keep[3] = -1                        # skipped
    k_want, v_want = check_append(ops, special_rows(T, H, D, 3), special_rows(T, H, D, 4), keep, kd, vd, k_want, v_want)
    # the same places again, smaller and larger: exponents stay or grow, flags go
    for scale in (2.0 ** -9, 2.0 ** 7, 1.0):
        k, v = (torch.randn((T, H, D), generator=g) * scale for _ in range(2))
        k_want, v_want = check_append(ops, k.to(BF16), v.to(BF16), slots, kd, vd, k_want, v_want)


@pytest.mark.parametrize("D,step", [(64, 1), (128, 1), (128, 3), (64, 7)])
def test_append_token_by_token(ops, D, step):
    """A sequence that grows by ``step`` tokens a call, magnitudes up and down by powers of two, NaN rows among
    them: exponents grow, rows are rounded again, flags are kept."""
    P, H, L = 32, 2, 70
    g = torch.Generator().manual_seed(D + step)
    pages = torch.tensor([2, 0, 3])
    at = torch.arange(L)
    slots = pages[at // P] * P + at % P
    size = 2.0 ** torch.randint(-12, 13, (L, H, 1), generator=g)
    k, v = (torch.randn((L, H, D), generator=g) * size for _ in range(2))
    k[11, 0, 3] = v[40, 1, 5] = float("nan")
    kd = torch.zeros((4, H, P, D + 1), dtype=torch.uint8, device=DEV)
    vd = kd.clone()
    k_want, v_want = kd.cpu().numpy(), vd.cpu().numpy()
    for t in range(0, L, step):
        i = slice(t, t + step)
        k_want, v_want = check_append(ops, k[i].to(BF16), v[i].to(BF16), slots[i], kd, vd, k_want, v_want)


def test_append_many_tokens_of_single_places(ops):
    """Enough rows for windows of 16 tokens, each token in a block of its own."""
    H, D, P, T = 16, 64, 16, 1100
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(T + 3, generator=g)[:T] * 16 + torch.randint(0, 16, (T,), generator=g)
    pools = [random_pool(T + 3, H, P, D, 17 + i, "cpu") for i in range(2)]
    kd, vd = (x.to(DEV) for x in pools)
    k, v = (torch.randn((T, H, D), generator=g).to(BF16) for _ in range(2))
    check_append(ops, k, v, slots, kd, vd, pools[0].numpy(), pools[1].numpy())


def test_slots_out_of_range_are_reported_and_skipped(ops):
    k = torch.randn((3, 2, 64), device=DEV).to(BF16)
    pool = torch.zeros((2, 2, 16, 65), dtype=torch.uint8, device=DEV)
    slots = torch.tensor([32, 1 << 40, 5], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kc, vc = pool.clone(), pool.clone()
    ops.kv_append_q8(k, k, slots, kc, vc, device_error=err)
    assert int(err) == 1
    assert not kc[1].any() and kc[0].any()
    err.zero_()
    kr, vr = ops.kv_read_q8(slots, kc, vc, device_error=err)
    assert int(err) == 1 and not kr[:2].any() and not vr[:2].any() and vr[2].any()


def test_append_no_tokens(ops):
    pool = torch.zeros((2, 2, 16, 65), dtype=torch.uint8, device=DEV)
    e = torch.empty((0, 2, 64), dtype=BF16, device=DEV)
    s = torch.empty(0, dtype=torch.int64, device=DEV)
    ops.kv_append_q8(e, e, s, pool, pool)
    kr, _ = ops.kv_read_q8(s, pool, pool)
    assert kr.shape == (0, 2, 64)


def test_offsets_past_32_bits(ops):
    """Pools of more than 2^32 bytes: append, read, decode and prefill at their end."""
    H, P, D = 8, 64, 128
    n = (1 << 32) // (H * P * 129) + 40
    kc = torch.empty((n, H, P, 129), dtype=torch.uint8, device=DEV)
    vc = torch.empty((n, H, P, 129), dtype=torch.uint8, device=DEV)
    L = 150
    pages = torch.tensor([n - 1, n - 3, n - 2])
    k = torch.randn((L, H, D), device=DEV).to(BF16)
    v = torch.randn((L, H, D), device=DEV).to(BF16)
    at = torch.arange(L)
    slots = (pages[at // P] * P + at % P).to(DEV)
    ops.kv_append_q8(k, v, slots, kc, vc)
    kr, vr = ops.kv_read_q8(slots, kc, vc)
    ks = torch.zeros((3, H, P, 129), dtype=torch.uint8, device=DEV)
    vs = ks.clone()
    s2 = (at // P * P + at % P).to(DEV)
    ops.kv_append_q8(k, v, s2, ks, vs)
    k2, v2 = ops.kv_read_q8(s2, ks, vs)
    assert np.array_equal(bits(kr), bits(k2)) and np.array_equal(bits(vr), bits(v2))
    inp = make([1], [L], 16, H, D, P, 0, 64, 3)
    far, near = pages.to(torch.int32).view(1, 3).to(DEV), torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3)
    kw = dict(window=0, scale=inp.scale)
    a, la = ops.decode_q8(inp.q, kc, vc, far, inp.seq_lens, inp.rel_logits, **kw)
    b, lb = ops.decode_q8(inp.q, ks, vs, near, inp.seq_lens, inp.rel_logits, **kw)
    assert np.array_equal(bits(a), bits(b)) and torch.equal(la, lb)
    kw.update(max_seq_len=L, max_q_len=1)
    a, _ = ops.prefill_q8(inp.q, inp.cu_seqlens_q, kc, vc, far, inp.seq_lens, inp.rel_logits, **kw)
    b, _ = ops.prefill_q8(inp.q, inp.cu_seqlens_q, ks, vs, near, inp.seq_lens, inp.rel_logits, **kw)
    assert np.array_equal(bits(a), bits(b))


# ------------------------------------------------------------------ decode

def run_decode(ops, inp, q_len, **kw):
    return ops.decode_q8(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits, q_len=q_len,
                         window=inp.window, scale=inp.scale, **kw)


DECODE = [
    # q_len, kv_lens, H_q, H_kv, D, P, window, R
    (1, [1], 1, 1, 64, 16, 0, 1),
    (1, [37, 100], 4, 2, 64, 16, 32, 32),
    (1, [16, 17, 15, 1, 0, 33], 6, 2, 128, 16, 0, 8),
    (1, [600, 64, 513, 511, 512], 6, 2, 128, 64, 512, 512),
    (1, [1000, 3, 0, 257], 16, 1, 128, 48, 0, 100),
    (1, [300, 41], 5, 5, 128, 256, 1, 7),
    (1, [5000, 20], 12, 2, 128, 64, 0, 1024),
    (1, [3000] * 3, 16, 2, 64, 32, 777, 64),
    (2, [2, 1, 0, 50, 300], 6, 2, 128, 16, 0, 16),
    (4, [600, 64, 515, 4, 3], 6, 2, 128, 64, 512, 512),
    (5, [300, 77], 3, 1, 64, 16, 20, 40),
    (7, [900, 133], 16, 1, 128, 64, 0, 32),
    (64, [64, 700], 4, 4, 64, 32, 100, 128),
    (3, [2100, 5], 9, 1, 128, 64, 0, 3000),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
@pytest.mark.parametrize("q_std", [1.0, 8.0])
def test_decode(ops, case, q_std):
    ql, kl, H_q, H_kv, D, P, win, R = DECODE[case]
    inp = make([ql] * len(kl), kl, H_q, H_kv, D, P, win, R, seed=50 + case, q_std=q_std)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(inp.q, float("nan"))
    out, lse = run_decode(ops, inp, ql, out=out, device_error=err)
    check(inp, out, lse, what=f"case {case}")
    assert int(err) == (8 if ql > 1 and min(kl) < ql else 0)


def test_decode_many_sequences(ops):
    """More sequences than blocks on the GPU, every length from 0 on, in a shuffled order."""
    kl = [int(x) for x in np.random.default_rng(1).permutation(700)]
    inp = make([1] * 700, kl, 2, 1, 64, 16, 0, 16, seed=80)
    check(inp, *run_decode(ops, inp, 1))


def test_decode_long_sequence_beside_short_ones(ops):
    inp = make([1] * 5, [3, 40000, 0, 129, 17], 3, 1, 64, 64, 0, 256, seed=81)
    check(inp, *run_decode(ops, inp, 1))


def test_decode_negative_scale(ops):
    inp = dataclasses.replace(make([2], [300], 6, 2, 128, 64, 0, 64, seed=79), scale=-0.1)
    check(inp, *run_decode(ops, inp, 2))


@pytest.mark.parametrize("spread,exp", [(15, 0), (0, 20), (19, 55), (10, -50)])
def test_decode_scales_of_every_size(ops, spread, exp):
    """Blocks whose scales differ by up to 2^19, large and small ones: the V base moves, q and the bias stay."""
    inp = make([2, 2], [700, 90], 6, 2, 128, 64, 0, 64, seed=78, spread=spread, exp=exp)
    inp = dataclasses.replace(inp, scale=inp.scale * 2.0 ** -(exp + 7))
    check(inp, *run_decode(ops, inp, 2), what=f"{spread} {exp}")


@pytest.mark.parametrize("power", [-100, -58, 40, 60])
def test_decode_q_of_every_size(ops, power):
    inp = make([1, 1], [300, 41], 6, 2, 64, 16, 0, 64, seed=77)
    q = (inp.q.float() * 2.0 ** power).to(BF16)
    inp = dataclasses.replace(inp, q=q, scale=inp.scale * 2.0 ** -max(power, -50))
    check(inp, *run_decode(ops, inp, 1), what=str(power))


@pytest.mark.parametrize("slope", [-0.3, -0.01, 0.3])
def test_decode_rising_and_falling_scores(ops, slope):
    """The bias carries the row maximum up or down along the keys by many powers of two."""
    inp = make([2, 2], [900, 130], 6, 2, 128, 64, 0, 1024, seed=82)
    rel = (slope * torch.arange(1024, device=DEV, dtype=torch.float32)).expand_as(inp.rel_logits).contiguous()
    inp = dataclasses.replace(inp, rel_logits=rel)
    check(inp, *run_decode(ops, inp, 2), what=f"slope {slope}")


def test_decode_one_hot_bias_reads_the_value(ops):
    """-1e4 at every distance but one: the output is that key's row, off by P's and the result's rounding only."""
    inp = make([1, 1], [200, 77], 4, 2, 128, 16, 0, 256, seed=83)
    vals = q8.read_pool(inp.v_cache.cpu().numpy(), True)
    pt = inp.page_table.cpu()
    for d in (0, 1, 15, 16, 63, 76):
        rel = torch.full_like(inp.rel_logits, -1e4)
        rel[:, :, d] = 0.0
        out, _ = run_decode(ops, dataclasses.replace(inp, rel_logits=rel), 1)
        for b, L in enumerate((200, 77)):
            j = L - 1 - d
            want = vals[int(pt[b, j // 16]), j % 16].repeat(2, axis=0)
            assert np.all(np.abs(f64(out[b]) - want) <= (P_BF16 + 2.0 ** -11) * 1.01 * np.abs(want))


def test_decode_infinite_bias(ops):
    """-inf at some distances hides those keys; at all of them the row is empty; the lowest number does neither."""
    inp = make([1, 1, 1], [100, 300, 40], 2, 1, 64, 16, 0, 64, seed=84)
    rel = inp.rel_logits.clone()
    rel[0, :, ::2] = -float("inf")
    rel[1] = -float("inf")
    rel[2] = torch.finfo(torch.float32).min
    out, lse = run_decode(ops, dataclasses.replace(inp, rel_logits=rel), 1)
    assert not out[1].any() and bool((lse[1] == -float("inf")).all())
    # row 0: the same as hiding those keys by a bias of -1e30
    r2 = rel.clone()
    r2[0, :, ::2] = -1e30
    r2[1] = 0.0
    r2[2] = 0.0
    ro, rl, size = reference(dataclasses.replace(inp, rel_logits=r2))
    tol = P_BF16 * np.abs(ro) + (2.0 ** -11 * 1.01 + 2 * score_error(inp) + 1e-5) * size
    assert np.all(np.abs(f64(out[0]) - ro[0]) <= tol[0])
    # row 2: every score is the same number (the products are far below its last bit): the mean of V, whose blocks
    # have scales that differ
    vals = q8.read_pool(inp.v_cache.cpu().numpy(), True)
    pt = inp.page_table.cpu()
    vv = np.stack([vals[int(pt[2, j // 16]), j % 16] for j in range(40)])
    want = vv.mean(0).repeat(2, axis=0)
    assert np.all(np.abs(f64(out[2]) - want) <= P_BF16 * np.abs(want) + 2.0 ** -11 * 1.01 * np.abs(vv).mean(0))


def test_decode_nan_reaches_its_rows_only(ops):
    inp = make([1, 1], [100, 300], 4, 2, 64, 16, 0, 64, seed=85)
    clean, lclean = run_decode(ops, inp, 1)
    rel = inp.rel_logits.clone()
    rel[0, 1, 5] = float("nan")
    q = inp.q.clone()
    q[1, 3, 7] = float("nan")
    out, lse = run_decode(ops, dataclasses.replace(inp, rel_logits=rel, q=q), 1)
    keep = torch.ones((2, 4), dtype=torch.bool, device=DEV)
    for r in ((0, 1), (1, 3)):
        assert bool(torch.isnan(out[r].float()).all()) and bool(torch.isnan(lse[r]))
        keep[r] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], lclean[keep])


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("D,P,window", [(64, 16, 0), (128, 64, 40)])
def test_decode_nan_rows_of_the_cache(ops, side, D, P, window):
    """A cached row with a NaN: NaN for the tokens and heads that see it, the same bits as without it for the
    others (4 tokens: some see it, some do not)."""
    H = 2
    inp = make([4, 4], [150, 90], 6, H, D, P, window, 64, seed=76)
    clean, lclean = run_decode(ops, inp, 4)
    # key 147 of sequence 0 (seen by its tokens at 147, 148, 149), KV head 1; and the key that leaves the window
    # first of sequence 1 (or key 3)
    for b, j, who in ((0, 147, {1, 2, 3}), (1, 88, {2, 3}), (1, 86 - window + 1 if window else 3, {0} if window else {0, 1, 2, 3})):
        pool = (inp.k_cache if side == "k" else inp.v_cache).clone()
        slot = int(inp.page_table[b, j // P]) * P + j % P
        block = pool.view(pool.shape[0], H, P // 16, -1)[slot // P, 1, slot % P // 16]
        block[16 * D + 4 + (slot % 16) // 8] |= 1 << slot % 8
        out, lse = run_decode(ops, dataclasses.replace(inp, **{side + "_cache": pool}), 4)
        hit = torch.zeros((8, 6), dtype=torch.bool, device=DEV)
        for i in who:
            hit[4 * b + i, 3:] = True
        assert bool(torch.isnan(out[hit].float()).all())
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit])
        assert bool(torch.isnan(lse[hit]).all()) if side == "k" else torch.equal(lse, lclean)


def test_decode_bad_pages_read_as_zeros(ops):
    inp = make([1, 1], [100, 300], 4, 2, 64, 16, 0, 64, seed=86)
    pt = inp.page_table.clone()
    pt[1, 2], pt[1, 7] = -5, 1 << 30
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run_decode(ops, dataclasses.replace(inp, page_table=pt), 1, device_error=err)
    assert int(err) == 1
    # the same with the two pages' rows standing for zeros
    k, v = inp.k_cache.clone(), inp.v_cache.clone()
    for lp in (2, 7):
        for pool in (k, v):
            pool.view(pool.shape[0], 2, 16 * 65)[int(inp.page_table[1, lp]), :, :16 * 64] = 0
    want, wl = run_decode(ops, dataclasses.replace(inp, k_cache=k, v_cache=v), 1)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    pre, _ = ops.prefill_q8(inp.q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, pt, inp.seq_lens, inp.rel_logits,
                            window=0, scale=inp.scale, max_seq_len=300, max_q_len=1, device_error=err)
    wp, _ = ops.prefill_q8(inp.q, inp.cu_seqlens_q, k, v, inp.page_table, inp.seq_lens, inp.rel_logits, window=0,
                           scale=inp.scale, max_seq_len=300, max_q_len=1)
    assert torch.equal(pre, wp)


def test_decode_longer_than_its_table(ops):
    inp = make([1], [64], 4, 2, 64, 16, 0, 64, seed=87)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, _ = run_decode(ops, dataclasses.replace(inp, seq_lens=inp.seq_lens + 1000), 1, device_error=err)
    b, _ = run_decode(ops, inp, 1)
    assert int(err) == 2 and torch.equal(a, b)


def test_decode_pages_before_the_window_may_be_gone(ops):
    """Ids of pages wholly before the window are not looked at, in decode and prefill."""
    inp = make([2], [500], 4, 2, 128, 16, 64, 64, seed=75)
    want, _ = run_decode(ops, inp, 2)
    pt = inp.page_table.clone()
    pt[:, :(500 - 2 - 64 + 1) // 16] = -7
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gone = dataclasses.replace(inp, page_table=pt)
    out, _ = run_decode(ops, gone, 2, device_error=err)
    run_prefill(ops, gone, device_error=err)
    assert int(err) == 0 and torch.equal(out, want)


def test_decode_page_permutation_bit_exact(ops):
    inp = make([2, 2], [1000, 129], 6, 2, 128, 64, 0, 512, seed=88)
    out0, lse0 = run_decode(ops, inp, 2)
    n = inp.k_cache.shape[0]
    for s in range(2):
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(s)).to(DEV)
        kc, vc = torch.empty_like(inp.k_cache), torch.empty_like(inp.v_cache)
        kc[perm], vc[perm] = inp.k_cache, inp.v_cache
        i2 = dataclasses.replace(inp, k_cache=kc, v_cache=vc, page_table=perm[inp.page_table.long()].to(torch.int32))
        out1, lse1 = run_decode(ops, i2, 2)
        assert torch.equal(out0, out1) and torch.equal(lse0, lse1)


def test_decode_repeats_bit_exact_and_lse_is_optional(ops):
    inp = make([1] * 40, [int(x) for x in np.random.default_rng(3).integers(1, 4000, 40)], 6, 1, 128, 64, 0, 64,
               seed=89)
    first, lse = run_decode(ops, inp, 1)
    for _ in range(5):
        again, l2 = run_decode(ops, inp, 1)
        assert torch.equal(first, again) and torch.equal(lse, l2)
    from paged_attention_relative_attn_gb300 import _lib
    need = ops.decode_q8_workspace_bytes(40, 1, 6, 1, 128)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(first)
    args = dict(q=inp.q.data_ptr(), k_cache=inp.k_cache.data_ptr(), v_cache=inp.v_cache.data_ptr(),
                page_table=inp.page_table.data_ptr(), page_table_stride=inp.page_table.shape[1],
                seq_lens=inp.seq_lens.data_ptr(), rel_logits=inp.rel_logits.data_ptr(), B=40, q_len=1, H_q=6, H_kv=1,
                D=128, page_size=64, num_pages=inp.num_pages, R=64, window=0, scale=inp.scale, out=out.data_ptr(),
                lse_out=None, workspace=ws.data_ptr(), workspace_bytes=need, device_error=None,
                stream=torch.cuda.current_stream().cuda_stream)
    assert _lib.inkling_rel_attn_decode_q8(**args) == 0
    assert torch.equal(first, out)
    if need:
        assert _lib.inkling_rel_attn_decode_q8(**{**args, "workspace_bytes": need - 1}) == -3


def test_decode_on_two_streams(ops):
    """Calls in flight on two streams, a workspace each; inputs used on another stream than their own."""
    a = make([1] * 20, [2000] * 20, 6, 2, 128, 64, 0, 64, seed=90)
    b = make([1] * 20, [1500] * 20, 6, 2, 128, 64, 700, 64, seed=91)
    wa, wb = run_decode(ops, a, 1), run_decode(ops, b, 1)
    need = max(1, ops.decode_q8_workspace_bytes(20, 1, 6, 2, 128))
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [(torch.empty_like(x.q), torch.empty(x.q.shape[:2], device=DEV)) for x in (a, b)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, x in enumerate((a, b)):
            run_decode(ops, x, 1, out=outs[i][0], lse=outs[i][1], workspace=ws[i], stream=s[i])
    torch.cuda.synchronize()
    for got, want in zip(outs, (wa, wb)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_captured_with_changing_lengths(ops):
    """Two captured graphs share a workspace; lengths change between replays."""
    inp = make([1] * 6, [2500, 10, 0, 700, 64, 1999], 6, 2, 128, 64, 0, 256, seed=92, poison=False)
    need = max(1, ops.decode_q8_workspace_bytes(6, 1, 6, 2, 128))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    sl = inp.seq_lens.clone()
    cap = dataclasses.replace(inp, seq_lens=sl)
    outs, graphs = [], []
    for win in (0, 300):
        o, l = torch.empty_like(inp.q), torch.empty(inp.q.shape[:2], device=DEV)
        c = dataclasses.replace(cap, window=win)
        run_decode(ops, c, 1, out=o, lse=l, workspace=ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run_decode(ops, c, 1, out=o, lse=l, workspace=ws)
        outs.append((o, l))
        graphs.append(gr)
    for lens in ([2500, 10, 0, 700, 64, 1999], [1, 10, 0, 0, 33, 512], [2500, 10, 0, 700, 64, 1]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        for o, l in outs:
            o.fill_(float("nan"))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for win, (o, l) in zip((0, 300), outs):
            e, el = run_decode(ops, dataclasses.replace(cap, window=win), 1)
            assert torch.equal(o, e) and torch.equal(l, el), (win, lens)


# ------------------------------------------------------------------ prefill

def run_prefill(ops, inp, **kw):
    return ops.prefill_q8(inp.q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens,
                          inp.rel_logits, window=inp.window, scale=inp.scale, max_seq_len=inp.max_seq_len,
                          max_q_len=inp.max_q_len, **kw)


PREFILL = [
    # q_lens, kv_lens, H_q, H_kv, D, P, window, R
    ([1], [1], 2, 1, 64, 16, 0, 4),
    ([5, 0, 3], [5, 9, 40], 4, 2, 128, 64, 0, 16),
    ([130, 129], [130, 500], 6, 2, 128, 64, 64, 64),
    ([200], [1000], 3, 1, 128, 48, 512, 512),
    ([150, 33], [900, 33], 4, 4, 64, 16, 100, 128),
    ([77], [1500], 4, 1, 128, 32, 0, 1024),
    ([64, 1], [640, 700], 2, 2, 64, 256, 1, 4),
    ([100], [1100], 2, 1, 64, 64, 65, 60),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
@pytest.mark.parametrize("q_std", [1.0, 4.0])
def test_prefill(ops, case, q_std):
    ql, kl, H_q, H_kv, D, P, win, R = PREFILL[case]
    inp = make(ql, kl, H_q, H_kv, D, P, win, R, seed=150 + case, q_std=q_std)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    need = ops.prefill_q8_workspace_bytes(len(kl), max(ql), H_kv, D, win, max(kl))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN in every bf16 of it
    out, lse = run_prefill(ops, inp, workspace=ws, device_error=err)
    check(inp, out, lse, what=f"case {case}", p_step=P_BF16)
    assert int(err) == 0


def test_prefill_rows_behind_the_last_sequence_are_left(ops):
    inp = make([30], [100], 4, 2, 128, 64, 0, 16, seed=172)
    q = torch.cat([inp.q, inp.q[:7]])
    rel = torch.cat([inp.rel_logits, inp.rel_logits[:7]])
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    run_prefill(ops, dataclasses.replace(inp, q=q, rel_logits=rel), out=out, lse=lse)
    assert bool((out[30:] == 7.0).all()) and bool((lse[30:] == 7.0).all())
    check(inp, out[:30], lse[:30], p_step=P_BF16)


def test_prefill_refuses_chunks_that_do_not_fit(ops):
    """A chunk longer than its sequence, and a sequence past max_seq_len: reported, rows left as they were."""
    inp = make([10, 10, 10], [20, 200, 30], 4, 2, 128, 64, 0, 16, seed=171, poison=False)
    good, _ = run_prefill(ops, inp)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(inp.q, 7.0)
    bad = dataclasses.replace(inp, seq_lens=torch.tensor([5, 200, 30], dtype=torch.int32, device=DEV), max_seq_len=64)
    run_prefill(ops, bad, out=out, device_error=err)
    assert int(err) == 8 | 2
    assert bool((out[:20] == 7.0).all()) and torch.equal(out[20:], good[20:])


def test_decode_and_prefill_agree(ops):
    inp = make([3, 3], [500, 90], 6, 2, 128, 64, 64, 64, seed=173)
    ref = reference(inp)
    check(inp, *run_decode(ops, inp, 3), ref)
    check(inp, *run_prefill(ops, inp), ref, p_step=P_BF16)


# ------------------------------------------------------------------ together

def test_serving_run(ops):
    """Prompts in two chunks, then decode steps, a draft verification of which some are rejected, requests ending
    and starting: the tables, the append, prefill and decode as a server uses them, each checked in float64."""
    B, H_q, H_kv, D, P, stride, window, R = 4, 4, 2, 64, 16, 20, 40, 48
    g = torch.Generator().manual_seed(5)
    n_pages = 40
    free = torch.randperm(n_pages, generator=g).to(torch.int32).to(DEV)
    count = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    pt = torch.zeros((B, stride), dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    kc = torch.full((n_pages, H_kv, P, 65), 255, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    kw, vw = kc.cpu().numpy(), vc.cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    steps = [[33, 50, 1, 0], [20, 7, 1, 60], [1, 1, 1, 1], [1, 1, 1, 1], [4, 4, 4, 4], [-1, 1, 1, 1], [70, 1, 1, 1],
             [1, -1, 1, 1], [1, 0, 1, 1]]
    for i, new in enumerate(steps):
        if i == 5:
            lens -= torch.tensor([0, 2, 3, 1], dtype=torch.int32, device=DEV)  # drafts that were rejected: the page stays
            assert bool(((lens + 15) // 16 == (lens + 3 + 15) // 16).any())
        nl = torch.tensor(new, dtype=torch.int32, device=DEV)
        _, cu, slots, _ = ops.build_tables(lens, nl, pt, free, count, page_size=P, max_tokens=130, kv_lens=lens,
                                           free_left=count, device_error=err)
        T = sum(max(x, 0) for x in new)
        k = torch.randn((130, H_kv, D), generator=g).to(BF16)
        v = torch.randn((130, H_kv, D), generator=g).to(BF16)
        kw, vw = check_append(ops, k, v, slots.cpu(), kc, vc, kw, vw)
        q = torch.randn((T, H_q, D), generator=g).to(BF16).to(DEV)
        rel = (0.5 * torch.randn((T, H_q, R), generator=g)).to(DEV)
        inp = W.PrefillInputs(q=q, cu_seqlens_q=cu, k_cache=kc, v_cache=vc, page_table=pt, seq_lens=lens,
                              rel_logits=rel, window=window, scale=D ** -0.5, max_seq_len=stride * P,
                              max_q_len=max(new))
        kr, _ = ops.kv_read_q8(slots[:T], kc, vc)
        x = k[:T].to(DEV).float()
        assert bool(((kr.float() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * largest(kc) / 448).all())
        ref = reference(inp)
        if len(set(new)) == 1:
            check(inp, *run_decode(ops, inp, new[0], device_error=err), ref, what=f"step {i}, decode")
        check(inp, *run_prefill(ops, inp, device_error=err), ref, what=f"step {i}, prefill", p_step=P_BF16)
    assert int(err) == 0


def test_captured_decode_loop_allocates_its_own_pages(ops):
    """One captured step -- tables, append, decode -- replayed: lengths, pages and cache move on without the host."""
    B, H_q, H_kv, D, P = 3, 4, 2, 128, 16
    g = torch.Generator().manual_seed(6)

    def state():
        return dict(free=torch.arange(30, dtype=torch.int32, device=DEV), count=torch.tensor([30], dtype=torch.int32, device=DEV),
                    pt=torch.zeros((B, 8), dtype=torch.int32, device=DEV), lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                    kc=torch.zeros((30, H_kv, P, 129), dtype=torch.uint8, device=DEV),
                    vc=torch.zeros((30, H_kv, P, 129), dtype=torch.uint8, device=DEV))

    n = 35
    ks, vs = (torch.randn((n, B, H_kv, D), generator=g).to(BF16).to(DEV) for _ in range(2))
    qs = torch.randn((n, B, H_q, D), generator=g).to(BF16).to(DEV)
    rel = torch.randn((B, H_q, 32), generator=g).to(DEV)
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, ops.decode_q8_workspace_bytes(B, 1, H_q, H_kv, D)), dtype=torch.uint8, device=DEV)
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    cu = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((B, H_q), device=DEV)

    def step(s):
        ops.build_tables(s["lens"], new, s["pt"], s["free"], s["count"], page_size=P, kv_lens=s["lens"],
                         cu_seqlens_q=cu, slot_map=slots, free_left=s["count"])
        ops.kv_append_q8(k, v, slots, s["kc"], s["vc"])
        ops.decode_q8(q, s["kc"], s["vc"], s["pt"], s["lens"], rel, window=20, scale=0.1, out=out, lse=lse, workspace=ws)

    step(state())  # warm up
    a, b = state(), state()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(a)
    for i in range(n):
        k.copy_(ks[i])
        v.copy_(vs[i])
        q.copy_(qs[i])
        gr.replay()
        got = out.clone(), lse.clone()
        step(b)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i
    for x in ("free", "count", "pt", "lens", "kc", "vc"):
        assert torch.equal(a[x], b[x]), x
    assert a["lens"].tolist() == [n] * B and int(a["count"]) == 30 - 3 * B


def test_stream_of_another_device(ops):
    from types import SimpleNamespace
    # stands for a stream of a second GPU: nothing may be launched on it or on another in its stead
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0, device_index=1, stream_id=0, device_type=1)
    inp = make([1, 1], [30, 40], 4, 2, 64, 16, 0, 8, seed=1)
    rows, slots = torch.zeros((4, 2, 64), dtype=BF16, device=DEV), torch.arange(4, device=DEV)
    pool = inp.k_cache.clone()
    out = torch.full_like(inp.q, 7.0)
    for call in (lambda: run_decode(ops, inp, 1, out=out, stream=other), lambda: run_prefill(ops, inp, out=out, stream=other),
                 lambda: ops.kv_append_q8(rows + 1, rows + 1, slots, pool, pool, stream=other),
                 lambda: ops.kv_read_q8(slots, pool, pool, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and torch.equal(pool, inp.k_cache)
