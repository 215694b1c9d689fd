"""The 4-bit cache on the GPU: append and read-back bit for bit against the oracle, decode and prefill against
float64 attention over the values the cache stands for, at the shapes and contents where they can go wrong."""

from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

import oracle.q4 as q4
from tests.helpers import bits, f64
from tests.q4_cases import check, make, reference, score_error

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
    """N(0, 1) rows with groups that hit the format's borders: exact ties, powers of two times 7, zeros, tiny,
    huge, infinite, NaN, a single outlier."""
    g = torch.Generator().manual_seed(seed)
    r = torch.randn((T, H, D), generator=g)
    s = 2.0 ** torch.randint(-8, 8, (T, H, 1), generator=g)
    ties = (torch.randint(-7, 8, (T, H, 32), generator=g) + 0.5).clamp(-6.5, 6.5) * s
    ties[..., :1] = 7 * s
    r[..., :32] = ties
    kind = torch.arange(T) % 9
    r[kind == 1, :, -32:] = 0.0
    r[kind == 2, :, -32:] *= 2.0 ** -103
    r[kind == 3, :, -32:] *= 2.0 ** -99
    r[kind == 4, :, -32:] *= 2.0 ** 125
    r[kind == 5, :, -1] = float("inf")
    r[kind == 6, :, -7] = float("nan")
    r[kind == 7, :, -5] = -200.0
    r[kind == 8, :, -32:] = 2.0 ** -133  # bf16 subnormals
    return r.to(BF16)


@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (19, 3, 64, 48), (37, 2, 128, 64), (18, 16, 128, 16),
                                     (9, 5, 128, 256)])
def test_append_and_read_bit_exact(ops, T, H, D, P):
    g = torch.Generator().manual_seed(T)
    n = (T + P - 1) // P + 2
    k, v = special_rows(T, H, D, 3), special_rows(T, H, D, 4)
    slots = torch.randperm(n * P, generator=g)[:T]
    if T > 4:
        slots[3] = -1                       # skipped
    kc = torch.randint(0, 256, (n, H, P, 9 * D // 16), dtype=torch.uint8, generator=g)
    vc = torch.randint(0, 256, (n, H, P, 9 * D // 16), dtype=torch.uint8, generator=g)
    want_k = q4.ref_append_q4(kc.numpy(), f64(k), slots.numpy(), False)
    want_v = q4.ref_append_q4(vc.numpy(), f64(v), slots.numpy(), True)
    kd, vd, sd = kc.to(DEV), vc.to(DEV), slots.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.kv_append_q4(k.to(DEV), v.to(DEV), sd, kd, vd, device_error=err)
    assert np.array_equal(kd.cpu().numpy(), want_k)     # every byte: the others are as they were
    assert np.array_equal(vd.cpu().numpy(), want_v)
    kr, vr = ops.kv_read_q4(sd, kd, vd, device_error=err)
    for got, pool, is_v in ((kr, want_k, False), (vr, want_v, True)):
        vals = q4.read_pool(pool, is_v)
        at = slots.numpy()
        live = at >= 0
        want = np.zeros((T, H, D))
        want[live] = vals[at[live] // P, at[live] % P]
        assert np.array_equal(f64(got), want, equal_nan=True)
    assert int(err) == 0


def test_slots_out_of_range_are_reported_and_skipped(ops):
    k = torch.randn((3, 2, 64), device=DEV).to(BF16)
    pool = torch.zeros((2, 2, 16, 36), dtype=torch.uint8, device=DEV)
    slots = torch.tensor([32, 1 << 40, 5], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kc, vc = pool.clone(), pool.clone()
    ops.kv_append_q4(k, k, slots, kc, vc, device_error=err)
    assert int(err) == 1
    blocks = kc.view(2, 2, 576)
    assert not blocks[1].any() and blocks[0, :, 5 * 32:6 * 32].any()
    err.zero_()
    kr, vr = ops.kv_read_q4(slots, kc, vc, device_error=err)
    assert int(err) == 1 and not kr[:2].any() and not vr[:2].any() and vr[2].any()


def test_append_no_tokens(ops):
    pool = torch.zeros((2, 2, 16, 36), dtype=torch.uint8, device=DEV)
    e = torch.empty((0, 2, 64), dtype=BF16, device=DEV)
    s = torch.empty(0, dtype=torch.int64, device=DEV)
    ops.kv_append_q4(e, e, s, pool, pool)
    kr, _ = ops.kv_read_q4(s, pool, pool)
    assert kr.shape == (0, 2, 64)


def test_offsets_past_32_bits(ops):
    """Pools of more than 2^32 bytes: append, read and decode at their end."""
    H, P, D = 8, 64, 128
    n = (1 << 32) // (H * P * 72) + 40
    kc = torch.empty((n, H, P, 72), dtype=torch.uint8, device=DEV)
    vc = torch.empty((n, H, P, 72), dtype=torch.uint8, device=DEV)
    L = 150
    pages = torch.tensor([n - 1, n - 3, n - 2])
    k = torch.randn((L, H, D), device=DEV).to(BF16)
    v = torch.randn((L, H, D), device=DEV).to(BF16)
    at = torch.arange(L)
    slots = (pages[at // P] * P + at % P).to(DEV)
    ops.kv_append_q4(k, v, slots, kc, vc)
    kr, vr = ops.kv_read_q4(slots, kc, vc)
    small = torch.zeros((3, H, P, 72), dtype=torch.uint8, device=DEV)
    ks, vs = small.clone(), small.clone()
    s2 = (at // P * P + at % P).to(DEV)
    ops.kv_append_q4(k, v, s2, ks, vs)
    k2, v2 = ops.kv_read_q4(s2, ks, vs)
    assert np.array_equal(bits(kr), bits(k2)) and np.array_equal(bits(vr), bits(v2))
    inp = make([1], [L], 16, H, D, P, 0, 64, 3)
    kw = dict(window=0, scale=inp.scale)
    a, la = ops.decode_q4(inp.q, kc, vc, pages.to(torch.int32).view(1, 3).to(DEV), inp.seq_lens, inp.rel_logits, **kw)
    b, lb = ops.decode_q4(inp.q, ks, vs, torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3), inp.seq_lens,
                          inp.rel_logits, **kw)
    assert np.array_equal(bits(a), bits(b)) and torch.equal(la, lb)


# ------------------------------------------------------------------ decode

def run_decode(ops, inp, q_len, **kw):
    return ops.decode_q4(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits, q_len=q_len,
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
    out, lse = run_decode(ops, inp, 1)
    check(inp, out, lse)


def test_decode_long_sequence_beside_short_ones(ops):
    inp = make([1] * 5, [3, 40000, 0, 129, 17], 3, 1, 64, 64, 0, 256, seed=81)
    out, lse = run_decode(ops, inp, 1)
    check(inp, out, lse)


@pytest.mark.parametrize("slope", [-0.3, -0.01, 0.3])
def test_decode_rising_and_falling_scores(ops, slope):
    """The bias carries the row maximum up or down along the keys by many powers of two."""
    inp = make([2, 2], [900, 130], 6, 2, 128, 64, 0, 1024, seed=82)
    rel = (slope * torch.arange(1024, device=DEV, dtype=torch.float32)).expand_as(inp.rel_logits).contiguous()
    inp = dataclasses.replace(inp, rel_logits=rel)
    out, lse = run_decode(ops, inp, 2)
    check(inp, out, lse, what=f"slope {slope}")


def test_decode_one_hot_bias_reads_the_value(ops):
    """-1e4 at every distance but one: the output is that key's row, off by P's and the result's rounding only."""
    inp = make([1, 1], [200, 77], 4, 2, 128, 16, 0, 256, seed=83)
    vals = q4.read_pool(inp.v_cache.cpu().numpy(), True)
    pt = inp.page_table.cpu()
    for d in (0, 1, 15, 16, 63, 76):
        rel = torch.full_like(inp.rel_logits, -1e4)
        rel[:, :, d] = 0.0
        out, _ = run_decode(ops, dataclasses.replace(inp, rel_logits=rel), 1)
        for b, L in enumerate((200, 77)):
            j = L - 1 - d
            want = vals[int(pt[b, j // 16]), j % 16].repeat(2, axis=0)
            assert np.all(np.abs(f64(out[b]) - want) <= 2.0 ** -7 * 1.01 * np.abs(want))


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
    i2 = dataclasses.replace(inp, rel_logits=r2)
    ro, rl, size = reference(i2)
    tol = 2.0 ** -8 * 1.01 * (np.abs(ro) + size) + 2 * score_error(inp) * size + 1e-5 * size
    assert np.all(np.abs(f64(out[0]) - ro[0]) <= tol[0])
    # row 2: every score is the same number (the products are far below its last bit): the mean of V
    vals = q4.read_pool(inp.v_cache.cpu().numpy(), True)
    pt = inp.page_table.cpu()
    vv = np.stack([vals[int(pt[2, j // 16]), j % 16] for j in range(40)])
    want = vv.mean(0).repeat(2, axis=0)
    assert np.all(np.abs(f64(out[2]) - want) <= 2.0 ** -8 * 1.01 * (np.abs(want) + np.abs(vv).mean(0)))


def test_decode_nan_reaches_its_rows_only(ops):
    inp = make([1, 1], [100, 300], 4, 2, 64, 16, 0, 64, seed=85)
    clean, lclean = run_decode(ops, inp, 1)
    rel = inp.rel_logits.clone()
    rel[0, 1, 5] = float("nan")
    out, lse = run_decode(ops, dataclasses.replace(inp, rel_logits=rel), 1)
    assert bool(torch.isnan(out[0, 1].float()).all()) and bool(torch.isnan(lse[0, 1]))
    keep = torch.ones((2, 4), dtype=torch.bool, device=DEV)
    keep[0, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], lclean[keep])


def test_decode_bad_pages_read_as_zeros(ops):
    inp = make([1, 1], [100, 300], 4, 2, 64, 16, 0, 64, seed=86)
    pt = inp.page_table.clone()
    pt[1, 2], pt[1, 7] = -5, 1 << 30
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run_decode(ops, dataclasses.replace(inp, page_table=pt), 1, device_error=err)
    assert int(err) == 1
    # the same with the two pages' bytes standing for zeros (scale 0)
    k, v = inp.k_cache.clone(), inp.v_cache.clone()
    for lp in (2, 7):
        k[int(inp.page_table[1, lp])] = 0
        v[int(inp.page_table[1, lp])] = 0
    want, wl = run_decode(ops, dataclasses.replace(inp, k_cache=k, v_cache=v), 1)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_decode_longer_than_its_table(ops):
    inp = make([1], [64], 4, 2, 64, 16, 0, 64, seed=87)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, _ = run_decode(ops, dataclasses.replace(inp, seq_lens=inp.seq_lens + 1000), 1, device_error=err)
    b, _ = run_decode(ops, inp, 1)
    assert int(err) == 2 and torch.equal(a, b)


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
    need = ops.decode_q4_workspace_bytes(40, 1, 6, 1, 128)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(first)
    args = dict(q=inp.q.data_ptr(), k_cache=inp.k_cache.data_ptr(), v_cache=inp.v_cache.data_ptr(),
                page_table=inp.page_table.data_ptr(), page_table_stride=inp.page_table.shape[1],
                seq_lens=inp.seq_lens.data_ptr(), rel_logits=inp.rel_logits.data_ptr(), B=40, q_len=1, H_q=6, H_kv=1,
                D=128, page_size=64, num_pages=inp.num_pages, R=64, window=0, scale=inp.scale, out=out.data_ptr(),
                lse_out=None, workspace=ws.data_ptr(), workspace_bytes=need, device_error=None,
                stream=torch.cuda.current_stream().cuda_stream)
    assert _lib.inkling_rel_attn_decode_q4(**args) == 0
    assert torch.equal(first, out)
    if need:
        assert _lib.inkling_rel_attn_decode_q4(**{**args, "workspace_bytes": need - 1}) == -3


def test_decode_on_two_streams(ops):
    """Calls in flight on two streams, a workspace each; inputs used on another stream than their own."""
    a = make([1] * 20, [2000] * 20, 6, 2, 128, 64, 0, 64, seed=90)
    b = make([1] * 20, [1500] * 20, 6, 2, 128, 64, 700, 64, seed=91)
    wa, wb = run_decode(ops, a, 1), run_decode(ops, b, 1)
    need = max(1, ops.decode_q4_workspace_bytes(20, 1, 6, 2, 128))
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
    inp = make([1] * 6, [2500, 10, 0, 700, 64, 1999], 6, 2, 128, 64, 0, 256, seed=92)
    need = max(1, ops.decode_q4_workspace_bytes(6, 1, 6, 2, 128))
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
    return ops.prefill_q4(inp.q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens,
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
    need = ops.prefill_q4_workspace_bytes(len(kl), max(ql), H_kv, D, win, max(kl))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN in every bf16 of it
    out, lse = run_prefill(ops, inp, workspace=ws, device_error=err)
    check(inp, out, lse, what=f"case {case}")
    assert int(err) == 0


def test_prefill_equals_prefill_of_the_values(ops):
    """The same bits as the bf16 cache's prefill over a cache that holds the values."""
    inp = make([200, 40], [900, 300], 6, 2, 128, 64, 128, 64, seed=170)
    out, lse = run_prefill(ops, inp)
    kc = torch.from_numpy(np.nan_to_num(q4.read_pool(inp.k_cache.cpu().numpy(), False))).to(BF16).to(DEV)
    vc = torch.from_numpy(np.nan_to_num(q4.read_pool(inp.v_cache.cpu().numpy(), True))).to(BF16).to(DEV)
    want, wl = ops.prefill(inp.q, inp.cu_seqlens_q, kc, vc, inp.page_table, inp.seq_lens, inp.rel_logits,
                           window=128, scale=inp.scale, max_seq_len=900, max_q_len=200)
    # tiles start at other keys (multiples of 64 of the visible range), so the running sums differ in order only
    ref = reference(inp)
    check(inp, out, lse, ref)
    check(inp, want, wl, ref)


def test_prefill_mask_of_the_lowest_value(ops):
    """fp32's lowest number as a bias hides far keys (whole tiles before the first that counts), and a row that has
    nothing else takes the mean of its values."""
    low = torch.finfo(torch.float32).min
    inp = make([140, 70], [400, 300], 2, 1, 64, 64, 0, 512, seed=174)
    rel = inp.rel_logits.clone()
    rel[:140, :, 10:] = low
    rel[140:] = low
    out, lse = run_prefill(ops, dataclasses.replace(inp, rel_logits=rel))
    r2 = rel.clone()
    r2[:140, :, 10:] = -1e30
    r2[140:] = 0.0
    ro, rl, size = reference(dataclasses.replace(inp, rel_logits=r2), q=f64(inp.q) * (np.arange(210) < 140)[:, None, None])
    e = score_error(inp)
    tol = 2.0 ** -8 * (np.abs(ro) + size) * (1 + 2.0 ** -7) + (2 * e + 2.0 ** -18) * size
    assert np.all(np.abs(f64(out) - ro) <= tol)
    assert np.all(np.abs(f64(lse[:140]) - rl[:140]) <= e[:140, :, 0] + 1e-5)


def test_prefill_refuses_chunks_that_do_not_fit(ops):
    """A chunk longer than its sequence, and a sequence past max_seq_len: reported, rows left as they were."""
    inp = make([10, 10, 10], [20, 200, 30], 4, 2, 128, 64, 0, 16, seed=171)
    good, _ = run_prefill(ops, inp)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(inp.q, 7.0)
    bad = dataclasses.replace(inp, seq_lens=torch.tensor([5, 200, 30], dtype=torch.int32, device=DEV), max_seq_len=64)
    run_prefill(ops, bad, out=out, device_error=err)
    assert int(err) == 8 | 2
    assert bool((out[:20] == 7.0).all()) and torch.equal(out[20:], good[20:])


def test_prefill_rows_behind_the_last_sequence_are_left(ops):
    inp = make([30], [100], 4, 2, 128, 64, 0, 16, seed=172)
    q = torch.cat([inp.q, inp.q[:7]])
    rel = torch.cat([inp.rel_logits, inp.rel_logits[:7]])
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    run_prefill(ops, dataclasses.replace(inp, q=q, rel_logits=rel), out=out, lse=lse)
    assert bool((out[30:] == 7.0).all()) and bool((lse[30:] == 7.0).all())
    check(inp, out[:30], lse[:30])


def test_decode_and_prefill_agree(ops):
    inp = make([3, 3], [500, 90], 6, 2, 128, 64, 64, 64, seed=173)
    ref = reference(inp)
    check(inp, *run_decode(ops, inp, 3), ref)
    check(inp, *run_prefill(ops, inp), ref)


# ------------------------------------------------------------------ together

def test_serving_run(ops):
    """Prompts in two chunks, then decode steps and a draft verification, requests ending and starting: the
    tables, the append, prefill and decode as a server uses them, each attention checked in float64."""
    B, H_q, H_kv, D, P, stride, window, R = 4, 4, 2, 64, 16, 20, 40, 48
    g = torch.Generator().manual_seed(5)
    n_pages = 40
    free = torch.randperm(n_pages, generator=g).to(torch.int32).to(DEV)
    count = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
    pt = torch.zeros((B, stride), dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    kc = torch.full((n_pages, H_kv, P, 36), 255, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    steps = [[33, 50, 1, 0], [20, 7, 1, 60], [1, 1, 1, 1], [1, 1, 1, 1], [4, 4, 4, 4], [-1, 1, 1, 1], [70, 1, 1, 1],
             [1, -1, 1, 1], [1, 0, 1, 1]]
    for i, new in enumerate(steps):
        nl = torch.tensor(new, dtype=torch.int32, device=DEV)
        _, cu, slots, _ = ops.build_tables(lens, nl, pt, free, count, page_size=P, max_tokens=130, kv_lens=lens,
                                           free_left=count, device_error=err)
        T = sum(max(x, 0) for x in new)
        k = torch.randn((130, H_kv, D), generator=g).to(BF16).to(DEV)
        v = torch.randn((130, H_kv, D), generator=g).to(BF16).to(DEV)
        ops.kv_append_q4(k, v, slots, kc, vc, device_error=err)
        q = torch.randn((T, H_q, D), generator=g).to(BF16).to(DEV)
        rel = (0.5 * torch.randn((T, H_q, R), generator=g)).to(DEV)
        import workloads as W
        inp = W.PrefillInputs(q=q, cu_seqlens_q=cu, k_cache=kc, v_cache=vc, page_table=pt, seq_lens=lens,
                              rel_logits=rel, window=window, scale=D ** -0.5, max_seq_len=stride * P,
                              max_q_len=max(new))
        kr, _ = ops.kv_read_q4(slots[:T], kc, vc)
        s = k[:T].float().view(T, H_kv, -1, 32).abs().amax(-1, keepdim=True) / 7
        step = (kr.float() - k[:T].float()).view(T, H_kv, -1, 32).abs() / s
        assert float(step.max()) <= 0.5 * (1 + 2.0 ** -4) + 1e-6  # half a step of a scale rounded up by 2^-4 at most
        ref = reference(inp)
        if len(set(new)) == 1:
            check(inp, *run_decode(ops, inp, new[0], device_error=err), ref, what=f"step {i}, decode")
        check(inp, *run_prefill(ops, inp, device_error=err), ref, what=f"step {i}, prefill")
    assert int(err) == 0
    held = set(pt[b, c].item() for b in range(B) for c in range(-(-int(lens[b]) // P)))
    assert held | set(free[:int(count)].tolist()) == set(range(n_pages)) and len(held) + int(count) == n_pages


def test_captured_decode_loop_allocates_its_own_pages(ops):
    """One captured step -- tables, append, decode -- replayed: lengths, pages and cache move on without the host."""
    B, H_q, H_kv, D, P = 3, 4, 2, 128, 16
    g = torch.Generator().manual_seed(6)

    def state():
        return dict(free=torch.arange(30, dtype=torch.int32, device=DEV), count=torch.tensor([30], dtype=torch.int32, device=DEV),
                    pt=torch.zeros((B, 8), dtype=torch.int32, device=DEV), lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                    kc=torch.zeros((30, H_kv, P, 72), dtype=torch.uint8, device=DEV),
                    vc=torch.zeros((30, H_kv, P, 72), dtype=torch.uint8, device=DEV))

    n = 35
    ks = torch.randn((n, B, H_kv, D), generator=g).to(BF16).to(DEV)
    vs = torch.randn((n, B, H_kv, D), generator=g).to(BF16).to(DEV)
    qs = torch.randn((n, B, H_q, D), generator=g).to(BF16).to(DEV)
    rel = torch.randn((B, H_q, 32), generator=g).to(DEV)
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, ops.decode_q4_workspace_bytes(B, 1, H_q, H_kv, D)), dtype=torch.uint8, device=DEV)
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    cu = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((B, H_q), device=DEV)

    def step(s):
        ops.build_tables(s["lens"], new, s["pt"], s["free"], s["count"], page_size=P, kv_lens=s["lens"],
                         cu_seqlens_q=cu, slot_map=slots, free_left=s["count"])
        ops.kv_append_q4(k, v, slots, s["kc"], s["vc"])
        ops.decode_q4(q, s["kc"], s["vc"], s["pt"], s["lens"], rel, window=20, scale=0.1, out=out, lse=lse, workspace=ws)

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


def test_convolved_rows_through_a_staging_pool(ops):
    """The short convolution ahead of the 4-bit append: kv_conv_append into a bf16 pool that holds only the step's
    rows, appended from there by slot."""
    B, H, D, P, width = 3, 2, 64, 16, 4
    g = torch.Generator().manual_seed(7)
    n = [1, 20, 5]
    T, per = sum(n), 2  # pages of staging per sequence
    cu = torch.tensor([0, 1, 21, 26], dtype=torch.int32, device=DEV)
    k = torch.randn((T, H, D), generator=g).to(BF16).to(DEV)
    v = torch.randn((T, H, D), generator=g).to(BF16).to(DEV)
    w = torch.randn((H, D, width), generator=g).to(DEV)
    st = [torch.randn((B, width - 1, H, D), generator=g).to(BF16).to(DEV) for _ in range(2)]
    stage = [torch.zeros((B * per, P, H, D), dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    lens = torch.tensor(n, dtype=torch.int32, device=DEV)  # positions within the step
    ops.kv_conv_append(k, v, cu, lens, table, stage[0], stage[1], w, w, st[0], st[1],
                       torch.arange(B, dtype=torch.int32, device=DEV), max_q_len=20)
    # slots of the staging rows: -1 where a sequence has no token
    slots = torch.full((B * per * P,), -1, dtype=torch.int64, device=DEV)
    for b, m in enumerate(n):
        slots[b * per * P:b * per * P + m] = torch.arange(m, device=DEV) + 40 * b
    kc = torch.zeros((10, H, P, 36), dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    rows = [s.view(B * per * P, H, D) for s in stage]
    ops.kv_append_q4(rows[0], rows[1], slots, kc, vc)
    want = q4.ref_append_q4(np.zeros((10, H, P, 36), dtype=np.uint8), f64(rows[0]), slots.cpu().numpy(), False)
    assert np.array_equal(kc.cpu().numpy(), want) and want.any()
