"""The 4-bit cache on the GPU, further: calls large enough for two heads per thread, rows of tokens hidden from
some of the drafts, odd group sizes, runs of many short items, tables whose pages come back and go at once."""

from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

import oracle.q4 as q4
from tests.helpers import f64
from tests.q4_cases import check, make, reference
from tests.test_q4_gpu import BF16, DEV, run_decode, special_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


@pytest.mark.parametrize("T,H,D,P", [(8001, 3, 128, 48), (9000, 5, 64, 16), (5000, 16, 64, 256)])
def test_large_append_and_read_bit_exact(ops, T, H, D, P):
    g = torch.Generator().manual_seed(T)
    n = (T + P - 1) // P + 2
    k, v = special_rows(T, H, D, 13), special_rows(T, H, D, 14)
    slots = torch.randperm(n * P, generator=g)[:T]
    slots[::17] = -1
    kc = torch.randint(0, 256, (n, H, P, 9 * D // 16), dtype=torch.uint8, generator=g)
    vc = torch.randint(0, 256, (n, H, P, 9 * D // 16), dtype=torch.uint8, generator=g)
    want_k = q4.ref_append_q4(kc.numpy(), f64(k), slots.numpy(), False)
    want_v = q4.ref_append_q4(vc.numpy(), f64(v), slots.numpy(), True)
    kd, vd, sd = kc.to(DEV), vc.to(DEV), slots.to(DEV)
    ops.kv_append_q4(k.to(DEV), v.to(DEV), sd, kd, vd)
    assert np.array_equal(kd.cpu().numpy(), want_k) and np.array_equal(vd.cpu().numpy(), want_v)
    kr, vr = ops.kv_read_q4(sd, kd, vd)
    at = slots.numpy()
    live = at >= 0
    for got, pool, is_v in ((kr, want_k, False), (vr, want_v, True)):
        want = np.zeros((T, H, D))
        want[live] = q4.read_pool(pool, is_v)[at[live] // P, at[live] % P]
        assert np.array_equal(f64(got), want, equal_nan=True)


@pytest.mark.parametrize("D,G", [(128, 3), (64, 2), (128, 1)])
def test_nan_rows_of_hidden_tokens_stay_out(ops, D, G):
    """Four drafts: the last one's row is NaN, and so is the oldest one that the first draft alone sees."""
    H, P, L, win = 2, 16, 90, 20
    inp = make([4, 4], [L, 55], H * G, H, D, P, win, 32, seed=90 + G)
    clean, lclean = run_decode(ops, inp, 4)
    kc, vc = inp.k_cache.clone(), inp.v_cache.clone()
    pt = inp.page_table.cpu()
    nan = torch.full((1, H, D), float("nan"), dtype=BF16, device=DEV)
    for pos in (L - 1, L - 4 - (win - 1)):
        slot = torch.tensor([int(pt[0, pos // P]) * P + pos % P], device=DEV)
        ops.kv_append_q4(nan, nan, slot, kc, vc)
    out, lse = run_decode(ops, dataclasses.replace(inp, k_cache=kc, v_cache=vc), 4)
    for row in (0, 3):                                   # see one of the two
        assert bool(torch.isnan(out[row].float()).all()) and bool(torch.isnan(lse[row]).all())
    assert torch.equal(out[4:], clean[4:]) and torch.equal(lse[4:], lclean[4:])  # the other sequence
    for row in (0, 3):                                   # rows 1 and 2 see neither: as exact as without them
        out[row], lse[row] = clean[row], lclean[row]
    check(inp, out, lse, reference(inp))


@pytest.mark.parametrize("q_len,kv_lens,G,H_kv,D,P,window,R", [
    (1, [300, 41, 1000], 11, 2, 128, 16, 0, 32),
    (2, [700, 33], 13, 1, 128, 64, 200, 64),
    (1, [513, 2], 15, 3, 64, 32, 0, 5),
    (3, [90, 400], 7, 2, 64, 16, 64, 64),
    (5, [1200], 2, 3, 128, 48, 0, 256),
    (9, [333, 9], 8, 1, 128, 16, 0, 1),
])
def test_group_sizes(ops, q_len, kv_lens, G, H_kv, D, P, window, R):
    inp = make([q_len] * len(kv_lens), kv_lens, G * H_kv, H_kv, D, P, window, R, seed=G)
    check(inp, *run_decode(ops, inp, q_len), reference(inp))


def test_runs_of_many_short_items(ops):
    """Hundreds of sequences of one to a few tiles: a thread block's run holds many items, some of them cut."""
    r = np.random.default_rng(3)
    lens = r.integers(0, 140, 700).tolist()
    inp = make([1] * 700, lens, 6, 2, 64, 16, 0, 16, seed=17)
    check(inp, *run_decode(ops, inp, 1), reference(inp))
    lens = (2 + r.integers(0, 60, 300)).tolist()
    inp = make([2] * 300, lens, 8, 4, 128, 16, 40, 16, seed=18)
    check(inp, *run_decode(ops, inp, 2), reference(inp))


def test_pages_go_from_ended_requests_to_several_others(ops):
    """The stack is nearly empty: most pages that 30 growing requests take are those of 20 ended ones."""
    P, B = 48, 50
    lens = np.array([P * 7 + 5] * B)
    held = -(-lens // P)
    ids = np.random.default_rng(5).permutation(int(held.sum()) + 3)
    pt = np.full((B, 20), -1)
    at = 0
    for b in range(B):
        pt[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(len(ids), -7)
    free[:3] = ids[at:]
    new = np.where(np.arange(B) % 5 < 2, -1, 4 * P + 3)
    want = q4.ref_build_tables(lens, new, pt, free, 3, P, 8000)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    d = [i32(x) for x in (lens, new, pt, free, [3])]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kv, cu, slots, left = ops.build_tables(*d, page_size=P, max_tokens=8000, device_error=err)
    assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(d[2].cpu().numpy(), want["table"])
    assert np.array_equal(d[3].cpu().numpy(), want["free"]) and int(left) == want["left"] and int(err) == 0
    live = slots[slots >= 0]
    assert live.unique().numel() == live.numel()


def test_buffers_made_for_another_stream(ops):
    """A freed tensor of the current stream, which still has a write to it in its queue, is not taken for the
    buffers of a call on another stream."""
    inp = make([1] * 3, [200, 77, 300], 4, 2, 128, 16, 0, 64, seed=95)
    want, lwant = run_decode(ops, inp, 1)
    slots = torch.arange(40, device=DEV)
    kw, vw = ops.kv_read_q4(slots, inp.k_cache, inp.v_cache)
    pf = dict(window=0, scale=inp.scale, max_seq_len=300, max_q_len=1)
    cu = torch.arange(4, dtype=torch.int32, device=DEV)
    args = (inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits)
    pwant, _ = ops.prefill_q4(inp.q, cu, *args, **pf)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, ref in ((lambda: run_decode(ops, inp, 1, stream=side)[0], want),
                      (lambda: run_decode(ops, inp, 1, stream=side)[1], lwant),
                      (lambda: ops.kv_read_q4(slots, inp.k_cache, inp.v_cache, stream=side)[1], vw),
                      (lambda: ops.prefill_q4(inp.q, cu, *args, stream=side, **pf)[0], pwant)):
        torch.cuda._sleep(20_000_000)
        old = [torch.zeros_like(ref) for _ in range(8)]      # written after the sleep
        del old
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
