"""Prefill over the 4-bit cache is the bf16 cache's prefill of the values it stands for, to the bit where pages hold 64
tokens: both walk the visible keys in the same tiles (larger pages let a tile start in mid-page, which the expanded ones
do not have, so sums are taken in another order).  At serving sizes too: whole chunks, many KV heads."""

from __future__ import annotations

import pytest
import torch

from tests.q4_cases import make
from tests.test_q4_gpu import DEV, run_prefill

pytestmark = pytest.mark.gpu


def values(ops, inp):
    """bf16 caches [pages, P, H_kv, D] of the values of the 4-bit pools (read back bit for bit)."""
    n, H, P, row = inp.k_cache.shape
    k, v = ops.kv_read_q4(torch.arange(n * P, device=DEV), inp.k_cache, inp.v_cache)
    return k.view(n, P, H, -1), v.view(n, P, H, -1)


CASES = [
    # q_lens, kv_lens, H_q, H_kv, D, P, window, R
    ([200, 40], [900, 300], 6, 2, 128, 64, 128, 64),
    ([130, 1, 64], [130, 700, 65], 4, 4, 64, 128, 0, 64),
    ([2048, 2048, 700], [4100, 2048, 1500], 16, 16, 128, 64, 512, 512),
    ([2048], [5000], 24, 8, 128, 64, 0, 1024),
    ([1500, 300], [1500, 3333], 16, 8, 64, 256, 0, 256),
    ([2048, 2048], [2500, 6000], 5, 5, 64, 64, 777, 128),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_bits_of_the_bf16_prefill(case):
    import paged_attention_relative_attn_gb300 as ops
    ql, kl, H_q, H_kv, D, P, win, R = CASES[case]
    inp = make(ql, kl, H_q, H_kv, D, P, win, R, seed=500 + case, poison=False)
    kc, vc = values(ops, inp)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run_prefill(ops, inp, device_error=err)
    want, wl = ops.prefill(inp.q, inp.cu_seqlens_q, kc, vc, inp.page_table, inp.seq_lens, inp.rel_logits, window=win,
                           scale=inp.scale, max_seq_len=inp.max_seq_len, max_q_len=inp.max_q_len, device_error=err)
    assert int(err) == 0 and bool(torch.isfinite(out.float()).all())
    if P == 64:
        assert torch.equal(out, want) and torch.equal(lse, wl)
        return
    # each is off by a bf16 rounding of the weights, 2^-8 of the |V|-weighted sum, and one of the result, 2^-8 of it;
    # the |V|-weighted sum is itself known to 2^-7 of it
    size = ops.prefill(inp.q, inp.cu_seqlens_q, kc, vc.abs(), inp.page_table, inp.seq_lens, inp.rel_logits, window=win,
                       scale=inp.scale, max_seq_len=inp.max_seq_len, max_q_len=inp.max_q_len)[0].double()
    d = (out.double() - want.double()).abs()
    assert bool((d <= 2 * 2.0 ** -8 * (1 + 2.0 ** -6) * (size + want.double().abs())).all())
    assert float((lse - wl).abs().max()) <= 2.0 ** -18 * float(wl.abs().max().clamp(min=1))
