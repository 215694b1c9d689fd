"""Prefill through many key tiles, the last of them partly visible inside its page, as pages of other than 64 tokens
leave it: close to the oracle and the same bits in every run."""

from __future__ import annotations

import pytest
import torch

import workloads as W
from tests.helpers import MEAN_ABS, f64, oracle_prefill

pytestmark = pytest.mark.gpu

CASES = [
    # q_lens, kv_lens, H_q, H_kv, D, P, window, R
    ([140, 70], [400, 300], 2, 1, 128, 16, 0, 512),
    ([140, 70], [400, 300], 2, 1, 64, 48, 0, 512),
    ([1, 129, 300], [777, 1000, 300], 6, 2, 128, 32, 0, 64),
    ([200, 33, 5], [1000, 2000, 450], 4, 4, 64, 80, 700, 256),
    ([260], [3000], 8, 1, 128, 16, 1500, 1024),
    ([140, 70], [410, 330], 2, 1, 128, 128, 0, 512),
    ([100, 140, 1], [1800, 600, 1360], 4, 2, 64, 256, 0, 64),
    ([130] * 3, [721, 980, 3000], 6, 1, 128, 192, 900, 512),
    ([64] * 12, [211 + 64 * i + i for i in range(12)], 16, 8, 128, 48, 0, 128),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_many_tiles(case):
    import paged_attention_relative_attn_gb300 as ops
    ql, kl, H_q, H_kv, D, P, win, R = CASES[case]
    cache = W.make_prefill_cache(kl, H_kv, D, P, device="cuda", seed=30 + case, poison=True)
    inp = W.make_prefill(cache, ql, kl, H_q, R, win, device="cuda", seed=40 + case)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = ops.prefill_inputs(inp, device_error=err)
    for _ in range(20):
        again, l2 = ops.prefill_inputs(inp)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    assert int(err) == 0
    ro, rl, rows = oracle_prefill(inp)
    # weights and result rounded to bf16, 2^-8 of a row's |V|-weighted sum (at most its largest |V|) and of the result
    vmax = float(inp.v_cache[~torch.isnan(inp.v_cache)].abs().max())
    d = abs(f64(out) - ro)
    assert d.max() <= 2.0 ** -8 * 1.02 * 2 * vmax and d.mean() <= MEAN_ABS
    assert abs(f64(lse) - rl).max() <= 1e-4 + 2.0 ** -20 * abs(rl).max()
