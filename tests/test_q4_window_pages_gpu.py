"""Pages that lie wholly behind a window may be gone (their entries anything): no call on the 4-bit cache looks at
them or reports them, as on the bf16 cache."""

from __future__ import annotations

import dataclasses

import pytest
import torch

from tests.q4_cases import check, make
from tests.test_q4_gpu import DEV, run_decode, run_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def without_old_pages(inp, q_lens):
    pt = inp.page_table.clone()
    P = inp.k_cache.shape[2]
    gone = 0
    for b, (L, n) in enumerate(zip(inp.seq_lens.tolist(), q_lens)):
        old = max(0, L - n - inp.window + 1) // P  # pages with no key that the oldest new token sees
        pt[b, :old] = torch.tensor([-1, 1 << 30, -(1 << 31)], dtype=torch.int32, device=DEV)[b % 3]
        gone += old
    assert gone
    return dataclasses.replace(inp, page_table=pt)


@pytest.mark.parametrize("P", [16, 32, 48, 64, 128])
@pytest.mark.parametrize("q_len,D,G", [(1, 64, 2), (1, 128, 3), (3, 64, 2), (5, 128, 16)])
def test_decode(ops, P, q_len, D, G):
    # first visible keys: every 16-key step of a 64-key period, and the last key of a page
    lens = [150 + 16 * i for i in range(5)] + [300, 305, 320, 40, 1000]
    window = 100 - q_len
    inp = make([q_len] * len(lens), lens, 2 * G, 2, D, P, window, 64, seed=P)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want, lwant = run_decode(ops, inp, q_len)
    out, lse = run_decode(ops, without_old_pages(inp, [q_len] * len(lens)), q_len, device_error=err)
    assert int(err) == 0
    assert torch.equal(out, want) and torch.equal(lse, lwant)
    check(inp, out, lse)


@pytest.mark.parametrize("P", [16, 32, 48, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill(ops, P, D):
    q_lens, lens = [1, 130, 7, 40, 3], [300, 500, 176, 161, 1000]
    inp = make(q_lens, lens, 4, 2, D, P, 50, 64, seed=200 + P)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    need = ops.prefill_q4_workspace_bytes(len(lens), 130, 2, D, 50, 1000)
    want, lwant = run_prefill(ops, inp)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN in every bf16 of it
    out, lse = run_prefill(ops, without_old_pages(inp, q_lens), workspace=ws, device_error=err)
    assert int(err) == 0
    assert torch.equal(out, want) and torch.equal(lse, lwant)
    check(inp, out, lse)


@pytest.mark.parametrize("P", [16, 64])
def test_widest_window(ops, P):
    """A window of 2^31 - 1 keys hides nothing."""
    inp = make([2, 2, 2], [2, 40, 300], 4, 2, 64, P, 0, 64, seed=9)
    wide = dataclasses.replace(inp, window=2 ** 31 - 1)
    for call in (lambda x: run_decode(ops, x, 2), lambda x: run_prefill(ops, x)):
        for a, b in zip(call(inp), call(wide)):
            assert torch.equal(a, b)
