"""A stream of another device than the tensors' is refused, whatever the call."""

from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from tests.q4_cases import make
from tests.test_q4_gpu import BF16, DEV, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def test_stream_of_another_device():
    import paged_attention_relative_attn_gb300 as ops
    # stands for a stream of a second GPU: nothing may be launched on it or on another in its stead
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0, device_index=1, stream_id=0, device_type=1)
    inp = make([1, 1], [30, 40], 4, 2, 64, 16, 0, 8, seed=1)
    rows, slots = torch.zeros((4, 2, 64), dtype=BF16, device=DEV), torch.arange(4, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    pool = inp.k_cache.clone()
    table, free = i32(2, 4), i32(8)
    out = torch.full_like(inp.q, 7.0)
    for call in (lambda: run_decode(ops, inp, 1, out=out, stream=other), lambda: run_prefill(ops, inp, out=out, stream=other),
                 lambda: ops.kv_append_q4(rows + 1, rows + 1, slots, pool, pool, stream=other),
                 lambda: ops.kv_read_q4(slots, pool, pool, stream=other),
                 lambda: ops.build_tables(i32(2), i32(2) + 1, table, free, i32(1) + 8, page_size=16, max_tokens=4,
                                          stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and torch.equal(pool, inp.k_cache) and not table.any()
