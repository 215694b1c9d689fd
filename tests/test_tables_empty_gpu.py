"""The tables of a step without requests: an empty packing, no slot, the stack as it was."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("max_tokens", [0, 1, 300])
def test_no_requests(max_tokens, in_place):
    import paged_attention_relative_attn_gb300 as ops
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    # buffers of the sizes that the call makes, full of something else and freed again
    old = [torch.full((n,), 77, dtype=t, device=DEV) for n, t in ((1, torch.int32), (max(max_tokens, 1), torch.int64))
           for _ in range(20)]
    del old
    count = torch.tensor([3], dtype=torch.int32, device=DEV)
    free = torch.tensor([5, 2, 1, 9, 9, 9], dtype=torch.int32, device=DEV)
    kw = dict(free_left=count) if in_place else {}
    kv, cu, slots, left = ops.build_tables(z(0), z(0), z(0, 4), free, count, page_size=16, max_tokens=max_tokens, **kw)
    assert kv.shape == (0,) and cu.tolist() == [0] and left.tolist() == [3] and count.tolist() == [3]
    assert slots.tolist() == [-1] * max_tokens and free.tolist() == [5, 2, 1, 9, 9, 9]


def test_no_requests_on_another_stream_and_captured():
    import paged_attention_relative_attn_gb300 as ops
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    args = (z(0), z(0), z(0, 4), z(6), torch.tensor([3], dtype=torch.int32, device=DEV))
    cu, slots, left = z(1) + 9, torch.full((5,), 9, device=DEV), z(1) + 9
    kw = dict(page_size=16, kv_lens=z(0), cu_seqlens_q=cu, slot_map=slots, free_left=left)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ops.build_tables(*args, stream=side, **kw)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and left.tolist() == [3]
    cu.fill_(9), slots.fill_(9), left.fill_(9)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.build_tables(*args, **kw)
    g.replay()
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and left.tolist() == [3]
