"""decode_q4's limit on the scale, without a GPU."""

from __future__ import annotations

import pytest


def test_scale_limit():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    a = dict(q=16, k_cache=16, v_cache=16, page_table=4, page_table_stride=4, seq_lens=4, rel_logits=4, B=2, q_len=1,
             H_q=4, H_kv=2, D=64, page_size=16, num_pages=16, R=32, window=32, scale=0.125, out=16, lse_out=None,
             workspace=8, workspace_bytes=0, device_error=None, stream=None)
    f = lambda s: _lib.inkling_rel_attn_decode_q4(**{**a, "scale": s})  # noqa: E731
    for s in (0.0, -0.1, 2.0 ** 54, -2.0 ** 54, 1e-40):
        assert f(s) == -2, s  # the next check, the workspace's alignment, is reached
    for s in (2.0 ** 54 * (1 + 2.0 ** -23), -2.0 ** 55, float("inf"), -float("inf"), float("nan")):
        assert f(s) == -1, s
