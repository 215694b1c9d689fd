"""Barriers over a cluster are reached out of loops whose trip counts differ within a warp, which the .aligned forms do
not allow."""

from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_relative_attn_gb300", "csrc")


def test_cluster_barriers_are_not_aligned():
    seen = 0
    for f in os.listdir(CSRC):
        for line in re.findall(r'"barrier\.cluster[^"]*"', open(os.path.join(CSRC, f)).read()):
            seen += 1
            assert ".aligned" not in line, (f, line)
    assert seen >= 2
