"""CPU oracle of shared pages (test infrastructure only): one request after the other, from the definitions in
include/inkling_rel_attn.h ("Shared pages")."""

from __future__ import annotations

import numpy as np


def pages_for(tokens: int, P: int) -> int:
    return -(-int(tokens) // P)


def ref_fork(source, seq_lens, table, refs, free, count, P):
    """Returns a dict of the outputs and the set of reported bits."""
    table, refs = table.copy(), refs.copy()
    B, stride = table.shape
    kv, bits = np.array(seq_lens), set()
    src, dst = np.full(B, -1), np.full(B, -1)
    top = int(count)
    for b in range(B):
        s = int(source[b])
        if s < 0:
            continue
        if s >= B or seq_lens[b] != 0:
            bits.add("bad_slot")
            continue
        n = int(seq_lens[s])
        if n > stride * P:
            bits.add("too_long")
            continue
        full = n // P
        if any(not 0 <= page < len(free) for page in table[s, :pages_for(n, P)]):
            bits.add("bad_page")
            continue
        if n % P and top == 0:
            bits.add("no_pages")
            continue
        if n % P:
            top -= 1
            if not 0 <= free[top] < len(free):
                bits.add("bad_page")
                continue
            src[b], dst[b] = table[s, full], free[top]
            table[b, full] = free[top]
        for c in range(full):
            table[b, c] = table[s, c]
            refs[table[s, c]] += 1
        kv[b] = n
    return dict(kv_lens=kv, table=table, refs=refs, src=src, dst=dst, left=top, bits=bits)


def ref_release(seq_lens, new_lens, table, refs, free, count, P):
    refs, free = refs.copy(), free.copy()
    bits, top = set(), int(count)
    entries = [(b, int(table[b, c])) for b in range(len(seq_lens)) if new_lens[b] < 0
               for c in range(pages_for(seq_lens[b], P))]
    last = {page: i for i, (_, page) in enumerate(entries)}
    owners = {page: int(refs[page]) + 1 for _, page in entries}
    for _, page in entries:
        owners[page] -= 1
    for i, (_, page) in enumerate(entries):
        if last[page] != i:
            continue
        if owners[page] > 0:
            refs[page] = owners[page] - 1
            continue
        if owners[page] < 0:
            bits.add("bad_page")
        refs[page] = 0
        if top < len(free):
            free[top] = page
            top += 1
        else:
            bits.add("bad_page")
    kv = np.where(np.array(new_lens) < 0, 0, seq_lens)
    return dict(kv_lens=kv, refs=refs, free=free, left=top, bits=bits)


def ref_compact(seq_lens, table, refs, free, count, P):
    table, refs, free = table.copy(), refs.copy(), free.copy()
    n = len(free)
    live = sorted({int(table[b, c]) for b in range(len(seq_lens)) for c in range(pages_for(seq_lens[b], P))})
    named = [int(x) for x in free[:count] if x != -1]  # (-1: a place without a page, as a compaction leaves it)
    stack = {x for x in named if 0 <= x < n}
    bits = {"bad_page"} if stack & set(live) or len(stack) < len(named) else set()
    known = sorted(set(live) | stack)
    low, high = known[:len(live)], known[len(live):]
    src = [x for x in high if x in live]
    dst = [x for x in low if x not in live]
    to = dict(zip(src, dst))
    for b in range(len(seq_lens)):
        for c in range(pages_for(seq_lens[b], P)):
            table[b, c] = to.get(int(table[b, c]), table[b, c])
    for a, z in to.items():
        refs[z], refs[a] = refs[a], 0
    free[:count] = [-1] * (count - len(high)) + high[::-1]
    pad = [-1] * (n - len(src))
    return dict(table=table, refs=refs, free=free, src=np.array(src + pad), dst=np.array(dst + pad), moves=len(src),
                bits=bits)
