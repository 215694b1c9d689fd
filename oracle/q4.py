"""CPU oracle of the 4-bit cache and the step tables (test infrastructure only).

Plain NumPy / Python, one small step per function, written from the definitions
in include/inkling_rel_attn.h ("The 4-bit cache", inkling_rel_attn_build_tables).
Attention over a 4-bit cache is ``oracle.ref``'s over the values it stands for.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

MOST = 2.0 ** 127  # larger magnitudes count as it: 7 s then stays finite


def group_scale(a: float) -> float:
    """Smallest number of 5 significant bits that is at least a / 7 (exact arithmetic)."""
    if a < 2.0 ** -100:
        return 0.0
    need = Fraction(a) / 7
    e = 0
    while Fraction(2) ** (e + 1) <= need:
        e += 1
    while Fraction(2) ** e > need:
        e -= 1
    step = Fraction(2) ** (e - 4)
    n = -((-need) // step)  # ceiling
    return float(n * step)


def round_x(v: float, s: float) -> int:
    """v / s to the nearest integer, ties toward zero."""
    if s == 0.0:
        return 0
    t = abs(Fraction(v)) / Fraction(s)
    n = -((Fraction(1, 2) - t) // 1)  # ceil(t - 1/2)
    n = max(0, int(n))
    return n if v > 0 else -n


def quantise_group(v: np.ndarray):
    """(x int [32], s) of 32 values; s is NaN when one of them is."""
    if np.isnan(v).any():
        return np.zeros(len(v), dtype=np.int64), float("nan")
    v = np.clip(v, -MOST, MOST)
    s = group_scale(float(np.abs(v).max()))
    return np.array([round_x(float(y), s) for y in v], dtype=np.int64), s


def nibble_of(c: int, D: int, is_v: bool) -> int:
    """Nibble position of channel c within its row of D / 2 bytes."""
    N = D // 32
    j, r = divmod(c, 32)
    w = 4 if is_v else 8
    return w * (N * (r // w) + j) + r % w


def block_at(head: int, place: int, P: int, D: int):
    """(offset of the 16-token block, row within it) inside a page of one KV head's bytes."""
    return (place // 16) * (9 * D), place % 16


def write_row(page: np.ndarray, place: int, x: np.ndarray, s: np.ndarray, is_v: bool):
    """Store one row: page = the bytes [P * 9 * D / 16] of one (page, KV head)."""
    D = len(x)
    base, r = block_at(0, place, len(page) * 16 // (9 * D), D)
    for c in range(D):
        n = nibble_of(c, D, is_v)
        at, sh = base + r * (D // 2) + n // 2, 4 * (n % 2)
        page[at] = (int(page[at]) & ~(15 << sh)) | ((int(x[c]) + 8) << sh)
    for j, sc in enumerate(s):
        bits = int(np.float32(sc).view(np.uint32)) >> 16
        at = base + 8 * D + 2 * (r * (D // 32) + j)
        page[at], page[at + 1] = bits & 255, bits >> 8


def read_pool(pool: np.ndarray, is_v: bool) -> np.ndarray:
    """float64 [num_pages, P, H_kv, D]: the values a pool [num_pages, H_kv, P, 9 * D / 16] stands for."""
    n, H, P, row = pool.shape
    D = row * 16 // 9
    flat = pool.reshape(n, H, P // 16, 9 * D)
    data = flat[..., :8 * D].reshape(n, H, P, D // 2)
    sc = np.ascontiguousarray(flat[..., 8 * D:]).view(np.uint16).reshape(n, H, P, D // 32)
    scale = (sc.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    out = np.empty((n, P, H, D))
    for c in range(D):
        nb = nibble_of(c, D, is_v)
        x = ((data[..., nb // 2] >> (4 * (nb % 2))) & 15).astype(np.float64) - 8
        out[..., c] = (x * scale[..., c // 32]).transpose(0, 2, 1)
    return out


def ref_append_q4(pool: np.ndarray, rows: np.ndarray, slots, is_v: bool) -> np.ndarray:
    """The pool after rows [T, H_kv, D] (float64 of bf16 values) went to their slots."""
    out = pool.copy()
    n, H, P, _ = pool.shape
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= n * P:
            continue
        for h in range(H):
            parts = [quantise_group(rows[t, h, g:g + 32]) for g in range(0, rows.shape[2], 32)]
            write_row(out[slot // P, h].reshape(-1), int(slot % P), np.concatenate([x for x, _ in parts]),
                      np.array([s for _, s in parts]), is_v)
    return out


def ref_build_tables(seq_lens, new_lens, page_table, free_pages, free_count, P, max_tokens):
    """One request after the other.  Returns a dict of the outputs and the set of reported bits."""
    table, free = page_table.copy(), free_pages.copy()
    B, stride = table.shape
    top, bits = int(free_count), set()
    for b in range(B):
        if new_lens[b] < 0:
            for c in range(-(-int(seq_lens[b]) // P)):
                if top < len(free):
                    free[top] = page_table[b, c]
                    top += 1
                else:
                    bits.add("bad_page")
    kv = np.zeros(B, dtype=np.int64)
    slots, cu, asked, left = [], [0], 0, top
    for b in range(B):
        L, n = int(seq_lens[b]), int(new_lens[b])
        cu.append(cu[-1] + max(n, 0))
        if n < 0:
            continue
        had, need = -(-L // P), -(-(L + n) // P) - (-(-L // P))
        if n > 0 and cu[-1] > max_tokens:
            bits.add("bad_chunk")
        if L + n > stride * P:
            bits.add("too_long")
            need, served = 0, False
        elif n > 0 and cu[-1] > max_tokens:
            served = False
        else:
            asked += need
            served = need == 0 or asked <= top
            if not served:
                bits.add("no_pages")
        if served:
            for c in range(need):
                left -= 1
                table[b, had + c] = free[left]
        kv[b] = L + n if served else L
        for p in range(L, L + n):
            slots.append(int(table[b, p // P]) * P + p % P if served else -1)
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return dict(kv_lens=kv, cu=np.array(cu), slots=np.array(slots, dtype=np.int64), table=table, free=free,
                left=left, bits=bits)
