"""CPU oracle of the 8-bit cache (test infrastructure only).

Plain NumPy / Python, one small step per function, written from the definition
in include/inkling_rel_attn.h ("The 8-bit cache", inkling_rel_attn_kv_append_q8).
Attention over an 8-bit cache is ``oracle.ref``'s over the values it stands for.
"""

from __future__ import annotations

import functools
from fractions import Fraction

import numpy as np

E_MIN, E_MAX, MOST = -60, 55, 448


def e4m3_values() -> np.ndarray:
    """The value of each byte, in float64 (0x7f and 0xff: NaN)."""
    out = np.empty(256)
    for b in range(256):
        ex, man = (b >> 3) & 15, b & 7
        mag = Fraction(man, 8) / 64 if ex == 0 else (1 + Fraction(man, 8)) * Fraction(2) ** (ex - 7)
        out[b] = np.nan if b & 127 == 127 else float(mag) * (-1 if b & 128 else 1)
    return out


VALUES = e4m3_values()


def e4m3_byte(x: float) -> int:
    """The byte of the nearest e4m3 number, ties to even, magnitudes past 448 as 448 (exact arithmetic)."""
    a = abs(Fraction(x))
    sign = 128 if np.copysign(1.0, x) < 0 else 0
    mags = [Fraction(float(VALUES[b])) for b in range(127)]
    lo = max(b for b in range(127) if mags[b] <= a)
    if lo == 126:
        return sign | 126
    mid = (mags[lo] + mags[lo + 1]) / 2
    up = a > mid or (a == mid and lo % 2 == 1)
    return sign | (lo + 1 if up else lo)


MAGS = VALUES[:127]


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """e4m3_byte of every value.  float64 holds all that occurs: a value of few bits over a power of two."""
    a = np.minimum(np.abs(x), MOST)
    step = np.exp2(np.maximum(np.frexp(a)[1] - 1, -6) - 3)  # a = m 2^e, m in [1/2, 1)
    q = np.rint(a / step) * step                            # (2 steps of one octave are one of the next)
    return (np.searchsorted(MAGS, q) + 128 * np.signbit(x)).astype(np.uint8)


def exponent_for(amax: float) -> int:
    """Smallest e in the range with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and Fraction(amax) > MOST * Fraction(2) ** e:
        e += 1
    return e


def place_of(r: int, c: int, D: int, is_v: bool) -> int:
    """Byte of channel c of row r in its block."""
    if D == 64 and not is_v:
        return 64 * r + c
    if D == 64:
        return 128 * (r // 2) + 8 * (4 * ((2 * (r % 2) + c // 32) ^ (r // 2 % 4)) + c // 8 % 4) + c % 8
    return 128 * r + 16 * ((c // 16) ^ (2 * (r // 2 % 4) if is_v else 4 * (r % 2))) + c % 16


@functools.lru_cache(None)
def places(D: int, is_v: bool) -> np.ndarray:
    return np.array([[place_of(r, c, D, is_v) for c in range(D)] for r in range(16)])


def block_of(pool: np.ndarray, slot: int, h: int) -> np.ndarray:
    """The bytes (a view) of the block that holds a slot."""
    n, H, P, row = pool.shape
    size = 16 * row
    page = pool.reshape(n, H, P * row)[slot // P, h]
    b = slot % P // 16
    return page[b * size:(b + 1) * size]


def tail_of(block: np.ndarray):
    """(exponent or None if the block has not been begun, NaN rows as a set)."""
    D = len(block) // 16 - 1
    s = block[16 * D:16 * D + 4].copy().view(np.float32)[0]
    m, e = np.frexp(s)
    begun = m == 0.5 and E_MIN <= e - 1 <= E_MAX
    bits = int(block[16 * D + 4]) | int(block[16 * D + 5]) << 8
    return (int(e) - 1 if begun else None), {r for r in range(16) if bits >> r & 1}


def write_tail(block: np.ndarray, e: int, nan_rows):
    D = len(block) // 16 - 1
    block[16 * D:] = 0
    block[16 * D:16 * D + 4] = np.array([2.0 ** e], dtype=np.float32).view(np.uint8)
    bits = sum(1 << r for r in nan_rows)
    block[16 * D + 4], block[16 * D + 5] = bits & 255, bits >> 8


def join_block(block: np.ndarray, rows: dict, is_v: bool):
    """Rows {place: float64 [D]} join a block (in place)."""
    D = len(block) // 16 - 1
    at = places(D, is_v)
    e_old, nan_rows = (None, set()) if 0 in rows else tail_of(block)
    if e_old is None:
        nan_rows = set()
    bad = {r for r, v in rows.items() if np.isnan(v).any()}
    big = max((float(np.abs(v).max()) for r, v in rows.items() if r not in bad), default=0.0)
    e = exponent_for(min(big, MOST * 2.0 ** E_MAX))
    if e_old is not None:
        e = max(e, e_old)
        for r in range(16):
            if r not in rows and e > e_old:
                x = VALUES[block[at[r]]] * 2.0 ** (e_old - e)
                # (a NaN byte is of a place without a row; what it becomes is nobody's matter)
                block[at[r]] = np.where(np.isnan(x), 0x7f, e4m3_bytes(np.nan_to_num(x)))
    for r, v in rows.items():
        x = np.clip(v, -MOST * 2.0 ** E_MAX, MOST * 2.0 ** E_MAX) * 2.0 ** -e
        block[at[r]] = 0 if r in bad else e4m3_bytes(x)
    write_tail(block, e, (nan_rows - set(rows)) | bad)


def ref_append_q8(pool: np.ndarray, rows: np.ndarray, slots, is_v: bool) -> np.ndarray:
    """The pool after rows [T, H_kv, D] (float64 of bf16 values) went to their slots, block by block."""
    out = pool.copy()
    n, H, P, _ = pool.shape
    blocks = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < n * P:
            blocks.setdefault(int(slot) // 16, []).append((t, int(slot)))
    for tokens in blocks.values():
        for h in range(H):
            join_block(block_of(out, tokens[0][1], h), {s % 16: rows[t, h] for t, s in tokens}, is_v)
    return out


def read_pool(pool: np.ndarray, is_v: bool) -> np.ndarray:
    """float64 [num_pages, P, H_kv, D]: the values a pool [num_pages, H_kv, P, D + 1] stands for."""
    n, H, P, row = pool.shape
    D = row - 1
    flat = pool.reshape(n, H, P // 16, 16 * row)
    x = VALUES[flat[..., places(D, is_v)]]  # [n, H, P / 16, 16, D]
    s = np.ascontiguousarray(flat[..., 16 * D:16 * D + 4]).view(np.float32)[..., 0].astype(np.float64)
    bits = flat[..., 16 * D + 4].astype(np.int64) | flat[..., 16 * D + 5].astype(np.int64) << 8
    bad = (bits[..., None] >> np.arange(16)) & 1 > 0
    with np.errstate(invalid="ignore"):
        x = np.where(bad[..., None], np.nan, x * s[..., None, None])
    return x.reshape(n, H, P, D).transpose(0, 2, 1, 3)
