"""Inputs and bounds shared by the tests of the 4-bit cache."""

from __future__ import annotations

import numpy as np
import torch

import workloads as W
from oracle.q4 import read_pool
from oracle.ref import ref_prefill
from tests.helpers import f64


S_MAX = 0.4  # the largest scale of random_pool


def random_pool(n, H, P, D, seed, device, std=1.0):
    """A pool of random nibbles (x in -7..7) and scales of 5 significant bits; D / 32 groups.  Drawn as
    bytes, so no quantiser is involved."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randint(1, 16, (n, H, P // 16, 16 * D), generator=g, dtype=torch.uint8)
    data = u[..., 0::2] | (u[..., 1::2] << 4)
    s = std * 0.2 * (1 + torch.rand((n, H, P // 16, D // 2), generator=g))
    s = (s.view(torch.int32) & ~0x7FFFF).view(torch.float32).to(torch.bfloat16)
    return torch.cat([data, s.view(torch.uint8)], -1).reshape(n, H, P, 9 * D // 16).to(device)


def poison_pool(pool, pt, lens):
    """Every byte of places that hold no token becomes 0xff (nibble 15, scale NaN)."""
    n, H, P, row = pool.shape
    D = row * 16 // 9
    live = torch.zeros((n, P), dtype=torch.bool)
    for b, L in enumerate(lens):
        for j in range(L):
            live[int(pt[b, j // P]), j % P] = True
    blocks = pool.view(n, H, P // 16, 9 * D)
    dead = ~live.view(n, 1, P // 16, 16, 1).to(pool.device)
    data = blocks[..., :8 * D].reshape(n, H, P // 16, 16, D // 2)
    scale = blocks[..., 8 * D:].reshape(n, H, P // 16, 16, D // 16)
    blocks[..., :8 * D] = torch.where(dead, torch.full_like(data, 255), data).flatten(-2)
    blocks[..., 8 * D:] = torch.where(dead, torch.full_like(scale, 255), scale).flatten(-2)


def make(q_lens, kv_lens, H_q, H_kv, D, P, window, R, seed, device="cuda", q_std=1.0, poison=True, extra=2):
    """A PrefillInputs whose caches are 4-bit pools; decode of equal q_lens takes the same inputs."""
    gc = torch.Generator().manual_seed(seed)
    n = sum(W.pages_for(L, P) for L in kv_lens) + extra
    pt, _ = W.build_page_table(kv_lens, P, max(1, max(W.pages_for(L, P) for L in kv_lens)), n, gc)
    k = random_pool(n, H_kv, P, D, seed + 1, device)
    v = random_pool(n, H_kv, P, D, seed + 2, device)
    if poison:
        poison_pool(k, pt, kv_lens)
        poison_pool(v, pt, kv_lens)
    T = sum(q_lens)
    q = (torch.randn((T, H_q, D), generator=gc) * q_std).to(torch.bfloat16)
    rel = torch.randn((T, H_q, R), generator=gc) * 0.5
    cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
    return W.PrefillInputs(q=q.to(device), cu_seqlens_q=cu.to(device), k_cache=k, v_cache=v, page_table=pt.to(device),
                           seq_lens=torch.tensor(kv_lens, dtype=torch.int32, device=device),
                           rel_logits=rel.to(device), window=window, scale=D ** -0.5, max_seq_len=max(kv_lens + [1]),
                           max_q_len=max(q_lens + [0]))


def reference(inp, q=None, rel=None):
    """(out, lse, |V|-weighted out) in float64.  A sequence with fewer keys than queries: no key visible."""
    cu = inp.cu_seqlens_q.cpu().numpy().astype(np.int64)
    sl = inp.seq_lens.cpu().numpy().astype(np.int64)
    q = f64(inp.q) if q is None else q
    rel = f64(inp.rel_logits) if rel is None else rel
    kc, vc = read_pool(inp.k_cache.cpu().numpy(), False), read_pool(inp.v_cache.cpu().numpy(), True)
    pt = inp.page_table.cpu().numpy()
    keep = [b for b in range(len(sl)) if cu[b + 1] - cu[b] <= sl[b]]
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in keep]) if keep else np.zeros(0, dtype=np.int64)
    sub = np.concatenate([[0], np.cumsum([cu[b + 1] - cu[b] for b in keep])]).astype(np.int64)
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    size = np.zeros(q.shape)
    a = (q[rows], sub, kc)
    b = (pt[keep], sl[keep], rel[rows], inp.window, inp.scale)
    out[rows], lse[rows] = ref_prefill(*a, vc, *b)
    size[rows], _ = ref_prefill(*a, np.abs(vc), *b)
    return out, lse, size


def score_error(inp):
    """Bound on the absolute error of a score [T, H_q, 1].
    fp32: a score is a sum of products q u s less 8 q s, terms of magnitude up to 23 |q| s, each addition off by at
    most 2^-23 of the largest partial sum (the matrix unit cuts rather than rounds), 4 additions of 32-term sums
    per group: 4 * 2^-23 * 23 * S_MAX * sum|q|."""
    return 4 * 2.0 ** -23 * 23 * S_MAX * abs(inp.scale) * np.abs(f64(inp.q)).sum(-1, keepdims=True)


def check(inp, out, lse, ref=None, what=""):
    """bf16 outputs: P is rounded to bf16 (2^-8 of every weight) and the result again (2^-8), and a score error
    e changes a weight by a factor within 1 + 2e (its own and the sum's); hardware exponentials and fp32 sums are
    worth 2^-20.  The logarithm of the sum moves by e; fp32 holds it to 2^-22 of itself.
    The products with V are P s u less 8 P s, summed apart: partial sums of at most 15 S_MAX and 8 S_MAX (P sums to
    1), each addition cut at 2^-23 of one, two per 16-key block; and 2^-23 of the sum so far, at most ``size``, for
    each of as many additions."""
    ro, rl, size = reference(inp) if ref is None else ref
    e = score_error(inp)
    g, gl = f64(out), f64(lse)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    blocks = inp.max_seq_len / 16 + 2
    tol = 2.0 ** -8 * (np.abs(ro) + size) * (1 + 2.0 ** -7) + (2 * e + 2.0 ** -20) * size
    tol += 2 * blocks * 2.0 ** -23 * (23 * S_MAX + size)
    bad = np.abs(g - ro) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(g - ro) / tol).max():.2f} of the bound"
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(gl), fin) and np.all(gl[~fin] == -np.inf), f"{what}: lse finiteness"
    le = np.abs(gl - rl)[fin] - (e[..., 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl))[fin]
    assert le.size == 0 or le.max() <= 0, f"{what}: lse off by {le.max():.2e} past its bound"
