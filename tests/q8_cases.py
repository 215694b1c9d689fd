"""Inputs and bounds shared by the tests of the 8-bit cache."""

from __future__ import annotations

import numpy as np
import torch

import workloads as W
from oracle.q8 import read_pool
from oracle.ref import ref_prefill
from tests.helpers import f64

SPREAD = 3  # block exponents of random_pool: EXP - SPREAD .. EXP
EXP = -7    # the largest magnitude of its values: 448 * 2^-7 = 3.5


def random_pool(n, H, P, D, seed, device, spread=SPREAD, exp=EXP):
    """A pool of random bytes (every finite e4m3 number alike) and exponents exp - spread .. exp; no quantiser is
    involved."""
    g = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 254, (n, H, P // 16, 16 * D), generator=g)
    data = (data + (data >= 127).long()).to(torch.uint8)  # without 0x7f, 0xff
    e = exp - torch.randint(0, spread + 1, (n, H, P // 16, 1), generator=g)
    tail = torch.zeros((n, H, P // 16, 16), dtype=torch.uint8)
    tail[..., :4] = torch.exp2(e.float()).view(torch.uint8)
    return torch.cat([data, tail], -1).reshape(n, H, P, D + 1).to(device)


def dead_places(pool, pt, lens):
    """[n, P / 16, 16] bool: places that hold no token of the sequences."""
    n, H, P, row = pool.shape
    dead = torch.ones((n, P), dtype=torch.bool)
    for b, L in enumerate(lens):
        for j in range(L):
            dead[int(pt[b, j // P]), j % P] = False
    return dead.view(n, P // 16, 16)


def poison_pool(pool, pt, lens, is_v):
    """Every byte of places that hold no token becomes 0xff (NaN); so do the tails of blocks without one."""
    from oracle.q8 import places
    n, H, P, row = pool.shape
    D = row - 1
    blocks = pool.view(n, H, P // 16, 16 * row)
    dead = dead_places(pool, pt, lens).to(pool.device)
    at = torch.from_numpy(places(D, is_v)).to(pool.device)
    data = blocks[..., at]  # [n, H, P / 16, 16, D]
    blocks[..., at] = torch.where(dead[:, None, :, :, None], torch.full_like(data, 255), data)
    none = dead.all(-1)[:, None, :, None]
    blocks[..., 16 * D:] = torch.where(none, torch.full_like(blocks[..., 16 * D:], 255), blocks[..., 16 * D:])


def make(q_lens, kv_lens, H_q, H_kv, D, P, window, R, seed, device="cuda", q_std=1.0, poison=True, extra=2, **pool):
    """A PrefillInputs whose caches are 8-bit pools; decode of equal q_lens takes the same inputs."""
    gc = torch.Generator().manual_seed(seed)
    n = sum(W.pages_for(L, P) for L in kv_lens) + extra
    pt, _ = W.build_page_table(kv_lens, P, max(1, max(W.pages_for(L, P) for L in kv_lens)), n, gc)
    k = random_pool(n, H_kv, P, D, seed + 1, device, **pool)
    v = random_pool(n, H_kv, P, D, seed + 2, device, **pool)
    if poison:
        poison_pool(k, pt, kv_lens, False)
        poison_pool(v, pt, kv_lens, True)
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


def largest(pool):
    """Largest magnitude among the values of blocks with a scale in the cache's range."""
    row = pool.shape[3]
    s = pool.view(-1, 16 * row)[:, 16 * (row - 1):][:, :4].contiguous().cpu().view(torch.float32)
    s = s[torch.isfinite(s)]
    return 448.0 * float(s.max()) if s.numel() else 0.0


def score_error(inp):
    """Bound on the absolute error of a score [T, H_q, 1].
    Products of e4m3 and fp16 numbers are exact in fp32; D / 16 additions of 16-term sums per score, each off by at
    most 2^-23 of the largest partial sum (the matrix unit cuts rather than rounds), which is at most
    max|k| sum|q|; one rounding more for the factor and one for the bias; what q loses as fp16 is 2^-39 of its row's
    largest for each of D channels."""
    D = inp.q.shape[2]
    q = np.abs(f64(inp.q))
    k = largest(inp.k_cache)
    return abs(inp.scale) * k * ((D / 16 + 2) * 2.0 ** -23 * q.sum(-1, keepdims=True)
                                 + D * 2.0 ** -39 * q.max(-1, keepdims=True))


F16, BF16 = 2.0 ** -11, 2.0 ** -8  # half a step of a rounding, relative to the value


def check(inp, out, lse, ref=None, what="", p_step=F16):
    """bf16 outputs: P is rounded to fp16 (decode) or bf16 (prefill) and the result to bf16, and a score error e
    changes a weight by a factor within 1 + 2e (its own and the sum's); hardware exponentials and fp32 sums are worth
    2^-20.  A weight below fp16's range loses at most 2^-32 of the largest times 448 times the largest scale, for
    each key.  Products with V: each addition is cut at 2^-23 of the partial sum, one per 16-key block.
    The logarithm of the sum moves by e; fp32 holds it to 2^-22 of itself."""
    ro, rl, size = reference(inp) if ref is None else ref
    e = score_error(inp)
    g, gl = f64(out), f64(lse)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    keys = inp.max_seq_len if inp.window <= 0 else min(inp.max_seq_len, inp.window + inp.max_q_len)
    blocks = keys / 16 + 2
    tol = BF16 * np.abs(ro) + (1 + BF16) * (p_step + 2 * e + 2.0 ** -20 + blocks * 2.0 ** -23) * size
    tol += keys * 2.0 ** -32 * largest(inp.v_cache)
    bad = np.abs(g - ro) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(g - ro) / tol).max():.2f} of the bound"
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(gl), fin) and np.all(gl[~fin] == -np.inf), f"{what}: lse finiteness"
    le = np.abs(gl - rl)[fin] - (e[..., 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl))[fin]
    assert le.size == 0 or le.max() <= 0, f"{what}: lse off by {le.max():.2e} past its bound"
