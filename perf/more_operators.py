"""The 8-bit key/value cache and shared pages: cases, plain forms and 64-bit values.

A case names one operator (``op``):

* ``append``   new K/V rows quantised into the paged 8-bit cache by slot, and the rows read back as
               the values they now stand for, each new row and the first row of its block
* ``decode``   attention with the relative-position bias over the 8-bit cache, ``q_len`` new tokens
               per sequence
* ``prefill``  the same for a chunk of new tokens per sequence
* ``fork``     requests that go on from another request's tokens: its full pages are shared, its last
               partial page is copied in every pool
* ``retire``   a wave of requests ends: pages without an owner go back on the free stack, and the
               live pages are moved together, in the tables and in every pool

The 8-bit format.  The tokens of a (page, KV head) come in blocks of 16, and a block has one scale
2^e: e is the smallest integer from -60 to 55 with max |v| <= 448 * 2^e over its rows (larger
magnitudes count as 448 * 2^55).  A value is stored as e4m3 of v / 2^e, rounded to nearest even.  Rows
that join a block raise e where they need to, and the rows that are there are rounded again from the
values they stand for; rows at place 0 begin the block anew.  A row with a NaN reads as NaN.
The pool is uint8 [num_pages, H_kv, page_size, D + 1]; a block is 16 rows of D bytes, the fp32 scale,
16 bits that mark rows with a NaN, and 10 zero bytes.  Channel c of row r of a block is at byte
  K, D = 128:  128 r + 16 (c / 16 ^ 4 (r % 2)) + c % 16          K, D = 64:  64 r + c
  V, D = 128:  128 r + 16 (c / 16 ^ 2 (r / 2 % 4)) + c % 16
  V, D = 64:   128 (r / 2) + 8 (4 (2 (r % 2) + c / 32 ^ r / 2 % 4) + c / 8 % 4) + c % 8

Pages.  page_refs counts a page's owners beyond the first; free_pages is a stack of free_count pages.
"""

from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
EMIN, EMAX = -60, 55


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the append of a decode step, 8 KV heads (global layer): one token joins a block that is begun
        dict(name="append_decode", op="append", T=128, runs=128, H_kv=8, D=128, P=64),
        # one chunk of 2048 tokens of 4 sequences, 16 KV heads (local layer), from inside a block on
        dict(name="append_chunk", op="append", T=8192, runs=4, H_kv=16, D=128, P=64),
        # two short sequences, small pages: what counts is latency
        dict(name="decode_tiny", op="decode", B=2, q_len=1, H_q=4, H_kv=2, D=64, P=16, window=32, R=32, lo=37, hi=100),
        # the local layer's decode batch: window of 512 keys, 16 KV heads
        dict(name="decode_local", op="decode", B=64, q_len=1, H_q=48, H_kv=16, D=128, P=64, window=512, R=512,
             lo=1024, hi=8192),
        # the global layer's: full causal, lengths up to 32768, 8 KV heads
        dict(name="decode_global", op="decode", B=32, q_len=1, H_q=48, H_kv=8, D=128, P=64, window=0, R=1024,
             lo=4096, hi=32768),
        # verification of 4 draft tokens per sequence, local layer
        dict(name="decode_draft", op="decode", B=64, q_len=4, H_q=48, H_kv=16, D=128, P=64, window=512, R=512,
             lo=1024, hi=8192),
        # a short ragged chunk: odd sizes, head size 64, small pages
        dict(name="prefill_ragged", op="prefill", B=3, chunk=257, H_q=6, H_kv=3, D=64, P=16, window=100, R=128,
             lo=300, hi=900),
        # the local layer's chunk: 4 sequences x 2048 new tokens behind a cached prefix
        dict(name="prefill_local", op="prefill", B=4, chunk=2048, H_q=48, H_kv=16, D=128, P=64, window=512, R=512,
             lo=4096, hi=8192),
        # 3 more samples of one prompt, one layer, small pages: latency
        dict(name="fork_samples", op="fork", parents=1, children=3, idle=4, layers=1, H_kv=2, D=64, P=16, lo=90, hi=120),
        # 8 samples of each of 16 prompts, 4 layers of a bf16 cache
        dict(name="fork_prompts", op="fork", parents=16, children=8, idle=0, layers=4, H_kv=8, D=128, P=64, lo=1024,
             hi=4096),
        # 3 of 11 requests end, small pages, one layer
        dict(name="retire_few", op="retire", B=11, ended=3, shared=4, layers=1, H_kv=2, D=64, P=16, lo=20, hi=300,
             spare=9),
        # a third of a full decode batch ends; samples of common prompts among them, 2 layers of a bf16 cache
        dict(name="retire_batch", op="retire", B=128, ended=42, shared=64, layers=2, H_kv=8, D=128, P=64, lo=512,
             hi=4096, spare=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "fork", "retire"])
    P = rng.choice([16, 32, 48, 64, 128])
    D = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 3, 5, 8, 16])
    if op == "append":
        T = _log(rng, 1, 8000)
        return dict(op=op, T=T, runs=rng.choice([T, _log(rng, 1, T)]), H_kv=H_kv, D=D, P=P)
    if op == "fork":
        lo = _log(rng, 1, 3000)
        return dict(op=op, parents=_log(rng, 1, 12), children=_log(rng, 1, 8), idle=rng.randint(0, 9),
                    layers=rng.randint(1, 3), H_kv=H_kv, D=D, P=P, lo=lo, hi=lo + rng.randint(0, 1000))
    if op == "retire":
        B = _log(rng, 2, 96)
        lo = _log(rng, 1, 1500)
        return dict(op=op, B=B, ended=rng.randint(1, B), shared=rng.randint(0, B), layers=rng.randint(1, 2),
                    H_kv=min(H_kv, 8), D=D, P=P, lo=lo, hi=lo + rng.randint(0, 1500), spare=_log(rng, 1, 300))
    G = rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g * H_kv <= 64])
    H_q = H_kv * G
    window = rng.choice([0, _log(rng, 1, 2048)])
    R = 4 * _log(rng, 1, 256)
    if op == "decode":
        hi = _log(rng, 8, 20000)
        most = max(1, 250000 * 8 // (hi * H_kv))  # at most about half of the largest listed case's keys
        return dict(op=op, B=min(_log(rng, 1, 96), most), q_len=rng.choice([1, 1, 1, 2, 3, 5, 8]), H_q=H_q, H_kv=H_kv,
                    D=D, P=P, window=window, R=R, lo=max(8, hi // 3), hi=hi)
    chunk = _log(rng, 1, 1500)
    hi = chunk + _log(rng, 1, 4000)
    most = max(1, 48 * 2048 * 8192 // (3 * H_q * chunk * hi))
    return dict(op=op, B=min(rng.randint(1, 4), most), chunk=chunk, H_q=H_q, H_kv=H_kv, D=D, P=P, window=window, R=R,
                lo=chunk, hi=hi)


# ------------------------------------------------------------------ inputs

def _gens(seed):
    c = torch.Generator()
    c.manual_seed(seed)
    d = torch.Generator(device=DEV)
    d.manual_seed(seed + 1)
    return c, d


def _ints(lo, hi, n, gen):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _random_rows(shape, gen, spread=0.4):
    """bf16 rows [..., D]; tokens differ in size, as keys and values do."""
    size = torch.exp(spread * torch.randn(shape[:-1], generator=gen, device=DEV)).unsqueeze(-1)
    return (torch.randn(shape, generator=gen, device=DEV) * size).to(BF16)


def _random_pool(num_pages, H_kv, P, D, gen, is_v):
    """A pool whose every row holds quantised values."""
    pool = torch.empty((num_pages, H_kv, P, D + 1), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (H_kv * P * D))
    for a in range(0, num_pages, step):
        n = min(step, num_pages - a)
        rows = _random_rows((n * H_kv * P // 16, 16, D), gen)
        _blocks(pool[a:a + n]).copy_(_block_bytes(*quantise(rows.float(), None), is_v))
    return pool


def _cache(case, lens, seed):
    """Pools, page table and generators of decode and prefill cases: random placement in a shuffled pool."""
    c, d = _gens(seed)
    P, B = case["P"], case["B"]
    n = (lens + P - 1) // P
    pool = int(n.sum()) + 3
    pages = torch.randperm(pool, generator=c)[:int(n.sum())].to(torch.int32)
    table = torch.zeros((B, int(n.max())), dtype=torch.int32)
    table[torch.arange(table.shape[1])[None, :] < n[:, None]] = pages
    k = _random_pool(pool, case["H_kv"], P, case["D"], d, False)
    v = _random_pool(pool, case["H_kv"], P, case["D"], d, True)
    return k, v, table.to(DEV), d


def _int_state(s, **parts):
    """The step's whole numbers in one buffer, with views by name, and a copy of how they are before the step."""
    s["before"] = torch.cat([t.flatten().to(torch.int32) for t in parts.values()]).to(DEV)
    s["now"] = s["before"].clone()
    at = 0
    for name, t in parts.items():
        s[name] = s["now"][at:at + t.numel()].view(t.shape)
        at += t.numel()


def _bf16_pools(case, n, gen):
    shape = (n, case["P"], case["H_kv"], case["D"])
    return [torch.randn(shape, generator=gen, device=DEV, dtype=BF16) for _ in range(2 * case["layers"])]


def prepare(case, seed):
    c, d = _gens(seed)
    s = dict(case=case)
    op, P = case["op"], case["P"]
    if op == "append":
        T, H, D = case["T"], case["H_kv"], case["D"]
        runs = min(case["runs"], T)
        # a run of tokens for each sequence: consecutive places from anywhere in its pages on
        cut = torch.sort(torch.randperm(T - 1, generator=c)[:runs - 1] + 1).values if runs > 1 else _ints(0, 0, 0, c)
        first = torch.cat([torch.zeros(1, dtype=torch.int64), cut])
        count = torch.diff(torch.cat([first, torch.tensor([T])]))
        offset = _ints(0, P - 1, runs, c)
        need = (offset + count + P - 1) // P
        base = torch.cumsum(need, 0) - need
        n = int(need.sum()) + 2
        pages = torch.randperm(n, generator=c)
        run = torch.repeat_interleave(torch.arange(runs), count)
        at = offset[run] + torch.arange(T) - first[run]
        slots = pages[base[run] + at // P] * P + at % P
        s.update(k_new=_random_rows((T, H, D), d, 1.0), v_new=_random_rows((T, H, D), d, 1.0), slots=slots.to(DEV),
                 read=torch.cat([slots, slots // 16 * 16]).to(DEV), k=_random_pool(n, H, P, D, d, False),
                 v=_random_pool(n, H, P, D, d, True), k_back=torch.empty((2 * T, H, D), dtype=BF16, device=DEV),
                 v_back=torch.empty((2 * T, H, D), dtype=BF16, device=DEV))
        return s
    if op == "fork":
        lens = torch.cat([_ints(case["lo"], case["hi"], case["parents"], c),
                          torch.zeros(case["parents"] * case["children"] + case["idle"], dtype=torch.int64)])
        source = torch.full_like(lens, -1)
        kids = case["parents"] * case["children"]
        source[case["parents"]:case["parents"] + kids] = torch.arange(case["parents"]).repeat_interleave(case["children"])
        order = torch.randperm(lens.numel(), generator=c)  # rows in any order
        place = torch.empty_like(order)
        place[order] = torch.arange(lens.numel())
        lens, source = lens[order], source[order]
        source = torch.where(source >= 0, place[source.clamp(min=0)], -1)
        n = (lens + P - 1) // P
        stride = case["hi"] // P + 2
        spare = kids + 5
        pool = case["parents"] * ((case["hi"] + P - 1) // P) + spare  # (pages that are left over are nobody's)
        perm = torch.randperm(pool, generator=c)
        table = torch.zeros((lens.numel(), stride), dtype=torch.int64)
        table[torch.arange(stride)[None, :] < n[:, None]] = perm[spare:spare + int(n.sum())]
        free = torch.zeros(pool, dtype=torch.int64)
        free[:spare] = perm[:spare]
        _int_state(s, table=table, refs=torch.zeros(pool), free=free, count=torch.tensor([spare]), lens=lens,
                   source=source)
        s.update(kv_lens=torch.empty_like(s["lens"]), src=torch.empty_like(s["lens"]), dst=torch.empty_like(s["lens"]),
                 left=torch.empty_like(s["count"]), pools=_bf16_pools(case, pool, d))
        return s
    if op == "retire":
        B = case["B"]
        lens = _ints(case["lo"], case["hi"], B, c)
        n = (lens + P - 1) // P
        stride = (case["hi"] + P - 1) // P
        total = int(n.sum())
        pool = B * stride + case["spare"]  # (pages that are left over are nobody's)
        perm = torch.randperm(pool, generator=c)
        table = torch.zeros((B, stride), dtype=torch.int64)
        table[torch.arange(stride)[None, :] < n[:, None]] = perm[:total]
        # the last requests but one are samples of an earlier one: they share its full pages, as far as both have them
        refs = torch.zeros(pool, dtype=torch.int64)
        lost = []
        for b in range(B - min(case["shared"], B - 1), B):
            p = int(_ints(0, max(0, B - case["shared"] - 1), 1, c))
            k = int(min(lens[p], lens[b])) // P
            lost.append(table[b, :k].clone())
            table[b, :k] = table[p, :k]
            refs[table[p, :k]] += 1
        spare = torch.cat([perm[total:total + case["spare"]]] + lost)
        spare = spare[torch.randperm(spare.numel(), generator=c)]
        free = torch.zeros(pool, dtype=torch.int64)
        free[:spare.numel()] = spare
        new = torch.ones(B, dtype=torch.int64)
        new[torch.randperm(B, generator=c)[:case["ended"]]] = -1
        _int_state(s, table=table, refs=refs, free=free, count=torch.tensor([spare.numel()]), lens=lens, new=new)
        s.update(src=torch.empty_like(s["free"]), dst=torch.empty_like(s["free"]), moves=torch.empty_like(s["count"]),
                 pools=_bf16_pools(case, pool, d))
        return s
    lens = _ints(case["lo"], case["hi"], case["B"], c)
    lens[0] = case["hi"]  # the bound is met
    k, v, table, d = _cache(case, lens, seed)
    s.update(k=k, v=v, table=table, lens=lens.to(torch.int32).to(DEV), scale=case["D"] ** -0.5)
    if op == "decode":
        T = case["B"] * case["q_len"]
    else:
        # some sequences get a whole chunk, the last one a shorter one
        q = torch.full((case["B"],), case["chunk"], dtype=torch.int64)
        if case["B"] > 2:
            q[-1] = max(1, case["chunk"] // 3)
        cu = torch.zeros(case["B"] + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(q, 0)
        T = int(cu[-1])
        s.update(cu=cu.to(DEV))
    s["q"] = torch.randn((T, case["H_q"], case["D"]), generator=d, device=DEV).to(BF16)
    s["rel"] = torch.randn((T, case["H_q"], case["R"]), generator=d, device=DEV) * 0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, case["H_q"]), dtype=torch.float32, device=DEV)
    s["ws"] = {}  # the workspace a program keeps, made by the first pass
    return s


# ------------------------------------------------------------------ the format, plainly

def _offsets(D, is_v, device):
    """[16, D]: byte of channel c of row r in its block."""
    r = torch.arange(16, device=device)[:, None]
    c = torch.arange(D, device=device)[None, :]
    if D == 64 and not is_v:
        return 64 * r + c
    if D == 64:
        return 128 * (r // 2) + 8 * (4 * ((2 * (r % 2) + c // 32) ^ (r // 2 % 4)) + c // 8 % 4) + c % 8
    return 128 * r + 16 * ((c // 16) ^ (2 * (r // 2 % 4) if is_v else 4 * (r % 2))) + c % 16


def _blocks(pool):
    """A pool's blocks [pages * H * P / 16, 16 (D + 1)]."""
    return pool.view(-1, 16 * pool.shape[3])


def quantise(rows, floor):
    """(bytes [n, 16, D], exponent [n], NaN rows [n, 16]) of blocks of fp32 rows [n, 16, D]; the exponent is
    at least ``floor`` [n], where that is given.  v / 2^e is exact in 32 bits or far below the smallest step."""
    bad = torch.isnan(rows).any(-1)
    rows = torch.where(bad.unsqueeze(-1), 0.0, rows).clamp(-448.0 * 2.0 ** EMAX, 448.0 * 2.0 ** EMAX)
    mant, ex = torch.frexp(rows.abs().amax((1, 2)))  # mant in [0.5, 1), 448 = 0.875 * 2^9
    e = (ex - 9 + (mant > 0.875)).clamp(EMIN, EMAX)
    if floor is not None:
        e = torch.maximum(e, floor)
    return torch.ldexp(rows, -e[:, None, None]).to(E4M3), e, bad


def _block_bytes(data, e, bad, is_v):
    """Blocks [n, 16 (D + 1)] of quantised rows."""
    n, _, D = data.shape
    out = torch.zeros((n, 16 * (D + 1)), dtype=torch.uint8, device=data.device)
    out[:, _offsets(D, is_v, data.device).flatten()] = data.view(torch.uint8).flatten(1)
    out[:, 16 * D:16 * D + 4] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[:, None].view(torch.uint8)
    bits = (bad.to(torch.int32) << torch.arange(16, device=data.device, dtype=torch.int32)).sum(-1)
    out[:, 16 * D + 4] = (bits & 255).to(torch.uint8)
    out[:, 16 * D + 5] = (bits >> 8).to(torch.uint8)
    return out


def _open(blocks, is_v):
    """(values [n, 16, D] fp32, exponent [n], NaN rows [n, 16]) of blocks [n, 16 (D + 1)]."""
    n, D = blocks.shape[0], blocks.shape[1] // 16 - 1
    x = blocks[:, _offsets(D, is_v, blocks.device).flatten()].view(E4M3).float().view(n, 16, D)
    s = blocks[:, 16 * D:16 * D + 4].contiguous().view(torch.float32)
    bits = blocks[:, 16 * D + 4].to(torch.int32) | blocks[:, 16 * D + 5].to(torch.int32) << 8
    bad = (bits[:, None] >> torch.arange(16, device=blocks.device, dtype=torch.int32)) & 1 > 0
    e = torch.frexp(s[:, 0]).exponent - 1
    return torch.where(bad.unsqueeze(-1), math.nan, x * s.unsqueeze(-1)), e, bad


def _block_ids(slots, H, P):
    """[T, H]: block of the slot for each head."""
    page, place = slots // P, slots % P
    return (page[:, None] * H + torch.arange(H, device=slots.device)) * (P // 16) + (place // 16)[:, None]


def _rows_at(pool, slots, is_v):
    """fp32 rows [..., H, D] at the slots (page * P + place)."""
    n, H, P, nb = pool.shape
    D = nb - 1
    flat = pool.view(-1)
    at = _block_ids(slots.flatten(), H, P) * (16 * nb)
    off = _offsets(D, is_v, pool.device)[slots.flatten() % 16]
    x = flat[at[:, :, None] + off[:, None, :]].view(E4M3).float()
    word = torch.arange(4, device=pool.device)
    s = flat[at[:, :, None] + 16 * D + word].view(torch.float32)
    nan = flat[at + 16 * D + 4 + (slots.flatten() % 16 // 8)[:, None]]
    bad = (nan.to(torch.int64) >> (slots.flatten() % 8)[:, None]) & 1 > 0
    return torch.where(bad.unsqueeze(-1), math.nan, x * s).view(*slots.shape, H, D)


# ------------------------------------------------------------------ plain forms

def _append_into(rows, pool, slots, is_v):
    H, P, D = pool.shape[1], pool.shape[2], pool.shape[3] - 1
    ids = _block_ids(slots, H, P)                              # the tokens of a block come next to each other
    _, group = torch.unique_consecutive(ids[:, 0], return_inverse=True)
    n = int(group[-1]) + 1
    first = torch.full((n,), 16, device=DEV).scatter_reduce(0, group, slots % 16, "amin")
    which = torch.zeros((n, H), dtype=torch.int64, device=DEV)
    which[group] = ids
    blocks = _blocks(pool)[which.flatten()]
    old, e_old, bad = _open(blocks, is_v)
    new = old.view(n, H, 16, D).clone()
    new[group, :, slots % 16] = rows.float()
    joins = torch.zeros((n, 16), dtype=torch.bool, device=DEV)
    joins[group, slots % 16] = True
    joins = joins[:, None, :].expand(n, H, 16).reshape(-1, 16)
    begun = (first > 0)[:, None].expand(n, H).flatten()
    # the exponent that the joining rows ask for, and that the block has
    mine = torch.where(joins.unsqueeze(-1), new.view(-1, 16, D), 0.0)
    floor = torch.where(begun, e_old, EMIN)
    data, e, nan_new = quantise(mine, floor)
    there = torch.ldexp(torch.where(bad.unsqueeze(-1), 0.0, old), -e[:, None, None])
    there = torch.where(begun[:, None, None], there, 0.0).clamp(-448.0, 448.0).to(E4M3)
    data = torch.where(joins.unsqueeze(-1), data.view(torch.uint8), there.view(torch.uint8)).view(E4M3)
    bad = torch.where(joins, nan_new, bad & begun[:, None])
    _blocks(pool)[which.flatten()] = _block_bytes(data, e, bad, is_v)


def _plain_append(s):
    _append_into(s["k_new"], s["k"], s["slots"], False)
    _append_into(s["v_new"], s["v"], s["slots"], True)
    return [_rows_at(s["k"], s["read"], False).to(BF16), _rows_at(s["v"], s["read"], True).to(BF16)]


def _attend(s, q, qpos, qvalid, lens, first, n, rel):
    """q [B, Q, H_q, D] at positions qpos [B, Q] over the n keys from ``first`` [B] on."""
    case = s["case"]
    B, Q, H_q, D = q.shape
    H, P, R = case["H_kv"], case["P"], case["R"]
    j = first[:, None] + torch.arange(n, device=q.device)
    there = j < lens[:, None]
    jj = torch.where(there, j, 0)
    slots = torch.gather(s["table"].long(), 1, jj // P) * P + jj % P
    k = _rows_at(s["k"], slots, False).permute(0, 2, 3, 1)  # [B, H, D, n]
    qh = q.float().view(B, Q, H, H_q // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    sc = torch.matmul(qh, k).view(B, H_q, Q, n)
    del k
    dist = qpos[:, :, None] - j[:, None, :]
    see = there[:, None, :] & (dist >= 0) & qvalid[:, :, None]
    if case["window"] > 0:
        see = see & (dist < case["window"])
    at = dist.clamp(0, R - 1)[:, None].expand(B, H_q, Q, n)
    sc = sc * s["scale"] + torch.gather(rel.permute(0, 2, 1, 3), 3, at)
    sc = sc.masked_fill(~see[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    e = torch.exp(sc - m)
    z = e.sum(-1, keepdim=True)
    lse = (m + torch.log(z))[..., 0].transpose(1, 2)
    v = _rows_at(s["v"], slots, True).permute(0, 2, 1, 3)  # [B, H, n, D]
    o = torch.matmul(e.view(B, H, -1, n), v).view(B, H_q, Q, D) / torch.where(z > 0, z, 1.0)
    return o.transpose(1, 2), lse


def _plain_attention(s):
    case = s["case"]
    B, W = case["B"], case["window"]
    lens = s["lens"].long()
    if case["op"] == "decode":
        Q = case["q_len"]
        cu = torch.arange(B + 1, device=DEV) * Q
    else:
        Q, cu = case["chunk"], s["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=DEV)
    valid = i[None, :] < count[:, None]
    row = torch.where(valid, cu[:-1, None] + i[None, :], 0)
    qpos = lens[:, None] - count[:, None] + i[None, :]
    n = case["hi"] if W <= 0 else min(case["hi"], W - 1 + Q)
    first = torch.clamp(lens - n, min=0)
    o, lse = _attend(s, s["q"][row], qpos, valid, lens, first, n, s["rel"][row])
    # rows of the batch that hold no query are left out; the others come in packed order
    return o[valid].to(BF16), lse[valid]


def _plain_fork(s):
    P, stride, count = s["case"]["P"], s["table"].shape[1], s["count"].long()
    lens, source = s["lens"].long(), s["source"].long()
    child = source >= 0
    parent = source.clamp(min=0)
    n = torch.where(child, lens[parent], 0)
    full = n // P
    need = n % P > 0
    rank = torch.cumsum(need, 0) - need.long()
    served = child & (~need | (rank < count))
    page = s["free"][(count - 1 - rank).clamp(min=0)]
    col = torch.arange(stride, device=DEV)
    shares = served[:, None] & (col < full[:, None])
    table = torch.where(shares, s["table"][parent], s["table"])
    takes = served & need
    table = torch.where((col == full[:, None]) & takes[:, None], page[:, None], table)
    refs = s["refs"].index_add(0, table[shares].long(), torch.ones_like(table[shares]))
    src = torch.where(takes, s["table"][parent, full.clamp(max=stride - 1)], -1)
    dst = torch.where(takes, page, -1)
    for pool in s["pools"]:
        pool[dst[takes].long()] = pool[src[takes].long()]
    kv = torch.where(child, torch.where(served, n, 0), lens).int()
    return dict(table=table, refs=refs, kv_lens=kv, src=src, dst=dst, left=(count - takes.sum()).int(),
                pools=s["pools"])


def _plain_retire(s):
    P, stride, n_pages = s["case"]["P"], s["table"].shape[1], s["free"].numel()
    lens, ended = s["lens"].long(), s["new"] < 0
    count = s["count"].long()
    col = torch.arange(stride, device=DEV)
    held = col < ((lens + P - 1) // P)[:, None]
    table = s["table"].long()
    # ---- pages come back: in row order, a page that several of the rows held at the last of them
    gone = held & ended[:, None]
    page, at = table[gone], torch.nonzero(gone.flatten()).flatten()
    refs = s["refs"].long().index_add(0, page, torch.full_like(page, -1))
    last = torch.full((n_pages,), -1, device=DEV).scatter_reduce(0, page, at, "amax")
    back = (refs[page] < 0) & (last[page] == at)
    refs = refs.clamp(min=0)
    free = torch.cat([s["free"].long(), torch.zeros_like(page)])
    place = count + torch.cumsum(back, 0) - 1
    free[place[back]] = page[back]
    height = count + back.sum()
    lens = torch.where(ended, 0, lens)
    # ---- live pages move to the lowest places
    held = held & ~ended[:, None]
    live = torch.zeros(n_pages, dtype=torch.bool, device=DEV)
    live[table[held]] = True
    spare = torch.zeros_like(live)
    spare[free[:int(height)]] = True
    rank = torch.cumsum(live | spare, 0) - 1
    src = torch.nonzero(live & (rank >= live.sum())).flatten()
    dst = torch.nonzero(spare & (rank < live.sum())).flatten()
    to = torch.arange(n_pages, device=DEV)
    to[src] = dst
    table = torch.where(held, to[table], table)
    refs[dst] = refs[src]
    refs[src] = 0
    left = torch.nonzero((live | spare) & (rank >= live.sum())).flatten()
    free = s["free"].long().clone()
    free[:left.numel()] = left.flip(0)
    for pool in s["pools"]:
        pool[dst] = pool[src]
    pad = torch.full((n_pages - src.numel(),), -1, dtype=torch.int64, device=DEV)
    return dict(table=table.int(), refs=refs.int(), lens=lens.int(), free=free.int(), count=height.int(),
                src=torch.cat([src, pad]).int(), dst=torch.cat([dst, pad]).int(),
                moves=torch.tensor([src.numel()], dtype=torch.int32, device=DEV), pools=s["pools"])


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "fork":
            s["now"].copy_(s["before"])
            return _plain_fork(s)
        if op == "retire":
            s["now"].copy_(s["before"])
            return _plain_retire(s)
        return _plain_attention(s)
    import paged_attention_relative_attn_gb300 as ira
    case = s["case"]
    if op == "append":
        ira.kv_append_q8(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
        return list(ira.kv_read_q8(s["read"], s["k"], s["v"], k_rows=s["k_back"], v_rows=s["v_back"]))
    if op == "fork":
        s["now"].copy_(s["before"])  # the state of another step
        kv, src, dst, left = ira.fork_pages(s["source"], s["lens"], s["table"], s["refs"], s["free"], s["count"],
                                            page_size=case["P"], kv_lens=s["kv_lens"], copy_src=s["src"],
                                            copy_dst=s["dst"], free_left=s["left"])
        ira.copy_pages(s["pools"], src, dst)
        return dict(table=s["table"], refs=s["refs"], kv_lens=kv, src=src, dst=dst, left=left, pools=s["pools"])
    if op == "retire":
        s["now"].copy_(s["before"])  # the state of another step
        ira.release_pages(s["lens"], s["new"], s["table"], s["refs"], s["free"], s["count"], page_size=case["P"],
                          kv_lens=s["lens"], free_left=s["count"])
        src, dst, moves = ira.compact_pages(s["lens"], s["table"], s["free"], s["count"], page_size=case["P"],
                                            page_refs=s["refs"], move_src=s["src"], move_dst=s["dst"],
                                            moves=s["moves"])
        ira.copy_pages(s["pools"], src, dst, count=moves)
        return dict(table=s["table"], refs=s["refs"], lens=s["lens"], free=s["free"], count=s["count"],
                    src=src, dst=dst, moves=moves, pools=s["pools"])
    if op == "decode":
        if "t" not in s["ws"]:
            need = ira.decode_q8_workspace_bytes(case["B"], case["q_len"], case["H_q"], case["H_kv"], case["D"])
            s["ws"]["t"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return ira.decode_q8(s["q"], s["k"], s["v"], s["table"], s["lens"], s["rel"], q_len=case["q_len"],
                             window=case["window"], scale=s["scale"], out=s["out"], lse=s["lse"],
                             workspace=s["ws"]["t"])
    if "t" not in s["ws"]:
        need = ira.prefill_q8_workspace_bytes(case["B"], case["chunk"], case["H_kv"], case["D"], case["window"],
                                              case["hi"])
        s["ws"]["t"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return ira.prefill_q8(s["q"], s["cu"], s["k"], s["v"], s["table"], s["lens"], s["rel"], window=case["window"],
                          scale=s["scale"], max_seq_len=case["hi"], max_q_len=case["chunk"], out=s["out"],
                          lse=s["lse"], workspace=s["ws"]["t"])


# ------------------------------------------------------------------ work

def work(case):
    op, D, H, P = case["op"], case["D"], case["H_kv"], case["P"]
    if op == "append":
        rows = 2 * case["T"] * H  # K and V; a row read and written once, and two read back
        return {"bytes": rows * (3 * 2 * D + 3 * D) + 24 * case["T"], "flops": rows * 3 * D}
    if op in ("fork", "retire"):
        page = 2 * case["layers"] * P * H * D * 2  # of all pools
        mean = (case["lo"] + case["hi"]) / 2 / P
        if op == "fork":
            kids = case["parents"] * case["children"]
            return {"bytes": kids * (2 * page + 16 * mean + 24), "flops": 0}
        live = (case["B"] - case["ended"]) * mean * (1 - 0.25 * case["shared"] / case["B"])
        spare = case["spare"] + case["ended"] * mean
        moved = live * spare / (live + spare)
        return {"bytes": moved * 2 * page + 12 * (live + spare) + 8 * case["B"] * mean, "flops": 0}
    W, R, H_q = case["window"], case["R"], case["H_q"]
    mean = (case["lo"] + case["hi"]) / 2
    if op == "decode":
        T, chunks = case["B"] * case["q_len"], case["q_len"]
    else:
        chunks = case["chunk"]
        T = case["B"] * chunks if case["B"] <= 2 else (case["B"] - 1) * chunks + max(1, chunks // 3)
    keys = min(mean, W - 1 + chunks) if W > 0 else mean  # keys read for a sequence
    past = max(0.0, mean - chunks)
    # visible keys of a query, and the bias entries it takes, over the chunk's positions
    pos = [past + (i + 0.5) * chunks / 64 for i in range(64)]
    vis = sum(min(p + 0.5, W) if W > 0 else p + 0.5 for p in pos) / 64
    bias = sum(min(min(p + 0.5, W) if W > 0 else p + 0.5, R) for p in pos) / 64
    return {"bytes": case["B"] * keys * 2 * H * (D + 0.25) + T * H_q * (4 * D + 4 + 4 * bias) + 4 * case["B"] * keys / P,
            "flops": 4 * D * H_q * T * vis}


# ------------------------------------------------------------------ 64 bits

def _exact_block(pool, which, is_v):
    """(float64 [n, 16, D], float64 scale [n]) of blocks, from their bytes' bit fields; NaN rows as they are marked."""
    D = pool.shape[3] - 1
    raw = pool.reshape(-1, 16 * (D + 1))[which].to(torch.int64)
    rows = []
    for r in range(16):
        c = torch.arange(D, device=pool.device)
        if is_v and D == 64:
            at = (r - r % 2) * 64 + ((c // 32 + 2 * (r % 2)) ^ ((r >> 1) & 3)) * 32 + c % 32
        elif is_v:
            at = r * 128 + (c ^ (((r >> 1) & 3) << 5))
        elif D == 128:
            at = r * 128 + (c ^ ((r & 1) << 6))
        else:
            at = r * D + c
        rows.append(raw[:, at])
    b = torch.stack(rows, 1)
    sign = 1.0 - 2.0 * (b >> 7).double()
    ex, man = (b >> 3) & 15, (b & 7).double()
    x = sign * torch.where(ex > 0, torch.exp2((ex - 7).double()) * (1 + man / 8), man * 2.0 ** -9)
    bits = raw[:, 16 * D] | raw[:, 16 * D + 1] << 8 | raw[:, 16 * D + 2] << 16 | raw[:, 16 * D + 3] << 24
    s = torch.exp2((bits >> 23).double() - 127)  # scales are powers of two
    flags = raw[:, 16 * D + 4] + 256 * raw[:, 16 * D + 5]
    for r in range(16):
        x[:, r] = torch.where(((flags >> r) & 1 == 1)[:, None], math.nan, x[:, r] * s[:, None])
    return x, s


def _e4m3_64(x):
    """x to the nearest number with 4 significant bits, at least 2^-9 apart, ties to even."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6) - 3)
    return torch.round(x / step) * step  # (a power of two whose logarithm is one off: the same number)


def _exact_append(rows, pool, slots, read, is_v):
    H, P, D = pool.shape[1], pool.shape[2], pool.shape[3] - 1
    T = slots.numel()
    # block of a token (a number for each page and 16 places), its tokens' places, its largest new magnitude
    number, group = torch.unique(slots // 16, return_inverse=True)
    page, sub = number // (P // 16), number % (P // 16)
    which = ((page[:, None] * H + torch.arange(H, device=DEV)) * (P // 16) + sub[:, None]).flatten()
    old, s_old = _exact_block(pool, which, is_v)
    old, s_old = old.view(-1, H, 16, D), s_old.view(-1, H)
    n = number.numel()
    v = rows.double()
    big = torch.zeros((n, H), dtype=torch.float64, device=DEV)
    big.scatter_reduce_(0, group[:, None].expand(T, H), v.abs().amax(-1), "amax")
    e = torch.full((n, H), float(EMIN), dtype=torch.float64, device=DEV)
    for k in range(EMIN, EMAX):  # counted up until the block's largest magnitude fits
        e = torch.where(big > 448.0 * 2.0 ** k, float(k + 1), e)
    fresh = torch.ones(n, dtype=torch.int64, device=DEV).scatter_reduce_(0, group, slots % 16, "amin") == 0
    s = torch.exp2(e)
    s = torch.where(fresh[:, None], s, torch.maximum(s, s_old))
    out = torch.where(fresh[:, None, None, None], 0.0, _e4m3_64(old / s[:, :, None, None]) * s[:, :, None, None])
    out[group, :, slots % 16] = _e4m3_64(v / s[group].unsqueeze(-1)) * s[group].unsqueeze(-1)
    return out[torch.cat([group, group]), :, read % 16]


def _exact_sequence(s, b, H, P, a, e, is_v):
    pool = s["v"] if is_v else s["k"]
    parts = []
    for lo in range(a // 16 * 16, e, 2048):
        j = torch.arange(lo, min(e, lo + 2048), 16, device=DEV)
        which = (s["table"][b].long()[j // P, None] * H + torch.arange(H, device=DEV)) * (P // 16) + (j % P // 16)[:, None]
        x, _ = _exact_block(pool, which.flatten(), is_v)
        parts.append(x.view(-1, H, 16, x.shape[-1]).transpose(1, 2).flatten(0, 1))
    return torch.cat(parts)[a % 16:a % 16 + e - a]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return [_exact_append(s["k_new"], s["k"], s["slots"], s["read"], False),
                _exact_append(s["v_new"], s["v"], s["slots"], s["read"], True)]
    if op in ("fork", "retire"):
        # whole numbers, and pools of which every page is another's or its own: the requests one after the other
        P, table, lens = case["P"], s["table"].tolist(), s["lens"].tolist()
        free = s["free"].tolist()[:int(s["count"])]
        pairs = []
        if op == "fork":
            for p in s["source"].tolist():
                if p >= 0 and lens[p] % P:
                    pairs.append((table[p][lens[p] // P], free.pop()))
            keys = ("table", "refs", "kv_lens", "src", "dst", "left")
        else:
            refs, kept = s["refs"].tolist(), set()
            for row, L, new in zip(table, lens, s["new"].tolist()):
                for page in row[:-(-L // P)]:
                    if new >= 0:
                        kept.add(page)
                    elif refs[page] == 0:
                        free.append(page)
                    else:
                        refs[page] -= 1
            known = sorted(kept | set(free))
            low = known[:len(kept)]
            pairs = list(zip([x for x in known[len(kept):] if x in kept], [x for x in low if x not in kept]))
            keys = ("table", "refs", "lens", "free", "count", "src", "dst", "moves")
        src, dst = (torch.tensor([p[i] for p in pairs], dtype=torch.int64, device=DEV) for i in (0, 1))
        out = {k: None for k in keys}
        out["pools"] = [p.double().index_copy(0, dst, p[src].double()) for p in s["pools"]]
        return out
    H, H_q, P, W, R = (case[x] for x in ("H_kv", "H_q", "P", "window", "R"))
    G = H_q // H
    lens = s["lens"].tolist()
    cu = [b * case["q_len"] for b in range(case["B"] + 1)] if op == "decode" else s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        Q = cu[b + 1] - cu[b]
        a0 = max(0, L - Q - W + 1) if W > 0 else 0
        K = _exact_sequence(s, b, H, P, a0, L, False)
        V = _exact_sequence(s, b, H, P, a0, L, True)
        for i in range(0, Q, 512):
            n = min(512, Q - i)
            p = torch.arange(L - Q + i, L - Q + i + n, device=DEV)
            a = max(a0, int(L - Q + i - W + 1)) if W > 0 else 0
            e = L - Q + i + n
            dist = p[:, None] - torch.arange(a, e, device=DEV)[None, :]
            hidden = dist < 0 if W <= 0 else (dist < 0) | (dist >= W)
            at = dist.clamp(0, R - 1)
            rows = slice(cu[b] + i, cu[b] + i + n)
            for h in range(H_q):
                sc = s["q"][rows, h].double() @ K[a - a0:e - a0, h // G].T * s["scale"]
                sc = sc + torch.gather(s["rel"][rows, h].double(), 1, at)
                sc = sc.masked_fill(hidden, -math.inf)
                l = torch.logsumexp(sc, 1)
                lse[rows, h] = l
                out[rows, h] = torch.exp(sc - l[:, None]) @ V[a - a0:e - a0, h // G]
    return out, lse
