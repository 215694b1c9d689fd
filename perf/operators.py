"""The 4-bit key/value cache and the step tables: cases, plain forms and 64-bit values.

A case names one operator (``op``):

* ``tables``   the tables of a serving step, built from request lengths: lengths
               after the step, cu_seqlens, page-table entries, the slot of each new token
* ``append``   new K/V rows quantised into the paged 4-bit cache by slot, and the
               rows read back as the values they now stand for
* ``decode``   attention with the relative-position bias over the 4-bit cache,
               ``q_len`` new tokens per sequence
* ``prefill``  the same for a chunk of new tokens per sequence

The 4-bit format.  A row is the D channels of one token and KV head, in groups
of 32 adjacent channels.  A group's scale s is its largest magnitude over 7,
rounded up to 5 significant bits; a value is x * s with x = v / s rounded to the
nearest integer, ties toward zero (|x| <= 7, so x * s is a bf16 number).
The pool is uint8 [num_pages, H_kv, page_size, 9 * D / 16]: within one (page,
head) the tokens are in blocks of 16, a block being 16 rows of D / 2 bytes
(nibble = x + 8) and then 16 rows of D / 32 bf16 scales.  With N = D / 32 groups
j: 32-bit word N * t + j of a K row holds channels 32 j + 8 t + 0..7, 16-bit unit
N * g + j of a V row holds channels 32 j + 4 g + 0..3, lowest nibble first.
"""

from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # every request of a full decode batch takes one token; a few have ended, a few page
        # boundaries are crossed: the tables of one step of the 128-sequence decode stack
        dict(name="tables_decode", op="tables", B=128, P=64, mean_len=2048, n_new=1, n_long=0, ended=4,
             max_len=8192, max_tokens=128),
        # a mixed step: 4 prompts get a chunk of 2048 tokens while 252 requests decode
        dict(name="tables_mixed", op="tables", B=256, P=64, mean_len=2048, n_new=1, n_long=4, ended=16,
             max_len=8192, max_tokens=16384),
        # the append of a decode step, 8 KV heads (global layer)
        dict(name="append_decode", op="append", T=128, H_kv=8, D=128, P=64),
        # an odd number of tokens, head size 64, small pages
        dict(name="append_odd", op="append", T=1001, H_kv=3, D=64, P=16),
        # one chunk of 2048 tokens of 4 sequences, 16 KV heads (local layer)
        dict(name="append_chunk", op="append", T=8192, H_kv=16, D=128, P=64),
        # two short sequences, small pages: what counts is latency
        dict(name="decode_tiny", op="decode", B=2, q_len=1, H_q=4, H_kv=2, D=64, P=16, window=32, R=32,
             lo=37, hi=100),
        # the local layer's decode batch: window of 512 keys, 16 KV heads
        dict(name="decode_local", op="decode", B=64, q_len=1, H_q=48, H_kv=16, D=128, P=64, window=512,
             R=512, lo=1024, hi=8192),
        # the global layer's: full causal, lengths up to 32768, 8 KV heads
        dict(name="decode_global", op="decode", B=32, q_len=1, H_q=48, H_kv=8, D=128, P=64, window=0,
             R=1024, lo=4096, hi=32768),
        # verification of 4 draft tokens per sequence, local layer
        dict(name="decode_draft", op="decode", B=64, q_len=4, H_q=48, H_kv=16, D=128, P=64, window=512,
             R=512, lo=1024, hi=8192),
        # a short ragged chunk: odd sizes, head size 64, small pages
        dict(name="prefill_ragged", op="prefill", B=3, chunk=257, H_q=6, H_kv=3, D=64, P=16, window=100,
             R=128, lo=300, hi=900),
        # the local layer's chunk: 4 sequences x 2048 new tokens behind a cached prefix
        dict(name="prefill_local", op="prefill", B=4, chunk=2048, H_q=48, H_kv=16, D=128, P=64, window=512,
             R=512, lo=4096, hi=8192),
        # the global layer's chunk: every key of the prefix is visible
        dict(name="prefill_global", op="prefill", B=2, chunk=2048, H_q=48, H_kv=8, D=128, P=64, window=0,
             R=1024, lo=6000, hi=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "prefill", "prefill"])
    P = rng.choice([16, 32, 48, 64, 128])
    if op == "tables":
        B = _log(rng, 1, 512)
        n_long = rng.randint(0, min(B, 4))
        return dict(op=op, B=B, P=P, mean_len=_log(rng, 8, 3000), n_new=rng.choice([1, 1, 2, 5]), n_long=n_long,
                    ended=rng.randint(0, B // 8), max_len=8192, max_tokens=8 * B + 2048 * n_long)
    D = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 3, 5, 8, 16])
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 8000), H_kv=H_kv, D=D, P=P)
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
    hi = chunk + _log(rng, 1, 5000)
    most = max(1, 48 * 2048 * 8192 * 2 // (3 * H_q * chunk * hi))  # at most a third of the largest listed case's scores
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


def _pages(n_pages, extra, gen):
    """Random physical placement: the pages of all sequences in a shuffled pool."""
    return torch.randperm(n_pages + extra, generator=gen)[:n_pages].to(torch.int32)


def _random_rows(n, D, gen):
    return torch.randn((n, D), generator=gen, device=DEV).to(BF16)


def _random_pool(num_pages, H_kv, P, D, gen, is_v):
    """A pool whose every row holds quantised N(0, 1) values."""
    pool = torch.empty((num_pages, H_kv, P, 9 * D // 16), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (H_kv * P * D))
    for a in range(0, num_pages, step):
        n = min(step, num_pages - a)
        rows = _random_rows(n * H_kv * P, D, gen).view(n, H_kv, P, D)
        x, s = quantise(rows)
        data, scales = _views(pool[a:a + n])
        data.copy_(pack(x, is_v).view(n, H_kv, P // 16, 16, D // 2))
        scales.copy_(s.to(BF16).view(n, H_kv, P // 16, 16, D // 32))
    return pool


def _lens(case, gen):
    lens = _ints(case["lo"], case["hi"], case["B"], gen)
    lens[0] = case["hi"]  # the bound is met
    return lens


def _cache(case, lens, seed):
    """Pools, page table and bias width shared by decode and prefill cases."""
    c, d = _gens(seed)
    P, B = case["P"], case["B"]
    n = (lens + P - 1) // P
    pages = _pages(int(n.sum()), 3, c)
    table = torch.zeros((B, int(n.max())), dtype=torch.int32)
    table[torch.arange(table.shape[1])[None, :] < n[:, None]] = pages
    pool = int(n.sum()) + 3
    k = _random_pool(pool, case["H_kv"], P, case["D"], d, False)
    v = _random_pool(pool, case["H_kv"], P, case["D"], d, True)
    return k, v, table.to(DEV), d


def prepare(case, seed):
    c, d = _gens(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "tables":
        B, P = case["B"], case["P"]
        lens = (torch.rand(B, generator=c) * 2 * case["mean_len"]).to(torch.int64).clamp(0, case["max_len"] - 2100)
        new = torch.full((B,), case["n_new"], dtype=torch.int64)
        who = torch.randperm(B, generator=c)
        new[who[:case["n_long"]]] = 2048
        new[who[case["n_long"]:case["n_long"] + case["ended"]]] = -1
        stride = (case["max_len"] + P - 1) // P
        n = (lens + P - 1) // P
        spare = int(((new.clamp(min=0) + P - 1) // P + 1).sum())
        perm = torch.randperm(int(n.sum()) + spare, generator=c).to(torch.int32)
        table = torch.zeros((B, stride), dtype=torch.int32)
        table[torch.arange(stride)[None, :] < n[:, None]] = perm[:int(n.sum())]
        free = torch.zeros(perm.numel(), dtype=torch.int32)
        free[:spare] = perm[int(n.sum()):]
        s.update(seq_lens=lens.to(torch.int32).to(DEV), new_lens=new.to(torch.int32).to(DEV), table=table.to(DEV),
                 free=free.to(DEV), count=torch.tensor([spare], dtype=torch.int32, device=DEV),
                 kv_lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                 cu=torch.zeros(B + 1, dtype=torch.int32, device=DEV),
                 slots=torch.zeros(case["max_tokens"], dtype=torch.int64, device=DEV),
                 left=torch.zeros(1, dtype=torch.int32, device=DEV))
    elif op == "append":
        T, H, D, P = case["T"], case["H_kv"], case["D"], case["P"]
        n = (T + P - 1) // P + 2
        # runs of tokens of some sequences: consecutive slots of shuffled pages
        pages = torch.randperm(n, generator=c)
        at = torch.arange(T) + int(_ints(0, P - 1, 1, c))
        slots = pages[at // P] * P + at % P
        s.update(k_new=_random_rows(T * H, D, d).view(T, H, D), v_new=_random_rows(T * H, D, d).view(T, H, D),
                 slots=slots.to(DEV), k=torch.zeros((n, H, P, 9 * D // 16), dtype=torch.uint8, device=DEV),
                 v=torch.zeros((n, H, P, 9 * D // 16), dtype=torch.uint8, device=DEV),
                 k_back=torch.empty((T, H, D), dtype=BF16, device=DEV),
                 v_back=torch.empty((T, H, D), dtype=BF16, device=DEV))
    else:
        lens = _lens(case, c)
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
            s.update(cu=cu.to(DEV), chunk=case["chunk"])
        s["q"] = torch.randn((T, case["H_q"], case["D"]), generator=d, device=DEV).to(BF16)
        s["rel"] = torch.randn((T, case["H_q"], case["R"]), generator=d, device=DEV) * 0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, case["H_q"]), dtype=torch.float32, device=DEV)
        s["ws"] = {}  # the workspace a program keeps, made by the first pass
    return s


# ------------------------------------------------------------------ the format, plainly

def _order(D, is_v, device):
    """Channel held at each nibble position of a row."""
    n, p = D // 32, torch.arange(D, device=device)
    w = 4 if is_v else 8
    unit, c = p // w, p % w
    return 32 * (unit % n) + w * (unit // n) + c


def quantise(rows):
    """(x, s) of bf16 rows [..., D]: integers [..., D] and scales [..., D / 32].
    32 bits decide as 64 would: a value is 8 significant bits and a scale 5, so
    no quotient lies nearer than 2^-12 to a border unless it is on it, and then the
    division is exact."""
    f = rows.float().unflatten(-1, (-1, 32))
    a = f.abs().amax(-1)
    mant, ex = torch.frexp(a / torch.full_like(a, 7.0))  # by a tensor: a true division, not a product with 1/7
    s = torch.ldexp(torch.ceil(mant * 32) / 32, ex)
    t = f / torch.where(s > 0, s, 1.0).unsqueeze(-1)
    x = torch.sign(t) * torch.ceil(t.abs() - 0.5)
    return x.flatten(-2).to(torch.int16), s


def pack(x, is_v):
    u = (x + 8).to(torch.uint8)[..., _order(x.shape[-1], is_v, x.device)]
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _views(pool):
    """Nibble rows [pages, H, blocks, 16, D / 2] and bf16 scales [pages, H, blocks, 16, D / 32] of a pool."""
    n, H, P, nb = pool.shape
    D = nb * 16 // 9
    b = pool.view(n, H, P // 16, 9 * D)
    return (b[..., :8 * D].unflatten(-1, (16, D // 2)),
            b[..., 8 * D:].view(BF16).unflatten(-1, (16, D // 32)))


def unpack(data, scales, is_v):
    """fp32 values [..., D] of nibble rows [..., D / 2] and scales [..., D / 32]."""
    D = data.shape[-1] * 2
    u = torch.stack((data & 15, data >> 4), -1).flatten(-2)
    x = torch.empty(u.shape, dtype=torch.float32, device=u.device)
    x[..., _order(D, is_v, u.device)] = u.float() - 8
    return (x.unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)


def _rows_at(pool, slots, is_v):
    """fp32 rows [..., H, D] at the slots (page * P + place)."""
    P = pool.shape[2]
    page, place = slots // P, slots % P
    data, scales = _views(pool)
    data, scales = data.permute(0, 2, 3, 1, 4), scales.permute(0, 2, 3, 1, 4)
    at = (page, place // 16, place % 16)
    return unpack(data[at], scales[at], is_v)


# ------------------------------------------------------------------ plain forms

def _plain_tables(s):
    P, stride = s["case"]["P"], s["table"].shape[1]
    L, new = s["seq_lens"].long(), s["new_lens"].long()
    F = s["count"].long()
    n = new.clamp(min=0)
    had = (L + P - 1) // P
    # requests that have ended give their pages back, in batch and page order, above the stack's top
    gone = torch.where(new < 0, had, 0)
    col = torch.arange(stride, device=L.device)
    back = torch.cumsum(gone, 0) - gone
    free = s["free"].clone()
    live = col[None, :] < gone[:, None]
    at = (F + back[:, None] + col[None, :])
    free = free.index_put((at[live],), s["table"][live])
    top = F + gone.sum()
    # the others take pages from the top, in the same order
    need = torch.where(new >= 0, (L + n + P - 1) // P - had, 0)
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= top)
    first = upto - need
    table = s["table"].clone()
    rank = first[:, None] + col[None, :] - had[:, None]
    takes = served[:, None] & (col[None, :] >= had[:, None]) & (col[None, :] < (had + need)[:, None])
    table = torch.where(takes, free[(top - 1 - rank).clamp(0, free.numel() - 1)], table)
    used = torch.where(served, need, 0).sum()
    kv = torch.where(new < 0, 0, torch.where(served, L + n, L))
    cu = torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])
    t = torch.arange(s["slots"].numel(), device=L.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    in_range = t < cu[-1]
    b = b.clamp(max=L.numel() - 1)
    pos = L[b] + t - cu[b]
    slot = table[b, (pos // P).clamp(max=stride - 1)].long() * P + pos % P
    slots = torch.where(in_range & served[b], slot, -1)
    return dict(kv_lens=kv.int(), cu=cu.int(), slots=slots, table=table, free_left=(top - used).int())


def _plain_append(s):
    H, D, P = s["case"]["H_kv"], s["case"]["D"], s["case"]["P"]
    back = []
    for rows, pool, is_v in ((s["k_new"], s["k"], False), (s["v_new"], s["v"], True)):
        x, sc = quantise(rows)
        data, scales = (t.permute(0, 2, 3, 1, 4) for t in _views(pool))
        at = (s["slots"] // P, s["slots"] % P // 16, s["slots"] % 16)
        data[at] = pack(x, is_v)
        scales[at] = sc.to(BF16)
        back.append(_rows_at(pool, s["slots"], is_v).to(BF16))
    return back


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


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "tables":
            return _plain_tables(s)
        return _plain_append(s) if op == "append" else _plain_attention(s)
    import paged_attention_relative_attn_gb300 as ira
    case = s["case"]
    if op == "tables":
        kv, cu, slots, left = ira.build_tables(s["seq_lens"], s["new_lens"], s["table"], s["free"], s["count"],
                                               page_size=case["P"], kv_lens=s["kv_lens"], cu_seqlens_q=s["cu"],
                                               slot_map=s["slots"], free_left=s["left"])
        return dict(kv_lens=kv, cu=cu, slots=slots, table=s["table"], free_left=left)
    if op == "append":
        ira.kv_append_q4(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
        return list(ira.kv_read_q4(s["slots"], s["k"], s["v"], k_rows=s["k_back"], v_rows=s["v_back"]))
    if op == "decode":
        if "t" not in s["ws"]:
            need = ira.decode_q4_workspace_bytes(case["B"], case["q_len"], case["H_q"], case["H_kv"], case["D"])
            s["ws"]["t"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return ira.decode_q4(s["q"], s["k"], s["v"], s["table"], s["lens"], s["rel"], q_len=case["q_len"],
                             window=case["window"], scale=s["scale"], out=s["out"], lse=s["lse"],
                             workspace=s["ws"]["t"])
    if "t" not in s["ws"]:
        need = ira.prefill_q4_workspace_bytes(case["B"], case["chunk"], case["H_kv"], case["D"], case["window"],
                                              case["hi"])
        s["ws"]["t"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return ira.prefill_q4(s["q"], s["cu"], s["k"], s["v"], s["table"], s["lens"], s["rel"], window=case["window"],
                          scale=s["scale"], max_seq_len=case["hi"], max_q_len=case["chunk"], out=s["out"],
                          lse=s["lse"], workspace=s["ws"]["t"])


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "tables":
        # lengths in and out, one table entry per request, popped or returned pages, one slot per token
        pages = case["n_long"] * 2048 // case["P"] + case["ended"] * case["mean_len"] // case["P"]
        return {"bytes": case["B"] * 20 + 8 * pages + 8 * case["max_tokens"], "flops": 0}
    D, H = case["D"], case["H_kv"]
    row = 9 * D // 16
    if op == "append":
        rows = 2 * case["T"] * H
        return {"bytes": rows * 2 * (2 * D + row) + 16 * case["T"], "flops": rows * 4 * D}
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
    return {"bytes": case["B"] * keys * 2 * H * row + T * H_q * (4 * D + 4 + 4 * bias) + 4 * case["B"] * keys / case["P"],
            "flops": 4 * D * H_q * T * vis}


# ------------------------------------------------------------------ 64 bits

def _exact_row(pool, H, page, place, is_v):
    """float64 [n, H, D] of rows (page[i], place[i]), read byte by byte from the pool."""
    n_pages, _, P, nb = pool.shape
    D = nb * 16 // 9
    N = D // 32
    flat = pool.reshape(n_pages, H, P * nb)[page]                       # [n, H, P * nb]
    ch = torch.arange(D, device=pool.device)
    j, r = ch // 32, ch % 32
    if is_v:
        nib = 4 * (N * (r // 4) + j) + r % 4
    else:
        nib = 8 * (N * (r // 8) + j) + r % 8
    base = (place // 16 * (9 * D))[:, None, None]
    at = base + (place % 16 * (D // 2))[:, None, None] + (nib // 2)[None, None, :]
    byte = torch.gather(flat, 2, at.expand(-1, H, -1)).to(torch.int64)
    x = ((byte >> (4 * (nib % 2))) & 15) - 8
    at = base + 8 * D + (place % 16 * (D // 16))[:, None, None] + (2 * j)[None, None, :]
    lo = torch.gather(flat, 2, at.expand(-1, H, -1)).to(torch.int64)
    hi = torch.gather(flat, 2, (at + 1).expand(-1, H, -1)).to(torch.int64)
    bits = lo | (hi << 8)
    ex, man = (bits >> 7) & 255, bits & 127
    s = torch.ldexp((128 + man).double(), (ex - 134).to(torch.int64))   # scales are normal numbers or 0
    return x.double() * torch.where(bits == 0, 0.0, s)


def _exact_sequence(s, b, H, P, a, e, is_v):
    pool = s["v"] if is_v else s["k"]
    parts = []
    for lo in range(a, e, 2048):
        j = torch.arange(lo, min(e, lo + 2048), device=DEV)
        parts.append(_exact_row(pool, H, s["table"][b].long()[j // P], j % P, is_v))
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    if op == "append":
        outs = []
        for rows in (s["k_new"], s["v_new"]):
            v = rows.double().view(*rows.shape[:2], -1, 32)
            a = v.abs().amax(-1, keepdim=True)
            # s = i * 2^(e - 4), 16 <= i <= 32: the smallest such number with 7 s >= a (at a power of two
            # an exponent one off gives the same number)
            e = torch.floor(torch.log2(a / torch.full_like(a, 7.0)))
            step = torch.exp2(e - 4)
            sc = torch.ceil(a / (7 * step)) * step
            x = torch.zeros_like(v)
            for level in range(7):  # |v| past the border between level and level + 1 (a tie stays below)
                x += (v.abs() > (level + 0.5) * sc).double()
            outs.append((torch.sign(v) * x * sc).view(rows.shape))
        return outs
    H, H_q, P, W, R, D = (case[x] for x in ("H_kv", "H_q", "P", "window", "R", "D"))
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
