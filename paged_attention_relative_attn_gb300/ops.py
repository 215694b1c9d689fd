"""PyTorch-facing wrappers: shape/dtype checks, default output buffers, the
current stream, then one call into the C ABI.  All arithmetic happens in the
CUDA kernels of libinkling_rel_attn.so; there is no CPU or PyTorch fallback.
"""

from __future__ import annotations

import torch

from . import _lib


class InklingError(RuntimeError):
    """A non-zero INKLING_* status from the C ABI."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_lib.inkling_rel_attn_error_string(code)} (code {code})")


def _check(rc: int, where: str):
    if rc != 0:
        raise InklingError(rc, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _need(t, name, dtype, dims):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def choose_splits(B, H_kv, window, max_seq_len, num_sms=0):
    return _lib.inkling_rel_attn_choose_splits(B, H_kv, window, max_seq_len, num_sms)


def decode_workspace_bytes(B, H_q, H_kv, D, window, max_seq_len, num_splits=0, num_sms=0):
    return _lib.inkling_rel_attn_decode_workspace_size(B, H_q, H_kv, D, window, max_seq_len,
                                                       num_splits, num_sms)


def decode(q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, window, scale,
           max_seq_len, out=None, lse=None, workspace=None, num_splits=0,
           device_error=None, stream=None):
    """Decode attention (one query per sequence).  See inkling_rel_attn_decode.

    q [B, H_q, D] bf16; k_cache, v_cache [num_pages, page_size, H_kv, D] bf16;
    page_table [B, stride] int32; seq_lens [B] int32; rel_logits [B, H_q, R] fp32.
    Returns (out bf16 [B, H_q, D], lse fp32 [B, H_q]).  Pass ``out``, ``lse`` and
    ``workspace`` to avoid allocations (required under CUDA-graph capture).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(rel_logits, "rel_logits", torch.float32, 3)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    B, H_q, D = q.shape
    num_pages, P, H_kv, Dk = k_cache.shape
    R = rel_logits.shape[2]
    if Dk != D or rel_logits.shape[:2] != (B, H_q) or seq_lens.shape[0] != B or page_table.shape[0] != B:
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    ws_need = decode_workspace_bytes(B, H_q, H_kv, D, window, max_seq_len, num_splits)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.inkling_rel_attn_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
        _ptr(seq_lens), _ptr(rel_logits), B, H_q, H_kv, D, P, num_pages, R, window,
        float(scale), max_seq_len, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        num_splits, _ptr(device_error), _stream(q.device, stream))
    _check(rc, "inkling_rel_attn_decode")
    return out, lse


def decode_multi_workspace_bytes(B, q_len, H_q, H_kv, D, window, max_seq_len, num_splits=0,
                                 num_sms=0):
    return _lib.inkling_rel_attn_decode_multi_workspace_size(B, q_len, H_q, H_kv, D, window,
                                                             max_seq_len, num_splits, num_sms)


def decode_multi(q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, q_len, window, scale,
                 max_seq_len, out=None, lse=None, workspace=None, num_splits=0,
                 device_error=None, stream=None):
    """Decode of ``q_len`` new tokens per sequence (the last q_len of each).
    See inkling_rel_attn_decode_multi.

    q [B * q_len, H_q, D] bf16 (row b * q_len + i); rel_logits [B * q_len, H_q, R]
    fp32; other tensors as ``decode``.  Returns (out [B * q_len, H_q, D] bf16,
    lse [B * q_len, H_q] fp32).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(rel_logits, "rel_logits", torch.float32, 3)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    T, H_q, D = q.shape
    B = seq_lens.shape[0]
    num_pages, P, H_kv, Dk = k_cache.shape
    R = rel_logits.shape[2]
    if (Dk != D or T != B * q_len or rel_logits.shape[:2] != (T, H_q)
            or page_table.shape[0] != B):
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((T, H_q), dtype=torch.float32, device=q.device)
    ws_need = decode_multi_workspace_bytes(B, q_len, H_q, H_kv, D, window, max_seq_len, num_splits)
    if workspace is None and ws_need > 0:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.inkling_rel_attn_decode_multi(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
        _ptr(seq_lens), _ptr(rel_logits), B, q_len, H_q, H_kv, D, P, num_pages, R, window,
        float(scale), max_seq_len, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        num_splits, _ptr(device_error), _stream(q.device, stream))
    _check(rc, "inkling_rel_attn_decode_multi")
    return out, lse


def prefill(q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, window,
            scale, max_seq_len, max_q_len, out=None, lse=None, device_error=None, stream=None):
    """Chunked / paged prefill.  See inkling_rel_attn_prefill.

    q [T, H_q, D] bf16; cu_seqlens_q [B+1] int32; rel_logits [T, H_q, R] fp32.
    Returns (out bf16 [T, H_q, D], lse fp32 [T, H_q]).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(rel_logits, "rel_logits", torch.float32, 3)
    T, H_q, D = q.shape
    num_pages, P, H_kv, _ = k_cache.shape
    B = seq_lens.shape[0]
    R = rel_logits.shape[2]
    if cu_seqlens_q.shape[0] != B + 1 or rel_logits.shape[:2] != (T, H_q):
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((T, H_q), dtype=torch.float32, device=q.device)
    rc = _lib.inkling_rel_attn_prefill(
        _ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
        page_table.shape[1], _ptr(seq_lens), _ptr(rel_logits), B, T, max_q_len, H_q, H_kv, D, P,
        num_pages, R, window, float(scale), max_seq_len, _ptr(out), _ptr(lse), None, 0,
        _ptr(device_error), _stream(q.device, stream))
    _check(rc, "inkling_rel_attn_prefill")
    return out, lse


def kv_append(k_new, v_new, cu_seqlens_q, seq_lens, page_table, k_cache, v_cache, *,
              device_error=None, stream=None):
    """Write the new tokens' K/V into the paged cache (in place).  See
    inkling_rel_attn_kv_append.

    k_new, v_new [T, H_kv, D] bf16; cu_seqlens_q [B+1] int32; seq_lens [B]
    int32 (totals including the new tokens); page_table [B, stride] int32;
    k_cache, v_cache [num_pages, page_size, H_kv, D] bf16, updated in place.
    """
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    T, H_kv, D = k_new.shape
    num_pages, P, H_kv_c, D_c = k_cache.shape
    B = seq_lens.shape[0]
    if (v_new.shape != k_new.shape or v_cache.shape != k_cache.shape or (H_kv_c, D_c) != (H_kv, D)
            or cu_seqlens_q.shape[0] != B + 1 or page_table.shape[0] != B):
        raise ValueError("inconsistent shapes")
    rc = _lib.inkling_rel_attn_kv_append(
        _ptr(k_new), _ptr(v_new), _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(page_table),
        page_table.shape[1], B, T, H_kv, D, P, num_pages, _ptr(k_cache), _ptr(v_cache),
        _ptr(device_error), _stream(k_new.device, stream))
    _check(rc, "inkling_rel_attn_kv_append")


def kv_conv_append(k_new, v_new, cu_seqlens_q, seq_lens, page_table, k_cache, v_cache,
                   conv_w_k, conv_w_v, conv_state_k, conv_state_v, state_slots, *,
                   max_q_len, device_error=None, stream=None):
    """The causal short convolutions on K and V of the new tokens, then the
    append of the convolved rows into the paged cache; the state pool rows of
    the sequences are rewritten in place.  See inkling_rel_attn_kv_conv_append.

    k_new, v_new [T, H_kv, D] bf16; conv_w_k, conv_w_v [H_kv, D, width] fp32;
    conv_state_k, conv_state_v [num_slots, width - 1, H_kv, D] bf16 (width 1:
    None); state_slots [B] int32; the rest as for ``kv_append``.  max_q_len is
    a host bound on any sequence's new tokens.
    """
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(conv_w_k, "conv_w_k", torch.float32, 3)
    _need(conv_w_v, "conv_w_v", torch.float32, 3)
    T, H_kv, D = k_new.shape
    num_pages, P, H_kv_c, D_c = k_cache.shape
    B = seq_lens.shape[0]
    width = conv_w_k.shape[2]
    if (v_new.shape != k_new.shape or v_cache.shape != k_cache.shape or (H_kv_c, D_c) != (H_kv, D)
            or cu_seqlens_q.shape[0] != B + 1 or page_table.shape[0] != B
            or tuple(conv_w_k.shape) != (H_kv, D, width) or conv_w_v.shape != conv_w_k.shape):
        raise ValueError("inconsistent shapes")
    num_slots = 0
    if width > 1:
        _need(conv_state_k, "conv_state_k", torch.bfloat16, 4)
        _need(conv_state_v, "conv_state_v", torch.bfloat16, 4)
        _need(state_slots, "state_slots", torch.int32, 1)
        num_slots = conv_state_k.shape[0]
        if (tuple(conv_state_k.shape) != (num_slots, width - 1, H_kv, D)
                or conv_state_v.shape != conv_state_k.shape or state_slots.shape[0] != B):
            raise ValueError("inconsistent state shapes")
    rc = _lib.inkling_rel_attn_kv_conv_append(
        _ptr(k_new), _ptr(v_new), _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(page_table),
        page_table.shape[1], _ptr(conv_w_k), _ptr(conv_w_v), width, _ptr(conv_state_k),
        _ptr(conv_state_v), _ptr(state_slots), num_slots, B, T, int(max_q_len), H_kv, D, P,
        num_pages, _ptr(k_cache), _ptr(v_cache), _ptr(device_error), _stream(k_new.device, stream))
    _check(rc, "inkling_rel_attn_kv_conv_append")


# ---------------------------------------------------------------------------
# Step tables, and the caches held in 4 and in 8 bits
# ---------------------------------------------------------------------------

# A decode step calls several of these with a few microseconds of GPU work each, so their
# checks are one expression per call; what fails it is named by _refuse.

_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _refuse(dev, specs):
    """Raise for the first (tensor, name, dtype, dims) that is not a contiguous tensor of that type and rank
    on device ``dev``; shapes that do not go together if each is."""
    for t, name, dtype, dims in specs:
        if t.dtype is not dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
        if t.dim() != dims:
            raise ValueError(f"{name}: expected {dims} dims, got shape {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{name}: on {t.device}, not on the other tensors' device")
    raise ValueError("inconsistent shapes")


def _launch(name, dev, stream, *args):
    """One call into the C ABI on device ``dev`` (made current for it) and the given or current stream, its
    arguments packed (converting them one by one takes longer than the rest of the call)."""
    if dev < 0:
        raise ValueError(f"{name}: needs CUDA tensors")
    call, pack, count = _lib.PACKED[name]
    handle = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        rc = _lib.load().inkling_rel_attn_packed(call, pack(*args, handle), count)
    else:
        with torch.cuda.device(dev):
            rc = _lib.load().inkling_rel_attn_packed(call, pack(*args, handle), count)
    if rc != 0:
        raise InklingError(rc, name)


def _own_stream(stream, t):
    """A given stream has to be of the tensors' device (of another one's the call would not run on it)."""
    if t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {t.device}")


def _error_word(device_error, dev):
    """Address of the optional error word."""
    if device_error is None:
        return 0
    if (device_error.dtype is not _I32 or device_error.get_device() != dev or device_error.dim() != 1
            or device_error.numel() < 1):
        raise TypeError("device_error: expected one int32 on the other tensors' device")
    return device_error.data_ptr()


def _workspace(workspace, need, q):
    """(workspace, bytes): the given one, or a new one of ``need()`` bytes."""
    if workspace is None:
        workspace = torch.empty(need(), dtype=_U8, device=q.device)
    elif workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the device of q")
    return workspace, workspace.nbytes


# The 4-bit and the 8-bit cache differ in their calls and in the bytes of a token's row of one KV head.
_CACHES = {"q4": ("9 * D / 16", {36: 64, 72: 128}), "q8": ("D + 1", {65: 64, 129: 128})}


def _block_cache(kind, k_cache, v_cache):
    """(num_pages, H_kv, page_size, D) of a pair of 4-bit or 8-bit pools; their devices are the caller's check."""
    last, rows = _CACHES[kind]
    if k_cache.dtype is not _U8 or v_cache.dtype is not _U8 or k_cache.dim() != 4:
        raise TypeError(f"k_cache, v_cache: uint8 pools [num_pages, H_kv, page_size, {last}] expected")
    n, H_kv, P, row = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if row not in rows:
        raise ValueError(f"k_cache: rows of {row} bytes; "
                         + " or ".join(f"{b} (D = {D})" for b, D in rows.items()) + " expected")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache, v_cache: must be contiguous")
    return n, H_kv, P, rows[row]


def build_tables(seq_lens, new_lens, page_table, free_pages, free_count, *, page_size, max_tokens=None,
                 kv_lens=None, cu_seqlens_q=None, slot_map=None, free_left=None, step_lens=None,
                 device_error=None, stream=None):
    """The tables of one serving step, from request lengths.  See
    inkling_rel_attn_build_tables.

    seq_lens, new_lens [B] int32 (new_lens < 0: the request has ended);
    page_table [B, stride] int32, extended in place; free_pages [num_pages]
    int32, a stack of free_count [1] int32 pages.  Returns (kv_lens [B] int32,
    cu_seqlens_q [B + 1] int32, slot_map [max_tokens] int64, free_left [1] int32);
    pass them to avoid allocations.  kv_lens=seq_lens and free_left=free_count
    step the state in place.  max_tokens is slot_map's length when that is given.
    Without requests: no tokens, no slot (-1), the stack as it is.
    step_lens [B] int32, if given, is written too: kv_lens, but 0 for a refused
    request.  Calls that place tokens by length (kv_append, kv_conv_append) take it
    instead of kv_lens, which would put refused rows over a request's last tokens.
    """
    if stream is not None:  # buffers made here are that stream's
        _own_stream(stream, seq_lens)
        with torch.cuda.stream(stream):
            return build_tables(seq_lens, new_lens, page_table, free_pages, free_count, page_size=page_size,
                                max_tokens=max_tokens, kv_lens=kv_lens, cu_seqlens_q=cu_seqlens_q, slot_map=slot_map,
                                free_left=free_left, step_lens=step_lens, device_error=device_error)
    B = seq_lens.numel()
    if kv_lens is None:
        kv_lens = torch.empty_like(seq_lens)
    if cu_seqlens_q is None:
        cu_seqlens_q = torch.empty(B + 1, dtype=_I32, device=seq_lens.device)
    if slot_map is None:
        if max_tokens is None:
            raise ValueError("max_tokens or slot_map is needed")
        slot_map = torch.empty(max_tokens, dtype=_I64, device=seq_lens.device)
    if free_left is None:
        free_left = torch.empty_like(free_count)
    dev = seq_lens.get_device()
    if not (seq_lens.dtype is new_lens.dtype is page_table.dtype is free_pages.dtype is free_count.dtype
            is kv_lens.dtype is cu_seqlens_q.dtype is free_left.dtype is _I32 and slot_map.dtype is _I64
            and new_lens.get_device() == page_table.get_device() == free_pages.get_device()
            == free_count.get_device() == kv_lens.get_device() == cu_seqlens_q.get_device()
            == slot_map.get_device() == free_left.get_device() == dev
            and seq_lens.is_contiguous() and new_lens.is_contiguous() and page_table.is_contiguous()
            and free_pages.is_contiguous() and kv_lens.is_contiguous() and cu_seqlens_q.is_contiguous()
            and slot_map.is_contiguous() and seq_lens.dim() == 1 and new_lens.shape == kv_lens.shape == seq_lens.shape
            and page_table.dim() == 2 and page_table.shape[0] == B and cu_seqlens_q.shape == (B + 1,)
            and free_pages.dim() == slot_map.dim() == 1 and free_count.shape == free_left.shape == (1,)
            and max_tokens in (None, slot_map.shape[0])):
        _refuse(dev, ((seq_lens, "seq_lens", _I32, 1), (new_lens, "new_lens", _I32, 1),
                      (page_table, "page_table", _I32, 2), (free_pages, "free_pages", _I32, 1),
                      (free_count, "free_count", _I32, 1), (kv_lens, "kv_lens", _I32, 1),
                      (cu_seqlens_q, "cu_seqlens_q", _I32, 1), (slot_map, "slot_map", _I64, 1),
                      (free_left, "free_left", _I32, 1)))
    if step_lens is not None and not (step_lens.dtype is _I32 and step_lens.get_device() == dev
                                      and step_lens.is_contiguous() and step_lens.shape == seq_lens.shape):
        _refuse(dev, ((step_lens, "step_lens", _I32, 1),))
    _launch("inkling_rel_attn_build_tables_step", dev, None,
            seq_lens.data_ptr(), new_lens.data_ptr(), page_table.data_ptr(), page_table.shape[1],
            free_pages.data_ptr(), free_count.data_ptr(), B, page_size, free_pages.shape[0],
            slot_map.shape[0], kv_lens.data_ptr(), cu_seqlens_q.data_ptr(), slot_map.data_ptr(),
            free_left.data_ptr(), 0 if step_lens is None else step_lens.data_ptr(), _error_word(device_error, dev))
    if B == 0:  # nothing was launched: an empty packing, no slot, the stack as it is
        cu_seqlens_q.zero_()
        slot_map.fill_(-1)
        if free_left.data_ptr() != free_count.data_ptr():
            free_left.copy_(free_count)
    return kv_lens, cu_seqlens_q, slot_map, free_left


def _append_rows(kind, k_new, v_new, slot_map, k_cache, v_cache, device_error, stream):
    if stream is not None:
        _own_stream(stream, k_new)
    n, H_kv, P, D = _block_cache(kind, k_cache, v_cache)
    T = slot_map.numel()
    dev = k_new.get_device()
    if not (k_new.dtype is v_new.dtype is _BF16 and slot_map.dtype is _I64
            and v_new.get_device() == slot_map.get_device() == k_cache.get_device() == v_cache.get_device() == dev
            and k_new.is_contiguous() and v_new.is_contiguous() and slot_map.is_contiguous()
            and k_new.shape == v_new.shape == (T, H_kv, D) and slot_map.dim() == 1):
        _refuse(dev, ((k_new, "k_new", _BF16, 3), (v_new, "v_new", _BF16, 3), (slot_map, "slot_map", _I64, 1),
                      (k_cache, "k_cache", _U8, 4), (v_cache, "v_cache", _U8, 4)))
    _launch(f"inkling_rel_attn_kv_append_{kind}", dev, stream,
            k_new.data_ptr(), v_new.data_ptr(), slot_map.data_ptr(), T, H_kv, D, P, n,
            k_cache.data_ptr(), v_cache.data_ptr(), _error_word(device_error, dev))


def kv_append_q4(k_new, v_new, slot_map, k_cache, v_cache, *, device_error=None, stream=None):
    """Quantise the new tokens' K/V rows into the 4-bit paged cache (in place).
    See inkling_rel_attn_kv_append_q4.

    k_new, v_new [T, H_kv, D] bf16; slot_map [T] int64 (page * page_size + place,
    negative: skipped); k_cache, v_cache [num_pages, H_kv, page_size, 9 * D / 16]
    uint8.
    """
    _append_rows("q4", k_new, v_new, slot_map, k_cache, v_cache, device_error, stream)


def kv_append_q8(k_new, v_new, slot_map, k_cache, v_cache, *, device_error=None, stream=None):
    """Quantise the new tokens' K/V rows into the 8-bit paged cache (in place).
    See inkling_rel_attn_kv_append_q8.

    k_new, v_new [T, H_kv, D] bf16; slot_map [T] int64 (page * page_size + place,
    negative: skipped; the tokens of one block of 16 places within 16 of the call,
    as build_tables gives them); k_cache, v_cache [num_pages, H_kv, page_size, D + 1]
    uint8, zeros before their first use.
    """
    _append_rows("q8", k_new, v_new, slot_map, k_cache, v_cache, device_error, stream)


def _read_rows(kind, slot_map, k_cache, v_cache, k_rows, v_rows, device_error, stream):
    if stream is not None:  # buffers made here are that stream's
        _own_stream(stream, k_cache)
        with torch.cuda.stream(stream):
            return _read_rows(kind, slot_map, k_cache, v_cache, k_rows, v_rows, device_error, None)
    n, H_kv, P, D = _block_cache(kind, k_cache, v_cache)
    T = slot_map.numel()
    if k_rows is None:
        k_rows = torch.empty((T, H_kv, D), dtype=_BF16, device=k_cache.device)
    if v_rows is None:
        v_rows = torch.empty((T, H_kv, D), dtype=_BF16, device=k_cache.device)
    dev = k_cache.get_device()
    if not (k_rows.dtype is v_rows.dtype is _BF16 and slot_map.dtype is _I64
            and v_cache.get_device() == slot_map.get_device() == k_rows.get_device() == v_rows.get_device() == dev
            and k_rows.is_contiguous() and v_rows.is_contiguous() and slot_map.is_contiguous()
            and k_rows.shape == v_rows.shape == (T, H_kv, D) and slot_map.dim() == 1):
        _refuse(dev, ((k_cache, "k_cache", _U8, 4), (v_cache, "v_cache", _U8, 4), (slot_map, "slot_map", _I64, 1),
                      (k_rows, "k_rows", _BF16, 3), (v_rows, "v_rows", _BF16, 3)))
    _launch(f"inkling_rel_attn_kv_read_{kind}", dev, None,
            slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), T, H_kv, D, P, n,
            k_rows.data_ptr(), v_rows.data_ptr(), _error_word(device_error, dev))
    return k_rows, v_rows


def kv_read_q4(slot_map, k_cache, v_cache, *, k_rows=None, v_rows=None, device_error=None, stream=None):
    """Rows of the 4-bit cache as the bf16 values they stand for.  See
    inkling_rel_attn_kv_read_q4.  Returns (k_rows, v_rows) [T, H_kv, D] bf16.
    """
    return _read_rows("q4", slot_map, k_cache, v_cache, k_rows, v_rows, device_error, stream)


def kv_read_q8(slot_map, k_cache, v_cache, *, k_rows=None, v_rows=None, device_error=None, stream=None):
    """Rows of the 8-bit cache as the bf16 values they stand for.  See
    inkling_rel_attn_kv_read_q8.  Returns (k_rows, v_rows) [T, H_kv, D] bf16.
    """
    return _read_rows("q8", slot_map, k_cache, v_cache, k_rows, v_rows, device_error, stream)


def decode_q4_workspace_bytes(B, q_len, H_q, H_kv, D, num_sms=0):
    return _lib.inkling_rel_attn_decode_q4_workspace_size(B, q_len, H_q, H_kv, D, num_sms)


def decode_q8_workspace_bytes(B, q_len, H_q, H_kv, D, num_sms=0):
    return _lib.inkling_rel_attn_decode_q8_workspace_size(B, q_len, H_q, H_kv, D, num_sms)


def _decode_blocks(kind, q, k_cache, v_cache, page_table, seq_lens, rel_logits, q_len, window, scale, out, lse, workspace,
                   device_error, stream):
    if stream is not None:  # buffers made here are that stream's
        _own_stream(stream, q)
        with torch.cuda.stream(stream):
            return _decode_blocks(kind, q, k_cache, v_cache, page_table, seq_lens, rel_logits, q_len, window, scale, out,
                                  lse, workspace, device_error, None)
    try:
        (T, H_q, _), (rel_T, rel_H, R), (rows, stride), (B,) = (q.shape, rel_logits.shape, page_table.shape,
                                                                seq_lens.shape)
    except ValueError:  # one of another rank: refused below
        T = H_q = rel_T = rel_H = R = rows = stride = B = -1
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    n, H_kv, P, D = _block_cache(kind, k_cache, v_cache)
    dev = q.get_device()
    if not (q.dtype is out.dtype is _BF16 and page_table.dtype is seq_lens.dtype is _I32
            and rel_logits.dtype is lse.dtype is _F32
            and k_cache.get_device() == v_cache.get_device() == page_table.get_device() == seq_lens.get_device()
            == rel_logits.get_device() == out.get_device() == lse.get_device() == dev
            and q.is_contiguous() and page_table.is_contiguous() and seq_lens.is_contiguous()
            and rel_logits.is_contiguous() and out.is_contiguous() and lse.is_contiguous()
            and q.shape == out.shape == (B * q_len, H_q, D) and lse.shape == (T, H_q)
            and rel_T == T and rel_H == H_q and rows == B):
        _refuse(dev, ((q, "q", _BF16, 3), (k_cache, "k_cache", _U8, 4), (v_cache, "v_cache", _U8, 4),
                      (page_table, "page_table", _I32, 2), (seq_lens, "seq_lens", _I32, 1),
                      (rel_logits, "rel_logits", _F32, 3), (out, "out", _BF16, 3), (lse, "lse", _F32, 2)))
    workspace, ws_bytes = _workspace(workspace, lambda: decode_q4_workspace_bytes(B, q_len, H_q, H_kv, D), q)
    _launch(f"inkling_rel_attn_decode_{kind}", dev, None,
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), stride,
            seq_lens.data_ptr(), rel_logits.data_ptr(), B, q_len, H_q, H_kv, D, P, n, R,
            window, scale, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), ws_bytes,
            _error_word(device_error, dev))
    return out, lse


def decode_q4(q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, q_len=1, window, scale, out=None,
              lse=None, workspace=None, device_error=None, stream=None):
    """Decode of the last ``q_len`` tokens of each sequence over the 4-bit cache.
    See inkling_rel_attn_decode_q4.

    q [B * q_len, H_q, D] bf16 (row b * q_len + i); k_cache, v_cache [num_pages,
    H_kv, page_size, 9 * D / 16] uint8; page_table [B, stride] int32; seq_lens
    [B] int32; rel_logits [B * q_len, H_q, R] fp32.  Returns (out bf16 like q,
    lse fp32 [B * q_len, H_q]).  Pass ``out``, ``lse`` and ``workspace``
    (decode_q4_workspace_bytes) to avoid allocations.
    """
    return _decode_blocks("q4", q, k_cache, v_cache, page_table, seq_lens, rel_logits, q_len, window, scale, out, lse,
                          workspace, device_error, stream)


def decode_q8(q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, q_len=1, window, scale, out=None,
              lse=None, workspace=None, device_error=None, stream=None):
    """Decode of the last ``q_len`` tokens of each sequence over the 8-bit cache.
    See inkling_rel_attn_decode_q8.

    k_cache, v_cache [num_pages, H_kv, page_size, D + 1] uint8; the rest as for
    ``decode_q4``.  Returns (out bf16 like q, lse fp32 [B * q_len, H_q]).  Pass
    ``out``, ``lse`` and ``workspace`` (decode_q8_workspace_bytes) to avoid
    allocations.
    """
    return _decode_blocks("q8", q, k_cache, v_cache, page_table, seq_lens, rel_logits, q_len, window, scale, out, lse,
                          workspace, device_error, stream)


def prefill_q4_workspace_bytes(B, max_q_len, H_kv, D, window, max_seq_len):
    return _lib.inkling_rel_attn_prefill_q4_workspace_size(B, max_q_len, H_kv, D, window, max_seq_len)


def prefill_q8_workspace_bytes(B, max_q_len, H_kv, D, window, max_seq_len):
    return _lib.inkling_rel_attn_prefill_q8_workspace_size(B, max_q_len, H_kv, D, window, max_seq_len)


def _prefill_blocks(kind, q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, window, scale, max_seq_len,
                    max_q_len, out, lse, workspace, device_error, stream):
    if stream is not None:  # buffers made here are that stream's
        _own_stream(stream, q)
        with torch.cuda.stream(stream):
            return _prefill_blocks(kind, q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, window,
                                   scale, max_seq_len, max_q_len, out, lse, workspace, device_error, None)
    try:
        (T, H_q, _), (rel_T, rel_H, R), (rows, stride), (B,) = (q.shape, rel_logits.shape, page_table.shape,
                                                                seq_lens.shape)
    except ValueError:  # one of another rank: refused below
        T = H_q = rel_T = rel_H = R = rows = stride = B = -1
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    n, H_kv, P, D = _block_cache(kind, k_cache, v_cache)
    dev = q.get_device()
    if not (q.dtype is out.dtype is _BF16
            and page_table.dtype is seq_lens.dtype is cu_seqlens_q.dtype is _I32
            and rel_logits.dtype is lse.dtype is _F32
            and k_cache.get_device() == v_cache.get_device() == page_table.get_device() == seq_lens.get_device()
            == cu_seqlens_q.get_device() == rel_logits.get_device() == out.get_device() == lse.get_device() == dev
            and q.is_contiguous() and page_table.is_contiguous() and seq_lens.is_contiguous()
            and cu_seqlens_q.is_contiguous() and rel_logits.is_contiguous() and out.is_contiguous()
            and lse.is_contiguous() and q.shape == out.shape == (T, H_q, D) and lse.shape == (T, H_q)
            and cu_seqlens_q.shape == (B + 1,) and rel_T == T and rel_H == H_q and rows == B >= 0):
        _refuse(dev, ((q, "q", _BF16, 3), (cu_seqlens_q, "cu_seqlens_q", _I32, 1), (k_cache, "k_cache", _U8, 4),
                      (v_cache, "v_cache", _U8, 4), (page_table, "page_table", _I32, 2),
                      (seq_lens, "seq_lens", _I32, 1), (rel_logits, "rel_logits", _F32, 3),
                      (out, "out", _BF16, 3), (lse, "lse", _F32, 2)))
    workspace, ws_bytes = _workspace(
        workspace, lambda: prefill_q4_workspace_bytes(B, max_q_len, H_kv, D, window, max_seq_len), q)
    _launch(f"inkling_rel_attn_prefill_{kind}", dev, None,
            q.data_ptr(), cu_seqlens_q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            page_table.data_ptr(), stride, seq_lens.data_ptr(), rel_logits.data_ptr(), B, T,
            max_q_len, H_q, H_kv, D, P, n, R, window, scale, max_seq_len, out.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), ws_bytes, _error_word(device_error, dev))
    return out, lse


def prefill_q4(q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, window, scale,
               max_seq_len, max_q_len, out=None, lse=None, workspace=None, device_error=None, stream=None):
    """Chunked / paged prefill over the 4-bit cache.  See inkling_rel_attn_prefill_q4.

    q [T, H_q, D] bf16; cu_seqlens_q [B + 1] int32; rel_logits [T, H_q, R] fp32;
    the cache, page_table and seq_lens as for ``decode_q4``; max_seq_len and
    max_q_len are host bounds.  Returns (out bf16 [T, H_q, D], lse fp32 [T, H_q]).
    Pass ``out``, ``lse`` and ``workspace`` (prefill_q4_workspace_bytes) to avoid
    allocations.
    """
    return _prefill_blocks("q4", q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, window, scale,
                           max_seq_len, max_q_len, out, lse, workspace, device_error, stream)


def prefill_q8(q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, *, window, scale,
               max_seq_len, max_q_len, out=None, lse=None, workspace=None, device_error=None, stream=None):
    """Chunked / paged prefill over the 8-bit cache.  See inkling_rel_attn_prefill_q8.

    k_cache, v_cache [num_pages, H_kv, page_size, D + 1] uint8; the rest as for
    ``prefill_q4``.  Returns (out bf16 [T, H_q, D], lse fp32 [T, H_q]).  Pass ``out``,
    ``lse`` and ``workspace`` (prefill_q8_workspace_bytes) to avoid allocations.
    """
    return _prefill_blocks("q8", q, cu_seqlens_q, k_cache, v_cache, page_table, seq_lens, rel_logits, window, scale,
                           max_seq_len, max_q_len, out, lse, workspace, device_error, stream)


# ---------------------------------------------------------------------------
# Shared pages
# ---------------------------------------------------------------------------

def _refuse_ints(dev, **tensors):
    """_refuse of int32 tensors; all are of rank 1 but page_table."""
    _refuse(dev, [(t, name, _I32, 2 if name == "page_table" else 1) for name, t in tensors.items()])


def _on_stream(stream, t, call):
    """``call()`` with ``stream`` as the current one: buffers made there are that stream's."""
    _own_stream(stream, t)
    with torch.cuda.stream(stream):
        return call()


def fork_pages(source, seq_lens, page_table, page_refs, free_pages, free_count, *, page_size, kv_lens=None,
               copy_src=None, copy_dst=None, free_left=None, device_error=None, stream=None):
    """Requests that go on from another one's tokens, its full pages shared.  See
    inkling_rel_attn_fork_pages.

    source [B] int32 (the row to go on from, -1: nothing to do; forks are empty rows);
    seq_lens [B] int32; page_table [B, stride] and page_refs [num_pages] int32, updated in
    place; free_pages [num_pages] int32, a stack of free_count [1] int32 pages.
    Returns (kv_lens [B], copy_src [B], copy_dst [B], free_left [1]), int32; pass them to
    avoid allocations.  kv_lens=seq_lens and free_left=free_count step the state in
    place.  ``copy_pages(pools, copy_src, copy_dst)`` then copies the partial pages.  A fork
    for which there is no page, or that meets a page id that is none, stays empty.
    """
    if stream is not None:
        return _on_stream(stream, seq_lens, lambda: fork_pages(
            source, seq_lens, page_table, page_refs, free_pages, free_count, page_size=page_size, kv_lens=kv_lens,
            copy_src=copy_src, copy_dst=copy_dst, free_left=free_left, device_error=device_error))
    B, n = seq_lens.numel(), free_pages.numel()
    kv_lens = torch.empty_like(seq_lens) if kv_lens is None else kv_lens
    copy_src = torch.empty_like(seq_lens) if copy_src is None else copy_src
    copy_dst = torch.empty_like(seq_lens) if copy_dst is None else copy_dst
    free_left = torch.empty_like(free_count) if free_left is None else free_left
    dev = seq_lens.get_device()
    if not (seq_lens.dtype is source.dtype is page_table.dtype is page_refs.dtype is free_pages.dtype is free_count.dtype
            is kv_lens.dtype is copy_src.dtype is copy_dst.dtype is free_left.dtype is _I32
            and source.get_device() == page_table.get_device() == page_refs.get_device() == free_pages.get_device()
            == free_count.get_device() == kv_lens.get_device() == copy_src.get_device() == copy_dst.get_device()
            == free_left.get_device() == dev
            and seq_lens.is_contiguous() and source.is_contiguous() and page_table.is_contiguous()
            and page_refs.is_contiguous() and free_pages.is_contiguous() and kv_lens.is_contiguous()
            and copy_src.is_contiguous() and copy_dst.is_contiguous()
            and seq_lens.dim() == free_pages.dim() == 1 and page_table.dim() == 2 and page_table.shape[0] == B
            and source.shape == kv_lens.shape == copy_src.shape == copy_dst.shape == seq_lens.shape
            and page_refs.shape == free_pages.shape and free_count.shape == free_left.shape == (1,)):
        _refuse_ints(dev, seq_lens=seq_lens, source=source, page_table=page_table, page_refs=page_refs,
                     free_pages=free_pages, free_count=free_count, kv_lens=kv_lens, copy_src=copy_src,
                     copy_dst=copy_dst, free_left=free_left)
    _launch("inkling_rel_attn_fork_pages", dev, None, source.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(),
            page_table.shape[1], page_refs.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), B, page_size, n,
            kv_lens.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(), free_left.data_ptr(),
            _error_word(device_error, dev))
    if B == 0 and free_left.data_ptr() != free_count.data_ptr():  # nothing was launched
        free_left.copy_(free_count)
    return kv_lens, copy_src, copy_dst, free_left


def release_pages(seq_lens, new_lens, page_table, page_refs, free_pages, free_count, *, page_size, kv_lens=None,
                  free_left=None, device_error=None, stream=None):
    """Pages of ended requests (new_lens < 0) lose an owner; those without one go back on the stack.  See
    inkling_rel_attn_release_pages.

    Arguments as for ``fork_pages``; free_pages is written above its top.  Returns
    (kv_lens [B]: seq_lens, but 0 for the ended, free_left [1]), int32.
    """
    if stream is not None:
        return _on_stream(stream, seq_lens, lambda: release_pages(
            seq_lens, new_lens, page_table, page_refs, free_pages, free_count, page_size=page_size, kv_lens=kv_lens,
            free_left=free_left, device_error=device_error))
    B, n = seq_lens.numel(), free_pages.numel()
    kv_lens = torch.empty_like(seq_lens) if kv_lens is None else kv_lens
    free_left = torch.empty_like(free_count) if free_left is None else free_left
    dev = seq_lens.get_device()
    if not (seq_lens.dtype is new_lens.dtype is page_table.dtype is page_refs.dtype is free_pages.dtype
            is free_count.dtype is kv_lens.dtype is free_left.dtype is _I32
            and new_lens.get_device() == page_table.get_device() == page_refs.get_device() == free_pages.get_device()
            == free_count.get_device() == kv_lens.get_device() == free_left.get_device() == dev
            and seq_lens.is_contiguous() and new_lens.is_contiguous() and page_table.is_contiguous()
            and page_refs.is_contiguous() and free_pages.is_contiguous() and kv_lens.is_contiguous()
            and seq_lens.dim() == free_pages.dim() == 1 and page_table.dim() == 2 and page_table.shape[0] == B
            and new_lens.shape == kv_lens.shape == seq_lens.shape and page_refs.shape == free_pages.shape
            and free_count.shape == free_left.shape == (1,)):
        _refuse_ints(dev, seq_lens=seq_lens, new_lens=new_lens, page_table=page_table, page_refs=page_refs,
                     free_pages=free_pages, free_count=free_count, kv_lens=kv_lens, free_left=free_left)
    _launch("inkling_rel_attn_release_pages", dev, None, seq_lens.data_ptr(), new_lens.data_ptr(),
            page_table.data_ptr(), page_table.shape[1], page_refs.data_ptr(), free_pages.data_ptr(),
            free_count.data_ptr(), B, page_size, n, kv_lens.data_ptr(), free_left.data_ptr(), _error_word(device_error, dev))
    if B == 0 and free_left.data_ptr() != free_count.data_ptr():  # nothing was launched
        free_left.copy_(free_count)
    return kv_lens, free_left


def compact_pages(seq_lens, page_table, free_pages, free_count, *, page_size, page_refs=None, move_src=None,
                  move_dst=None, moves=None, device_error=None, stream=None):
    """The pages in use brought together at the low end of the pool.  See inkling_rel_attn_compact_pages.

    page_table, free_pages (up to its height) and page_refs, if given, are updated in
    place.  Returns (move_src [num_pages], move_dst [num_pages], moves [1]), int32;
    ``copy_pages(pools, move_src, move_dst, count=moves)`` then moves the pages' content.
    """
    if stream is not None:
        return _on_stream(stream, seq_lens, lambda: compact_pages(
            seq_lens, page_table, free_pages, free_count, page_size=page_size, page_refs=page_refs, move_src=move_src,
            move_dst=move_dst, moves=moves, device_error=device_error))
    B, n = seq_lens.numel(), free_pages.numel()
    move_src = torch.empty_like(free_pages) if move_src is None else move_src
    move_dst = torch.empty_like(free_pages) if move_dst is None else move_dst
    moves = torch.empty_like(free_count) if moves is None else moves
    dev = seq_lens.get_device()
    refs = free_pages if page_refs is None else page_refs  # (checked alike)
    if not (seq_lens.dtype is page_table.dtype is free_pages.dtype is free_count.dtype is move_src.dtype
            is move_dst.dtype is moves.dtype is refs.dtype is _I32
            and page_table.get_device() == free_pages.get_device() == free_count.get_device() == move_src.get_device()
            == move_dst.get_device() == moves.get_device() == refs.get_device() == dev
            and seq_lens.is_contiguous() and page_table.is_contiguous() and free_pages.is_contiguous()
            and move_src.is_contiguous() and move_dst.is_contiguous() and refs.is_contiguous()
            and seq_lens.dim() == free_pages.dim() == 1 and page_table.dim() == 2 and page_table.shape[0] == B
            and move_src.shape == move_dst.shape == refs.shape == free_pages.shape
            and free_count.shape == moves.shape == (1,)):
        _refuse_ints(dev, seq_lens=seq_lens, page_table=page_table, free_pages=free_pages, free_count=free_count,
                     page_refs=refs, move_src=move_src, move_dst=move_dst, moves=moves)
    _launch("inkling_rel_attn_compact_pages", dev, None, seq_lens.data_ptr(), page_table.data_ptr(), page_table.shape[1],
            0 if page_refs is None else page_refs.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), B,
            page_size, n, move_src.data_ptr(), move_dst.data_ptr(), moves.data_ptr(), _error_word(device_error, dev))
    return move_src, move_dst, moves


def copy_pages(pools, src, dst, *, count=None, device_error=None, stream=None):
    """Page src[i] copied to page dst[i] in every pool (in place).  See inkling_rel_attn_copy_pages.

    pools: a list of tensors of any type with pages along dimension 0, the same number of pages of
    the same size (K and V of the layers with one kind of cache, in bf16, 4 or 8
    bits); src, dst [n] int32 (negative: skipped); count [1] int32: the pairs to copy,
    all without it.
    """
    if not pools:
        return
    first = pools[0]
    if stream is not None:
        _own_stream(stream, first)
    dev, n, size = first.get_device(), src.numel(), first.nbytes
    pages = first.shape[0] if first.dim() > 0 else 0
    for i, t in enumerate(pools):
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"pools[{i}]: must be contiguous and on the other pools' device")
        if t.nbytes != size or t.dim() < 1 or t.shape[0] != pages:
            raise ValueError(f"pools[{i}]: pages of another number or size than those of the first pool")
    if not (src.dtype is dst.dtype is _I32 and src.get_device() == dst.get_device() == dev and src.is_contiguous()
            and dst.is_contiguous() and src.dim() == 1 and src.shape == dst.shape):
        _refuse_ints(dev, src=src, dst=dst)
    if count is not None and not (count.dtype is _I32 and count.get_device() == dev and count.shape == (1,)):
        _refuse_ints(dev, count=count)
    table = _lib.pointers([t.data_ptr() for t in pools])
    _launch("inkling_rel_attn_copy_pages", dev, stream, _lib.address_of(table), len(pools), size // max(pages, 1), pages,
            src.data_ptr(), dst.data_ptr(), n, 0 if count is None else count.data_ptr(),
            _error_word(device_error, dev))


def decode_inputs(inp, **kw):
    """``decode`` on a workloads.DecodeInputs-like object."""
    return decode(inp.q, inp.k_cache, inp.v_cache, inp.page_table, inp.seq_lens, inp.rel_logits,
                  window=inp.window, scale=inp.scale, max_seq_len=inp.max_seq_len, **kw)


def prefill_inputs(inp, **kw):
    """``prefill`` on a workloads.PrefillInputs-like object."""
    return prefill(inp.q, inp.cu_seqlens_q, inp.k_cache, inp.v_cache, inp.page_table,
                   inp.seq_lens, inp.rel_logits, window=inp.window, scale=inp.scale,
                   max_seq_len=inp.max_seq_len, max_q_len=inp.max_q_len, **kw)
