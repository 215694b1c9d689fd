"""Shared pages without a GPU: pins of the oracle, refusals of the C ABI, of its packed form and of the wrappers."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.pages import ref_compact, ref_fork, ref_release


@pytest.fixture(scope="module")
def lib():
    from paged_attention_relative_attn_gb300 import build, _lib
    build.build()
    return _lib


# ------------------------------------------------------------------ the oracle

def test_fork_release_compact_by_hand():
    # page size 16: row 0 has 40 tokens in pages 7, 2, 5; rows 2 and 3 go on from it
    table = np.array([[7, 2, 5, 0], [9, 0, 0, 0], [0, 0, 0, 0], [0, 0, 0, 0]])
    refs, free = np.zeros(10, dtype=int), np.array([1, 4, 8, 0, 0, 0, 0, 0, 0, 0])
    f = ref_fork([-1, -1, 0, 0], [40, 16, 0, 0], table, refs, free, 3, 16)
    assert list(f["table"][2]) == [7, 2, 8, 0] and list(f["table"][3]) == [7, 2, 4, 0]
    assert f["refs"][7] == f["refs"][2] == 2 and f["refs"].sum() == 4 and f["left"] == 1
    assert list(f["src"]) == [-1, -1, 5, 5] and list(f["dst"]) == [-1, -1, 8, 4]
    assert list(f["kv_lens"]) == [40, 16, 40, 40] and not f["bits"]
    # the prompt's row and one sample end: the shared pages stay with the last owner
    r = ref_release(f["kv_lens"], [-1, 1, -1, 1], f["table"], f["refs"], free, 1, 16)
    assert list(r["free"][:3]) == [1, 5, 8] and r["left"] == 3
    assert r["refs"][7] == r["refs"][2] == 0 and list(r["kv_lens"]) == [0, 16, 0, 40]
    # live: 9; 7, 2, 4.  known: 1 2 4 5 7 8 9 (0, 3, 6 are nobody's): the lowest four are 1 2 4 5
    c = ref_compact(r["kv_lens"], f["table"], r["refs"], r["free"], 3, 16)
    assert c["moves"] == 2 and list(c["src"][:2]) == [7, 9] and list(c["dst"][:2]) == [1, 5]
    assert list(c["table"][3, :3]) == [1, 2, 4] and c["table"][1, 0] == 5
    assert list(c["free"][:3]) == [9, 8, 7] and not c["bits"]


def test_last_owner_gives_the_page_back():
    table = np.array([[3, 1], [3, 2], [3, 0]])
    refs = np.array([0, 0, 0, 2])
    r = ref_release([32, 32, 32], [-1, -1, -1], table, refs, np.zeros(4, dtype=int), 0, 16)
    assert list(r["free"]) == [1, 2, 3, 0] and r["left"] == 4 and not r["refs"].any()


# ------------------------------------------------------------------ refusals

def plain_args():
    a4 = lambda n: (n, 4, 2, -2)  # noqa: E731
    ok = lambda n, v: (n, v, None, None)  # noqa: E731
    shape = [("B", 2, -1, -1), ("page_size", 16, 40, -1), ("num_pages", 8, 0, -1)]
    return {
        "fork_pages": [a4("source"), a4("seq_lens"), a4("page_table"), ("stride", 4, 0, -1), a4("page_refs"),
                       a4("free_pages"), a4("free_count"), *shape, a4("kv_lens"), a4("copy_src"), a4("copy_dst"),
                       a4("free_left"), a4("device_error"), ok("stream", 0)],
        "release_pages": [a4("seq_lens"), a4("new_lens"), a4("page_table"), ("stride", 4, 0, -1), a4("page_refs"),
                          a4("free_pages"), a4("free_count"), *shape, a4("kv_lens"), a4("free_left"),
                          a4("device_error"), ok("stream", 0)],
        "compact_pages": [a4("seq_lens"), a4("page_table"), ("stride", 4, 0, -1), a4("page_refs"), a4("free_pages"),
                          a4("free_count"), *shape, a4("move_src"), a4("move_dst"), a4("moves"), a4("device_error"),
                          ok("stream", 0)],
    }


@pytest.mark.parametrize("name", sorted(plain_args()))
def test_calls_and_packed_calls_check_every_argument(lib, name):
    spec = plain_args()[name]
    call, pack, count = lib.PACKED["inkling_rel_attn_" + name]
    f = getattr(lib, "inkling_rel_attn_" + name)
    assert count == len(spec)
    good = [s[1] for s in spec]
    for i, (arg, value, bad, code) in enumerate(spec):
        if bad is None:
            continue
        args = good[:i] + [bad] + good[i + 1:]
        assert f(*args) == code and lib.inkling_rel_attn_packed(call, pack(*args), count) == code, arg
        if arg in ("B", "stride", "page_size", "num_pages"):
            wide = good[:i] + [value + (1 << 32)] + good[i + 1:]
            assert lib.inkling_rel_attn_packed(call, pack(*wide), count) == -1, arg
        elif arg != "device_error" and (name, arg) != ("compact_pages", "page_refs"):
            args[i] = 0
            assert f(*args) == -1, arg  # required
    assert lib.inkling_rel_attn_packed(call, pack(*good), count - 1) == -1
    at = [s[0] for s in spec].index("B")
    assert f(*(good[:at] + [8193] + good[at + 1:])) == -1
    assert f(*(good[:at - 0] + [0] + good[at + 1:])) == (0 if name != "compact_pages" else f(*good))
    assert f(*[1 << 28 if s[0] == "stride" else g for s, g in zip(spec, good)]) == -1


def test_release_table_size(lib):
    f = lib.inkling_rel_attn_release_pages
    assert f(4, 4, 4, (1 << 17) + 1, 4, 4, 4, 8192, 16, 8, 4, 4, 4, 0) == -1
    assert f(4, 4, 4, 1 << 17, 4, 4, 2, 8192, 16, 8, 4, 4, 4, 0) == -2  # the size is taken, the address is not


def test_row_that_holds_a_page_twice():
    r = ref_release([48, 16], [-1, -1], np.array([[3, 3, 2], [1, 0, 0]]), np.zeros(4, dtype=int), np.zeros(4, dtype=int), 0, 16)
    assert list(r["free"]) == [3, 2, 1, 0] and r["left"] == 3 and r["bits"] == {"bad_page"} and not r["refs"].any()


def test_compact_pool_size(lib):
    spec = plain_args()["compact_pages"]
    args = [(1 << 19) + 1 if s[0] == "num_pages" else s[1] for s in spec]
    assert lib.inkling_rel_attn_compact_pages(*args) == -1


def test_copy_validation(lib):
    pools = lib.pointers([16, 32])
    f = lambda pools=pools, n_pools=2, page_bytes=64, num_pages=8, src=4, dst=4, n=2, count=None, err=None: (  # noqa: E731
        lib.inkling_rel_attn_copy_pages(pools, n_pools, page_bytes, num_pages, src, dst, n, count, err, None))
    assert f(n_pools=-1) == -1 and f(n=-1) == -1 and f(page_bytes=0) == -1 and f(page_bytes=24) == -1
    assert f(page_bytes=1 << 31) == -1 and f(num_pages=0) == -1 and f(src=None) == -1 and f(dst=None) == -1
    assert f(pools=None) == -1 and f(pools=lib.pointers([16, None])) == -1
    assert f(n=0) == 0 and f(n_pools=0) == 0
    assert f(pools=lib.pointers([16, 24])) == -2 and f(src=2) == -2 and f(count=2) == -2 and f(err=2) == -2
    call, pack, count = lib.PACKED["inkling_rel_attn_copy_pages"]
    words = [lib.address_of(pools), 2, 64, 8, 4, 4, 2, 0, 0, 0]
    for i, bad, code in ((1, -1, -1), (2, 24, -1), (2, 1 << 40, -1), (3, 0, -1), (4, 2, -2), (6, 1 << 33, -1), (7, 2, -2)):
        args = words[:i] + [bad] + words[i + 1:]
        assert lib.inkling_rel_attn_packed(call, pack(*args), count) == code, i
    assert lib.inkling_rel_attn_packed(13, pack(*words), count) == -1


def test_wrappers_refuse_wrong_tensors():
    import paged_attention_relative_attn_gb300 as ira
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kw = dict(page_size=16)
    with pytest.raises(TypeError, match="source"):
        ira.fork_pages(i32(2).long(), i32(2), i32(2, 4), i32(8), i32(8), i32(1), **kw)
    with pytest.raises(ValueError, match="page_table"):
        ira.fork_pages(i32(2), i32(2), i32(8), i32(8), i32(8), i32(1), **kw)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.fork_pages(i32(2), i32(2), i32(2, 4), i32(7), i32(8), i32(1), **kw)
    with pytest.raises(ValueError, match="contiguous"):
        ira.release_pages(i32(2), i32(2), i32(2, 8)[:, ::2], i32(8), i32(8), i32(1), **kw)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.release_pages(i32(2), i32(3), i32(2, 4), i32(8), i32(8), i32(1), **kw)
    with pytest.raises(ValueError, match="inconsistent"):
        ira.compact_pages(i32(2), i32(2, 4), i32(8), i32(1), move_src=i32(4), **kw)
    with pytest.raises(TypeError, match="page_refs"):
        ira.compact_pages(i32(2), i32(2, 4), i32(8), i32(1), page_refs=i32(8).float(), **kw)
    pool = torch.zeros((4, 2, 16, 65), dtype=torch.uint8)
    with pytest.raises(ValueError, match=r"pools\[1\]"):
        ira.copy_pages([pool, pool[:3]], i32(1), i32(1))
    with pytest.raises(ValueError, match=r"pools\[0\]"):
        ira.copy_pages([pool[:, :, ::2]], i32(1), i32(1))
    with pytest.raises(ValueError, match="inconsistent"):
        ira.copy_pages([pool], i32(1), i32(2))
    with pytest.raises(TypeError, match="count"):
        ira.copy_pages([pool], i32(1), i32(1), count=i32(1).long())
    ira.copy_pages([], i32(1), i32(1))
    # the right types and shapes, but on the CPU
    for call in (lambda: ira.fork_pages(i32(2), i32(2), i32(2, 4), i32(8), i32(8), i32(1), **kw),
                 lambda: ira.release_pages(i32(2), i32(2), i32(2, 4), i32(8), i32(8), i32(1), **kw),
                 lambda: ira.compact_pages(i32(2), i32(2, 4), i32(8), i32(1), **kw),
                 lambda: ira.copy_pages([pool], i32(1), i32(1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
