"""What the pages' calls refuse, on the host, before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_landmark_gb300 import build
    build.build()
    return kvo.lib()


P = 1 << 20       # an aligned address that is never read


def refused(lib, st, frag):
    assert st == kvo.KVO_ERR_INVALID
    assert frag in lib.kvo_last_error(None).decode()


def book(**kw):
    a = dict(table=P, held=2 * P, refs=3 * P, batch=4, max_pages=8, n_pages=100, page=16)
    a.update(kw)
    return kvo._PageBook(a["table"], a["held"], a["refs"], a["batch"], a["max_pages"], a["n_pages"], a["page"])


def reserve(lib, b, want=4 * P):
    return lib.kvo_paged_reserve(b, want, None, None)


def fork(lib, b, parent=4 * P, keep=5 * P, src=6 * P, dst=7 * P, count=8 * P, ws=9 * P, size=P):
    return lib.kvo_paged_fork(b, parent, keep, src, dst, count, ws, size, None, None)


def compact(lib, b, table_out=None, refs_out=None, src=6 * P, dst=7 * P, count=8 * P, ws=9 * P, size=P):
    return lib.kvo_paged_compact(b, table_out, refs_out, src, dst, count, ws, size, None, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(batch=-1), "batch"), (dict(batch=8193), "batch"), (dict(max_pages=0), "max_pages"), (dict(n_pages=0), "n_pages"),
    (dict(page=0), "page_size"), (dict(max_pages=2 ** 20, page=4096), "2^31"), (dict(batch=8192, max_pages=2 ** 18), "31 bits"),
    (dict(table=None), "null"), (dict(held=None), "null"), (dict(refs=None), "null"), (dict(refs=P + 4), "aligned")])
def test_all_calls_refuse_bad_books(lib, kw, frag):
    b = book(**kw)
    refused(lib, reserve(lib, b), frag)
    refused(lib, fork(lib, b), frag)
    refused(lib, compact(lib, b), frag)
    for f in (lib.kvo_paged_fork_workspace, lib.kvo_paged_compact_workspace):
        n = ctypes.c_size_t(7)
        refused(lib, f(b, ctypes.byref(n)), frag)
        assert n.value == 0
        refused(lib, f(book(), None), "null")
    refused(lib, reserve(lib, None), "null book")
    refused(lib, fork(lib, None), "null book")
    refused(lib, compact(lib, None), "null book")


def test_calls_refuse_missing_and_small_buffers(lib):
    refused(lib, reserve(lib, book(), None), "null")
    for x in ("parent", "keep", "src", "dst", "count"):
        refused(lib, fork(lib, book(), **{x: None}), "null")
    for x in ("src", "dst", "count"):
        refused(lib, compact(lib, book(), **{x: None}), "null")
    for call, size in ((fork, lib.kvo_paged_fork_workspace), (compact, lib.kvo_paged_compact_workspace)):
        n = ctypes.c_size_t(0)
        assert size(book(), ctypes.byref(n)) == kvo.KVO_OK and n.value > 0
        refused(lib, call(lib, book(), size=n.value - 1), "too small")
        refused(lib, call(lib, book(), ws=None), "too small")
        refused(lib, call(lib, book(), ws=9 * P + 16), "aligned")


def test_calls_refuse_buffers_that_meet(lib):
    """table: 128 bytes, held: 16, refs: 400."""
    for kw in (dict(held=P + 124), dict(refs=P + 112), dict(held=3 * P + 396)):
        refused(lib, reserve(lib, book(**kw)), "apart")
        refused(lib, fork(lib, book(**kw)), "apart")
    for want in (P, P + 124, 2 * P, 3 * P + 396):
        refused(lib, reserve(lib, book(), want), "apart")
    for kw in (dict(src=P), dict(dst=2 * P + 4), dict(count=3 * P), dict(dst=6 * P + 12), dict(parent=6 * P), dict(keep=P), dict(ws=P),
               dict(keep=9 * P), dict(count=4 * P + 12)):
        refused(lib, fork(lib, book(), **kw), "apart")
    for kw in (dict(src=P), dict(dst=3 * P), dict(count=2 * P), dict(dst=6 * P + 196), dict(ws=P), dict(table_out=P + 4), dict(refs_out=3 * P + 16),
               dict(table_out=3 * P), dict(refs_out=P), dict(table_out=2 * P - 4), dict(table_out=6 * P), dict(table_out=4 * P, refs_out=4 * P)):
        refused(lib, compact(lib, book(), **kw), "apart")


def cache(**kw):
    a = dict(k=P, v=2 * P, ks=3 * P, vs=4 * P, hkv=2, d=64, page=16, n_pages=8, fmt=1)
    a.update(kw)
    return kvo._PagedCache(a["k"], a["v"], a["ks"], a["vs"], None, 0, a["hkv"], a["d"], a["page"], a["n_pages"], 0, a["fmt"])


@pytest.mark.parametrize("kw,call,frag", [
    (dict(d=96), {}, "head_dim"), (dict(page=48), {}, "page_size"), (dict(n_pages=0), {}, "n_pages"), (dict(fmt=3), {}, "format"),
    (dict(k=None), {}, "null"), (dict(ks=None), {}, "k_scale"), (dict(v=2 * P + 8), {}, "aligned"), ({}, dict(layers=-1), "layers"),
    ({}, dict(moves=-1), "moves"), ({}, dict(layers=70000), "layers"), ({}, dict(src=None), "null"), ({}, dict(dst=None), "null"),
    (dict(v=P), {}, "apart"), (dict(v=P + 16384), dict(layers=2), "apart"), (dict(vs=3 * P), {}, "apart"), ({}, dict(src=P), "apart"),
    ({}, dict(count=4 * P + 60), "apart"), (dict(hkv=2 ** 17, page=128, d=128, n_pages=1, fmt=0), {}, "2^30")])
def test_copy_refuses(lib, kw, call, frag):
    a = dict(layers=1, src=5 * P, dst=6 * P, moves=3, count=None)
    a.update(call)
    refused(lib, lib.kvo_paged_copy(cache(**kw), a["layers"], a["src"], a["dst"], a["moves"], a["count"], None, None), frag)


def test_nothing_to_copy(lib):
    assert lib.kvo_paged_copy(cache(), 0, None, None, 3, None, None, None) == kvo.KVO_OK
    assert lib.kvo_paged_copy(cache(), 2, None, None, 0, None, None, None) == kvo.KVO_OK
    assert lib.kvo_paged_reserve(book(batch=0, table=None, held=None), None, None, None) == kvo.KVO_OK


def test_wrappers_check_buffers():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pool = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.paged_reserve(i(2, 3), i(2), i(4), i(2), 16)
    with pytest.raises(kvo.KvoError, match="held must have shape"):
        kvo.paged_fork(i(2, 3), i(3), i(4), i(2), i(2), 16)
    with pytest.raises(kvo.KvoError, match="must be torch.int32"):
        kvo.paged_compact(i(2, 3).long(), i(2), i(4))
    with pytest.raises(kvo.KvoError, match="table must be"):
        kvo.paged_compact(i(6), i(2), i(4))
    with pytest.raises(kvo.KvoError, match="table_out must have shape"):
        kvo.paged_compact(i(2, 3), i(2), i(4), i(2, 4))
    with pytest.raises(kvo.KvoError, match="refs must be contiguous"):
        kvo.paged_reserve(i(2, 3), i(2), i(8)[::2], i(2), 16)
    with pytest.raises(kvo.KvoError, match="pages must be"):
        kvo.paged_copy(pool[0], pool[0], i(1), i(1))
    with pytest.raises(kvo.KvoError, match="dst must have shape"):
        kvo.paged_copy(pool, pool.clone(), i(1), i(2))
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.paged_copy(pool, pool.clone(), i(1), i(1))
