"""What attention of new tokens over a paged cache refuses, on the host, before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo

P = 1 << 24       # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_landmark_gb300 import build
    build.build()
    return kvo.lib()


def refused(lib, st, frag):
    assert st == kvo.KVO_ERR_INVALID
    assert frag in lib.kvo_last_error(None).decode()


def cache(**kw):
    a = dict(k=P, v=2 * P, ks=3 * P, vs=4 * P, table=5 * P, batch=2, hkv=2, d=128, page=32, n_pages=8, max_pages=4, fmt=1)
    a.update(kw)
    return kvo._PagedCache(a["k"], a["v"], a["ks"], a["vs"], a["table"], a["batch"], a["hkv"], a["d"], a["page"], a["n_pages"],
                           a["max_pages"], a["fmt"])


def call(lib, c=None, **kw):
    a = dict(q=6 * P, stride=1024, total=40, hq=8, cu=7 * P, lens=8 * P, max_new=0, max_len=0, o=9 * P, lse=10 * P, ws=11 * P, size=1 << 30)
    a.update(kw)
    return lib.kvo_paged_chunk_attn(c or cache(), a["q"], a["stride"], a["total"], a["hq"], a["cu"], a["lens"], a["max_new"], a["max_len"],
                                    a["o"], a["lse"], a["ws"], a["size"], None, None)


def size(lib, c=None, hq=8, total=40, max_new=0, max_len=0):
    n = ctypes.c_size_t(7)
    st = lib.kvo_paged_chunk_attn_workspace(c or cache(), hq, total, max_new, max_len, ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("kw,frag", [
    (dict(batch=-1), "batch"), (dict(hkv=0), "n_kv_heads"), (dict(d=96), "head_dim"), (dict(page=48), "page_size"), (dict(n_pages=0), "n_pages"),
    (dict(max_pages=0), "max_pages"), (dict(fmt=2), "format"), (dict(k=None), "null"), (dict(table=None), "null"), (dict(v=2 * P + 4), "aligned"),
    (dict(ks=None), "k_scale"), (dict(max_pages=2 ** 27), "30 bits"), (dict(n_pages=2 ** 27), "31 bits")])
def test_bad_caches(lib, kw, frag):
    for max_new in (0, 4):
        refused(lib, call(lib, cache(**kw), max_new=max_new), frag)
        st, n = size(lib, cache(**kw), max_new=max_new)
        refused(lib, st, frag)
        assert n == 0


@pytest.mark.parametrize("max_new", [0, 4])         # both kernels
@pytest.mark.parametrize("kw,frag", [
    (dict(hq=7), "multiple"), (dict(hq=1), "multiple"), (dict(hq=34), "<= 16"), (dict(total=-1), "total_q"), (dict(total=2 ** 30 + 1), "total_q"),
    (dict(total=2 ** 30, hq=32), "total_q"), (dict(max_new=-1), "max_new"), (dict(max_len=-1), "max_len"), (dict(q=None), "null"),
    (dict(o=None), "null"), (dict(cu=None), "null"), (dict(lens=None), "null"), (dict(q=6 * P + 8), "aligned"), (dict(o=9 * P + 2), "aligned"),
    (dict(ws=11 * P + 16), "aligned"), (dict(stride=1028), "multiples of 8"), (dict(stride=1016), "cover"), (dict(stride=-1024), "cover"),
    (dict(stride=2 ** 38 + 8), "2^38")])
def test_bad_calls(lib, kw, frag, max_new):
    refused(lib, call(lib, **{**dict(max_new=max_new), **kw}), frag)


def test_workspaces(lib):
    """Long chunks always need one; few new tokens need one where a request's keys may be split."""
    for c, kw in ((cache(), {}), (cache(fmt=0), {}), (cache(d=64), dict(hq=16)), (cache(n_pages=10 ** 5, max_pages=10 ** 4), dict(max_new=2))):
        st, n = size(lib, c, **kw)
        assert st == kvo.KVO_OK and n > 0
        refused(lib, call(lib, c, size=n - 1, **kw), "too small")
        refused(lib, call(lib, c, ws=None, **kw), "too small")
    assert size(lib, max_new=4, max_len=1) == (kvo.KVO_OK, 0)
    refused(lib, lib.kvo_paged_chunk_attn_workspace(cache(), 8, 40, 0, 0, None), "null")
    # the pieces of q are laid out for e4m3 pages: two bytes to a value and one to a row
    assert size(lib, total=2 ** 12)[1] - size(lib, total=2 ** 11)[1] == 2 ** 11 * 8 * (2 * 128 + 1)
    assert size(lib, cache(fmt=0), total=2 ** 12) == size(lib, cache(fmt=0), total=2 ** 11)


@pytest.mark.parametrize("max_new", [0, 4])
def test_buffers_that_meet(lib, max_new):
    """q and o: 40 x 1024 of two bytes; lse: 40 x 8 of four; a pool: 8 x 2 x 32 x 128 bytes; scales 64, table 32, lens 8, cu 12 bytes."""
    for o in (6 * P, 6 * P + 81904, P, 2 * P + 65520, 3 * P, 4 * P + 48, 5 * P + 16, 7 * P, 8 * P, 10 * P + 1264, 10 * P - 16):
        refused(lib, call(lib, o=o, max_new=max_new), "apart")
    for lse in (6 * P + 81916, P, 2 * P + 65532, 3 * P + 60, 4 * P, 5 * P + 28, 7 * P + 8, 8 * P + 4, 9 * P + 81916):
        refused(lib, call(lib, lse=lse, max_new=max_new), "apart")
    for ws in (6 * P, P, 2 * P + 65280, 3 * P, 4 * P, 5 * P, 7 * P, 8 * P, 9 * P, 10 * P):
        refused(lib, call(lib, cache(max_pages=4000, n_pages=8, table=100 * P), ws=ws, max_new=max_new), "apart")


def test_nothing_to_do(lib):
    assert call(lib, total=0, q=None, o=None, ws=None) == kvo.KVO_OK
    assert call(lib, cache(batch=0), q=None, cu=None, lens=None) == kvo.KVO_OK


def test_wrapper_checks_buffers():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pool = bf(4, 1, 16, 64)
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.paged_chunk_attn(bf(6, 4, 64), pool, pool.clone(), i(2, 2), i(2), i(3))
    with pytest.raises(kvo.KvoError, match="bfloat16"):
        kvo.paged_chunk_attn(bf(6, 4, 64).float(), pool, pool.clone(), i(2, 2), i(2), i(3))
    with pytest.raises(kvo.KvoError, match="pages must be"):
        kvo.paged_chunk_attn(bf(6, 4, 64), pool[0], pool[0], i(2, 2), i(2), i(3))
    with pytest.raises(kvo.KvoError, match="q must have shape"):
        kvo.paged_chunk_attn(bf(6, 4, 128), pool, pool.clone(), i(2, 2), i(2), i(3))
    with pytest.raises(kvo.KvoError, match="lens must have shape"):
        kvo.paged_chunk_attn(bf(6, 4, 64), pool, pool.clone(), i(2, 2), i(3), i(3))
    with pytest.raises(kvo.KvoError, match="cu must have shape"):
        kvo.paged_chunk_attn(bf(6, 4, 64), pool, pool.clone(), i(2, 2), i(2), i(2))
    with pytest.raises(kvo.KvoError, match="pages must be"):
        kvo.paged_chunk_attn(bf(6, 4, 64), pool, pool.clone(), i(4), i(2), i(3))
