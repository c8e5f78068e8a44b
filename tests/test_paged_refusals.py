"""What the rotary and paged-cache calls refuse, on the host, before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

from sparse_kv_cache_landmark_gb300 import kvo


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_landmark_gb300 import build
    build.build()
    return kvo.lib()


P = 4096          # an aligned address that is never read


def refused(lib, st, frag):
    assert st == kvo.KVO_ERR_INVALID
    assert frag in lib.kvo_last_error(None).decode()


@pytest.mark.parametrize("kw,frag", [
    (dict(tokens=-1), "tokens"), (dict(heads=0), "heads"), (dict(head_dim=24), "head_dim"), (dict(rot=8), "rot_dim"),
    (dict(rot=144), "rot_dim"), (dict(x=None), "null"), (dict(out=None), "null"), (dict(pos=None), "null"),
    (dict(freq=None), "null"), (dict(x=P + 8), "aligned"), (dict(xs=132), "strides"), (dict(out=P, os=256), "in place")])
def test_rope_refuses(lib, kw, frag):
    a = dict(x=P, xs=128, xh=128, out=2 * P, os=128, oh=128, pos=P, freq=P, tokens=4, heads=1, head_dim=128, rot=128)
    a.update(kw)
    refused(lib, lib.kvo_rope(a["x"], a["xs"], a["xh"], a["out"], a["os"], a["oh"], a["pos"], a["freq"], a["tokens"],
                              a["heads"], a["head_dim"], a["rot"], 0, 1.0, None), frag)


def test_nothing_to_do_launches_nothing(lib):
    assert lib.kvo_rope(None, 0, 0, None, 0, 0, None, None, 0, 1, 128, 128, 0, 1.0, None) == kvo.KVO_OK
    c = cache()
    assert lib.kvo_paged_append(c, None, 0, None, 0, 0, None, None, None, 0, 0, 1.0, None, 0, 0, None, None, None,
                                None) == kvo.KVO_OK
    c.batch = 0
    assert lib.kvo_paged_attn(c, None, 8, None, 0, None, None, 0, None, None, None, 0, None, None) == kvo.KVO_OK


def cache(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, table=P, batch=2, hkv=2, d=128, page=32, n_pages=8, max_pages=4, fmt=1)
    a.update(kw)
    return kvo._PagedCache(a["k"], a["v"], a["ks"], a["vs"], a["table"], a["batch"], a["hkv"], a["d"], a["page"],
                           a["n_pages"], a["max_pages"], a["fmt"])


BAD_CACHES = [(dict(batch=-1), "batch"), (dict(hkv=0), "n_kv_heads"), (dict(d=96), "head_dim"), (dict(page=48), "page_size"),
              (dict(n_pages=0), "n_pages"), (dict(max_pages=0), "max_pages"), (dict(fmt=2), "format"),
              (dict(k=None), "null"), (dict(table=None), "null"), (dict(v=P + 4), "aligned"), (dict(ks=None), "k_scale"),
              (dict(max_pages=2 ** 27), "30 bits"), (dict(n_pages=2 ** 27), "31 bits")]


@pytest.mark.parametrize("kw,frag", BAD_CACHES)
def test_both_calls_refuse_bad_caches(lib, kw, frag):
    c = cache(**kw)
    refused(lib, lib.kvo_paged_append(c, P, 256, P, 256, 2, None, P, None, 0, 0, 1.0, None, 0, 0, None, None, None, None), frag)
    refused(lib, lib.kvo_paged_attn(c, P, 8, P, 0, None, None, 0, P, P, P, 1 << 30, None, None), frag)
    n = ctypes.c_size_t(7)
    refused(lib, lib.kvo_paged_attn_workspace(c, 8, 0, 0, ctypes.byref(n)), frag)
    assert n.value == 0


@pytest.mark.parametrize("kw,frag", [
    (dict(tokens=-1), "tokens"), (dict(tokens=3), "appends one token"), (dict(k=None), "null"), (dict(start=None), "null"),
    (dict(freq=P, rot=8), "rot_dim"), (dict(freq=P, rot=256), "rot_dim"), (dict(q=P, q_out=None), "q_out"),
    (dict(q=P, q_out=P, hq=0), "n_q_heads"), (dict(v=P + 2), "aligned"), (dict(kt=250), "strides")])
def test_append_refuses(lib, kw, frag):
    a = dict(k=P, kt=256, v=P, tokens=2, start=P, freq=None, rot=0, q=None, hq=8, q_out=None)
    a.update(kw)
    refused(lib, lib.kvo_paged_append(cache(), a["k"], a["kt"], a["v"], 256, a["tokens"], None, a["start"], a["freq"],
                                      a["rot"], 0, 1.0, a["q"], 1024, a["hq"], a["q_out"], None, None, None), frag)
    refused(lib, lib.kvo_paged_append(None, P, 256, P, 256, 2, None, P, None, 0, 0, 1.0, None, 0, 0, None, None, None,
                                      None), "null cache")


@pytest.mark.parametrize("kw,frag", [
    (dict(hq=7), "multiple"), (dict(hq=34), "<= 16"), (dict(q=None), "null"), (dict(lens=None), "null"),
    (dict(o=None), "null"), (dict(ws=None, mp=8192), "too small"), (dict(max_len=-1), "max_len"),
    (dict(blocks=P, n=0), "n_blocks"), (dict(counts=P), "counts"), (dict(q=P + 2), "aligned"),
    (dict(ws=P + 16), "aligned"), (dict(size=64, mp=8192), "too small"),
    (dict(blocks=P, n=2 ** 28), "30 bits")])
def test_attention_refuses(lib, kw, frag):
    a = dict(q=P, hq=8, lens=P, max_len=0, blocks=None, counts=None, n=0, o=P, ws=P, size=1 << 30, mp=4)
    a.update(kw)
    refused(lib, lib.kvo_paged_attn(cache(max_pages=a["mp"]), a["q"], a["hq"], a["lens"], a["max_len"], a["blocks"], a["counts"], a["n"],
                                    a["o"], P, a["ws"], a["size"], None, None), frag)


def test_workspace_grows_with_the_work(lib):
    n = ctypes.c_size_t(0)
    sizes = []
    for max_len in (1, 128, 100000, 0):
        assert lib.kvo_paged_attn_workspace(cache(max_pages=8192), 8, 0, max_len, ctypes.byref(n)) == kvo.KVO_OK
        sizes.append(n.value)
    assert sizes[0] == sizes[1] == 0 < sizes[2] <= sizes[3]


def test_wrappers_check_buffers():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    freq, amp = kvo.rope_frequencies(64, device="cpu")
    assert amp == 1.0 and freq.shape == (32,)
    with pytest.raises(kvo.KvoError, match="bfloat16"):
        kvo.rope(torch.zeros(2, 1, 64), i(2), freq)
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.rope(bf(2, 1, 64), i(2), freq)
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.paged_append(bf(2, 1, 64), bf(2, 1, 64), bf(4, 1, 16, 64), bf(4, 1, 16, 64), i(2, 2), i(2))
    with pytest.raises(kvo.KvoError, match="pages must be"):
        kvo.paged_attn(bf(2, 4, 64), bf(4, 16, 64), bf(4, 16, 64), i(2, 2), i(2))
    with pytest.raises(kvo.KvoError, match="bfloat16 or float8"):
        kvo.paged_attn(bf(2, 4, 64), i(4, 1, 16, 64), i(4, 1, 16, 64), i(2, 2), i(2))
    for bad in (dict(scaling="cubic"), dict(factor=0.0), dict(rot_dim=20), dict(base=1.0), dict(low=4.0, high=1.0)):
        with pytest.raises(kvo.KvoError):
            kvo.rope_frequencies(**{**dict(rot_dim=64, device="cpu"), **bad})


def test_rope_frequencies():
    """Turns per position in units of 2^-64: base^(-2i/rot) radians, and what each scaling leaves alone or divides."""
    import math
    turns = lambda t: [(x % 2 ** 64) / 2.0 ** 64 for x in t.tolist()]
    plain = turns(kvo.rope_frequencies(128, 500000.0, device="cpu")[0])
    for i, f in enumerate(plain):
        assert math.isclose(f, 500000.0 ** (-2 * i / 128) / (2 * math.pi), rel_tol=1e-12)
    lin = turns(kvo.rope_frequencies(128, 500000.0, "linear", 4.0, device="cpu")[0])
    assert all(math.isclose(4 * a, b, rel_tol=1e-12) for a, b in zip(lin, plain))
    for kind in ("banded", "ramp"):
        f, amp = kvo.rope_frequencies(128, 500000.0, kind, 8.0, original_len=8192, low=1.0, high=4.0, device="cpu")
        f = turns(f)
        fast = [i for i, p in enumerate(plain) if p * 8192 > 8.0]
        slow = [i for i, p in enumerate(plain) if p * 8192 < 0.5]
        assert fast and slow
        assert all(math.isclose(f[i], plain[i], rel_tol=1e-12) for i in fast)
        assert all(math.isclose(8 * f[i], plain[i], rel_tol=1e-12) for i in slow)
        assert all(f[i] <= plain[i] * (1 + 1e-12) and 8 * f[i] >= plain[i] * (1 - 1e-12) for i in range(64))
        assert math.isclose(amp, 1.0 if kind == "banded" else 0.1 * math.log(8.0) + 1.0)


@pytest.mark.parametrize("kw,frag", [
    (dict(batch=-1), "batch"), (dict(tq=-1), "total_q"), (dict(hq=7), "multiple"), (dict(hkv=0), "multiple"),
    (dict(hq=34), "<= 16"), (dict(d=96), "head_dim"), (dict(q=None), "null"), (dict(k=None), "null"),
    (dict(cu_q=None), "null"), (dict(o=None), "null"), (dict(v=P + 8), "aligned"), (dict(qs=1028), "strides"),
    (dict(ks=128), "cover"), (dict(qs=1 << 40), "2^38")])
def test_prompt_attention_refuses(lib, kw, frag):
    a = dict(q=P, qs=1024, k=P, ks=256, v=P, cu_q=P, batch=2, tq=10, hq=8, hkv=2, d=128, o=P)
    a.update(kw)
    refused(lib, lib.kvo_prompt_attn(a["q"], a["qs"], a["k"], a["ks"], a["v"], 256, a["cu_q"], P, a["batch"], a["tq"],
                                     10, a["hq"], a["hkv"], a["d"], 1, a["o"], P, None, None), frag)


def test_prompt_attention_without_tokens(lib):
    assert lib.kvo_prompt_attn(None, 0, None, 0, None, 0, None, None, 0, 5, 5, 8, 2, 128, 1, None, None, None,
                               None) == kvo.KVO_OK
    assert lib.kvo_prompt_attn(None, 0, None, 0, None, 0, None, None, 3, 0, 5, 8, 2, 128, 1, None, None, None,
                               None) == kvo.KVO_OK
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(kvo.KvoError, match="CUDA device"):
        kvo.prompt_attn(bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64), cu)


@pytest.mark.parametrize("kw", [dict(ot=0), dict(oh=0), dict(ot=0, oh=0)])
def test_rope_refuses_outputs_that_share_rows(lib, kw):
    a = dict(ot=256, oh=128)
    a.update(kw)
    refused(lib, lib.kvo_rope(P, 256, 128, 2 * P, a["ot"], a["oh"], P, P, 4, 2, 128, 128, 0, 1.0, None), "share memory")


@pytest.mark.parametrize("kw,frag", [
    (dict(k_out=P + 128), "apart"), (dict(k_out=P, kt=512), "apart"), (dict(k_out=2 * P), "apart"),
    (dict(q_out=3 * P + 1024), "apart"), (dict(q_out=3 * P, qt=2048), "apart"), (dict(q_out=P), "apart"),
    (dict(k_out=3 * P), "apart"), (dict(q_out=5 * P, k_out=5 * P + 1024), "must not overlap")])
def test_append_refuses_overlapping_outputs(lib, kw, frag):
    """Two tokens of 2 and 8 heads of 128: rows of 512 and 2048 bytes; k, v and q at P, 2 P and 3 P."""
    a = dict(kt=256, qt=1024, q_out=4 * P, k_out=6 * P)
    a.update(kw)
    refused(lib, lib.kvo_paged_append(cache(), P, a["kt"], 2 * P, 256, 2, None, P, None, 0, 0, 1.0, 3 * P, a["qt"], 8,
                                      a["q_out"], a["k_out"], None, None), frag)


def test_attention_refuses_outputs_over_inputs(lib):
    for o in (P, P + 1024, P - 2048):                   # q: 2 x 8 x 128 values, 4096 bytes
        refused(lib, lib.kvo_paged_attn(cache(), P, 8, P, 0, None, None, 0, o, P, None, 0, None, None), "overlap q")
    for o in (16 * P, 32 * P, 48 * P, 48 * P - 256):
        refused(lib, lib.kvo_prompt_attn(16 * P, 1024, 32 * P, 256, 48 * P, 256, P, P, 2, 10, 10, 8, 2, 128, 1, o, P, None,
                                         None), "overlap")


def test_calls_for_no_requests(lib):
    """A table without rows has no address."""
    c = cache(batch=0, table=None)
    assert lib.kvo_paged_attn(c, None, 8, None, 0, None, None, 0, None, None, None, 0, None, None) == kvo.KVO_OK
    assert lib.kvo_paged_append(c, None, 256, None, 256, 0, None, None, None, 0, 0, 1.0, None, 0, 0, None, None, None,
                                None) == kvo.KVO_OK
    assert lib.kvo_paged_append(c, P, 256, P, 256, 3, P, P, None, 0, 0, 1.0, None, 0, 0, None, None, None,
                                None) == kvo.KVO_OK
    refused(lib, lib.kvo_paged_append(c, P, 256, P, 256, 3, None, P, None, 0, 0, 1.0, None, 0, 0, None, None, None, None),
            "tokens must equal batch")


@pytest.mark.parametrize("limit,skip", [(999999, -1), (10 ** 10 + 1, -1), (10 ** 9, -2)])
def test_wait_switch_refuses_bad_limits(limit, skip):
    with pytest.raises(kvo.KvoError, match="limit_ns"):
        kvo.set_call_wait_test(limit, skip)
    kvo.set_call_wait_test()


# x: 8 heads of 128 of a projection of 22, 4 tokens, at 16 P
@pytest.mark.parametrize("out,ot,oh,frag", [
    (16 * P + 4 * 256, 2816, 128, "apart"),                             # heads 4 .. 11 of the same projection
    (16 * P - 256, 2816, 128, "apart"),                                # one head before
    (16 * P + 16, 2816, 128, "apart"),                                 # 8 values further
    (16 * P + 2816 * 2, 2816, 128, "apart"),                           # one token further
    (16 * P + 7 * 256, 2816, 256, "apart"),                            # every other head from the last one on
    (16 * P + 8 * 256, 1024, 128, "apart"),                            # contiguous, across the rows of x
    (64 * P, 1024, 64, "share memory"), (64 * P, 896, 128, "share memory"), (64 * P, 64, 4 * 128, "share memory"),
    (64 * P, 128, 256, "share memory"), (64 * P, -120, 1024, "share memory"), (64 * P, 1024, -120, "share memory")])
def test_rope_refuses_overlaps(lib, out, ot, oh, frag):
    refused(lib, lib.kvo_rope(16 * P, 2816, 128, out, ot, oh, P, P, 4, 8, 128, 128, 0, 1.0, None), frag)


APART = dict(k=64 * P, v=96 * P, ks=128 * P, vs=129 * P, table=130 * P)      # pages of 16 P bytes, scales of 64, a table of 32


@pytest.mark.parametrize("kw,frag", [
    (dict(v=64 * P), "of their own"), (dict(v=80 * P - 16), "of their own"), (dict(k=96 * P + 1024), "of their own"),
    (dict(vs=128 * P), "of their own"), (dict(vs=128 * P + 60), "of their own"),
    (dict(k_out=64 * P + 512), "nothing else"), (dict(k_out=112 * P - 16), "nothing else"), (dict(q_out=96 * P), "nothing else"),
    (dict(q_out=128 * P), "nothing else"), (dict(k_out=129 * P + 48), "nothing else"), (dict(k_out=130 * P + 16), "nothing else"),
    (dict(q_out=131 * P), "nothing else"), (dict(k_out=132 * P), "nothing else"), (dict(k_out=133 * P), "nothing else")])
def test_append_refuses_shared_pools_and_outputs_over_the_cache(lib, kw, frag):
    """start, cu and freq at 131 P, 132 P and 133 P."""
    c = cache(**{**APART, **{k: v for k, v in kw.items() if k in APART}})
    a = {**dict(q_out=4 * P, k_out=6 * P), **kw}
    refused(lib, lib.kvo_paged_append(c, P, 256, 2 * P, 256, 2, 132 * P, 131 * P, 133 * P, 128, 0, 1.0, 3 * P, 1024, 8, a["q_out"],
                                      a["k_out"], None, None), frag)


@pytest.mark.parametrize("kw", [dict(o=x * P) for x in (64, 128, 129, 130, 147, 148, 149, 400, 1000)]
                         + [dict(lse=x * P) for x in (1, 64, 96, 128, 130, 147, 148, 149, 1000, 300)] + [dict(lse=301 * P - 4)]
                         + [dict(o=112 * P - 16), dict(o=300 * P, lse=300 * P), dict(ws=96 * P), dict(ws=140 * P), dict(ws=P)])
def test_attention_refuses_outputs_over_what_it_reads(lib, kw):
    """q at P, pages, scales and table as above (the table long), lens, counts and blocks at 147 P to 149 P, the workspace
    from 400 P on, o at 300 P and lse at 302 P."""
    c = cache(**{**APART, "max_pages": 8192})
    n = ctypes.c_size_t(0)
    assert lib.kvo_paged_attn_workspace(c, 8, 2000, 0, ctypes.byref(n)) == kvo.KVO_OK and 1000 * P < n.value < 2000 * P
    a = {**dict(o=300 * P, lse=302 * P, ws=400 * P), **kw}
    refused(lib, lib.kvo_paged_attn(c, P, 8, 147 * P, 0, 149 * P, 148 * P, 2000, a["o"], a["lse"], a["ws"], n.value, None, None),
            "o, lse and the workspace must be apart")


@pytest.mark.parametrize("o,lse", [(P, None), (None, P + 8), (None, 16 * P), (None, 32 * P), (None, 48 * P + 4), (None, 64 * P + 20476)])
def test_prompt_attention_refuses_outputs_over_what_it_reads(lib, o, lse):
    """10 tokens; q, k, v at 16 P, 32 P and 48 P, offsets at P, o at 64 P."""
    refused(lib, lib.kvo_prompt_attn(16 * P, 1024, 32 * P, 256, 48 * P, 256, P, P, 2, 10, 10, 8, 2, 128, 1, o or 64 * P, lse or 80 * P,
                                     None, None), "o and lse must be apart")
