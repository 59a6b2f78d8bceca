"""The operators of include/gdn_cache.h on the host (no GPU): every bad call returns its status before anything touches
CUDA, scratch sizes, and the binding's own checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

FAKE = 0x7f0000000000  # never dereferenced: validation must fail first
INV, UNS, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


def cache(layers=2, pages=10, page=16, H=2, D=64, rows=4, W=8, **ptrs):
    p = dict(pages=FAKE, scales=FAKE, table=FAKE, lens=FAKE, refs=FAKE)
    p.update(ptrs)
    return gdn._Cache(layers, pages, page, H, D, rows, W, *(p[n] for n in ("pages", "scales", "table", "lens", "refs")))


def batch(B=3, max_new=4, T=9, max_len=0, cu=FAKE, rows=None):
    return gdn._Batch(B, max_new, T, max_len, cu, rows)


CACHES = [
    (dict(layers=0), INV), (dict(pages=0), INV), (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=256), UNS), (dict(H=0), INV),
    (dict(H=4097), UNS), (dict(D=96), UNS), (dict(rows=0), INV), (dict(W=0), INV), (dict(W=2 ** 27), UNS),
    (dict(pages=2 ** 30), UNS), (dict(scales=None), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(table=FAKE + 2), INV), (dict(lens=FAKE + 1), INV), (dict(scales=FAKE + 3), INV)]
BATCHES = [(dict(B=0), INV), (dict(B=4097, rows=FAKE), UNS), (dict(B=5), INV), (dict(max_new=0), INV), (dict(T=-1), INV),
           (dict(T=2 ** 30), UNS), (dict(max_len=-1), INV), (dict(cu=None), INV), (dict(cu=FAKE + 2), INV), (dict(rows=FAKE + 1), INV)]


def append(L, c=None, b=None, layer=0, k=FAKE, v=FAKE, dtype=gdn.GDN_BF16, ks=0, vs=0, ws=FAKE, nws=256):
    return L.gdn_cache_append(ctypes.byref(c or cache()), layer, ctypes.byref(b or batch()), k, v, dtype, ks, vs, ws, nws, None)


def attend(L, c=None, b=None, layer=0, q=FAKE, dtype=gdn.GDN_BF16, Hq=4, qs=0, scale=0.1, o=FAKE, lse=FAKE, scratch=FAKE,
           n=1 << 40, ws=FAKE, nws=256):
    return L.gdn_paged_attention(ctypes.byref(c or cache()), layer, ctypes.byref(b or batch()), q, dtype, Hq, qs, scale, o, lse,
                                 scratch, n, ws, nws, None)


def update(L, c=None, nd=0, drop=None, nf=0, src=None, dst=None, grow=FAKE, granted=None, scratch=FAKE, n=1 << 40, ws=FAKE, nws=256):
    return L.gdn_cache_update(ctypes.byref(c or cache()), nd, drop, nf, src, dst, grow, granted, scratch, n, ws, nws, None)


@pytest.mark.parametrize("bad, want", CACHES)
def test_caches(L, bad, want):
    c = cache(**bad)
    assert append(L, c) == want and attend(L, c) == want and update(L, c) == want
    assert L.gdn_cache_compact(ctypes.byref(c), FAKE, FAKE, 1 << 40, FAKE, 256, None) == want
    assert L.gdn_cache_scratch_bytes(ctypes.byref(c)) == 0


@pytest.mark.parametrize("bad, want", BATCHES)
def test_batches(L, bad, want):
    assert append(L, b=batch(**bad)) == want and attend(L, b=batch(**bad)) == want


def test_null_structs(L):
    assert L.gdn_cache_append(None, 0, ctypes.byref(batch()), FAKE, FAKE, 1, 0, 0, FAKE, 256, None) == INV
    assert L.gdn_cache_append(ctypes.byref(cache()), 0, None, FAKE, FAKE, 1, 0, 0, FAKE, 256, None) == INV
    assert L.gdn_qk_norm_rope(None, *[FAKE] * 8, None) == INV
    assert L.gdn_cache_scratch_bytes(None) == 0 and L.gdn_paged_scratch_bytes(None, None, 1, 4) == 0


@pytest.mark.parametrize("bad, want", [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(dtype=5), INV), (dict(k=None), INV), (dict(v=FAKE + 8), INV), (dict(ks=64), INV),
    (dict(ks=132), INV), (dict(vs=2 ** 36), UNS), (dict(ws=None), INV), (dict(nws=128), INV), (dict(ws=FAKE + 4), INV)])
def test_append(L, bad, want):
    assert append(L, **bad) == want


@pytest.mark.parametrize("bad, want", [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(dtype=2), INV), (dict(Hq=3), INV), (dict(Hq=0), INV), (dict(Hq=258), UNS),
    (dict(q=None), INV), (dict(q=FAKE + 4), INV), (dict(o=None), INV), (dict(o=FAKE + 8), INV), (dict(lse=FAKE + 2), INV),
    (dict(qs=128), INV), (dict(qs=257), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(scale=3e38), INV),
    (dict(scratch=None), INV), (dict(scratch=FAKE + 16), INV), (dict(n=64), INV), (dict(ws=None), INV), (dict(nws=0), INV)])
def test_attention(L, bad, want):
    assert attend(L, **bad) == want


def test_too_many_rows(L):
    c = cache(H=1, D=32, W=4, rows=5000)
    assert attend(L, c, batch(B=1, max_new=2 ** 24, T=2 ** 24), Hq=128) == UNS


def test_attention_too_large(L):
    c = cache(H=4096, D=32, W=2 ** 20, rows=5000)
    assert attend(L, c, batch(B=4096, max_new=2 ** 20, T=2 ** 29), Hq=4096) == UNS


@pytest.mark.parametrize("bad, want", [
    (dict(c=cache(refs=None)), INV), (dict(c=cache(rows=16385)), UNS), (dict(nd=-1), INV), (dict(nd=1), INV), (dict(nf=1), INV),
    (dict(nf=1, src=FAKE), INV), (dict(nf=-1), INV), (dict(nd=2 ** 24 + 1, drop=FAKE), UNS), (dict(nd=1, drop=FAKE + 2), INV),
    (dict(grow=FAKE + 1), INV), (dict(granted=FAKE + 3), INV), (dict(scratch=None), INV), (dict(scratch=FAKE + 8), INV),
    (dict(n=64), INV), (dict(ws=None), INV), (dict(nws=255), INV)])
def test_update(L, bad, want):
    assert update(L, **bad) == want


def test_nothing_to_do(L):
    assert update(L, grow=None) == OK
    assert append(L, b=batch(T=0), k=None, v=None) == OK and attend(L, b=batch(T=0), q=None, o=None) == OK
    assert L.gdn_cache_compact(ctypes.byref(cache()), None, FAKE, 1 << 40, FAKE, 256, None) == INV


def test_scratch_sizes(L):
    c = cache(pages=1000)
    n = L.gdn_cache_scratch_bytes(ctypes.byref(c))
    assert n == 16 + 3 * 4000
    assert update(L, c, n=n - 1) == INV
    m = L.gdn_paged_scratch_bytes(ctypes.byref(c), ctypes.byref(batch()), gdn.GDN_BF16, 4)
    assert m > 0 and attend(L, c, n=m - 1) == INV


def rope(L, T=5, Hq=4, Hk=2, D=64, rd=64, dtype=gdn.GDN_BF16, layout=0, norm=1, eps=1e-6, mscale=1.0, strides=(0, 0, 0, 0), q=FAKE,
         k=FAKE, pos=FAKE, freq=FAKE, qw=None, kw=None, qo=FAKE + 65536, ko=FAKE + 65536):
    pr = gdn._Rope(T, Hq, Hk, D, rd, dtype, layout, norm, eps, mscale, *strides)
    return L.gdn_qk_norm_rope(ctypes.byref(pr), q, k, pos, freq, qw, kw, qo, ko, None)


@pytest.mark.parametrize("bad, want", [
    (dict(T=-1), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(D=96), UNS), (dict(rd=-16), INV), (dict(rd=24), INV),
    (dict(rd=80), INV), (dict(dtype=4), INV), (dict(layout=2), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(eps=math.inf), INV), (dict(mscale=math.nan), INV), (dict(strides=(128, 0, 0, 0)), INV), (dict(strides=(0, 129, 0, 0)), INV),
    (dict(strides=(0, 0, 2 ** 36, 0)), UNS), (dict(strides=(0, 0, 0, -128)), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(q=FAKE + 8), INV), (dict(pos=None), INV), (dict(freq=None), INV), (dict(freq=FAKE + 4), INV), (dict(pos=FAKE + 1), INV),
    (dict(qw=FAKE + 8), INV), (dict(qo=None), INV), (dict(ko=FAKE + 2), INV), (dict(qo=FAKE, strides=(512, 0, 0, 0)), INV),
    (dict(T=2 ** 31), UNS), (dict(Hq=2 ** 17), UNS)])
def test_rope(L, bad, want):
    assert rope(L, **bad) == want


def test_rope_without_tokens(L):
    assert rope(L, T=0, q=None, k=None, pos=None, qo=None, ko=None) == OK


def test_status_of_a_bad_index_is_named():
    assert gdn.status_string(INV)


def test_host_tensors_are_refused():
    q = torch.zeros(3, 4, 64, dtype=BF)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_qk_norm_rope(q, None, torch.zeros(3, dtype=torch.int32), gdn.gdn_rope_frequencies(64, device="cpu"))
    c = gdn.PagedCache.empty(1, 4, 2, 64, 2, 3, page_size=16, device="cpu")
    cu = torch.tensor([0, 1, 3], dtype=torch.int32)
    k = torch.zeros(3, 2, 64, dtype=BF)
    for call in (lambda: gdn.gdn_cache_append(k, k, c, cu), lambda: gdn.gdn_paged_attention(q, c, cu),
                 lambda: gdn.gdn_cache_update(c, grow=torch.zeros(2, dtype=torch.int32)), lambda: gdn.gdn_cache_compact(c)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_caches_of_wrong_tensors_are_refused():
    c = gdn.PagedCache.empty(1, 4, 2, 64, 2, 3, page_size=16, device="cpu")
    good = dict(pages=c.pages, scales=c.scales, table=c.table, lens=c.lens, refs=c.refs)
    made = gdn.PagedCache(**good)
    assert made.pages is c.pages and made.page_size == 16
    with pytest.raises(AttributeError):   # (the calls go to the tensors that it was made of)
        made.lens = c.lens + 1
    for name, bad in (("pages", c.pages.view(torch.uint8)), ("pages", c.pages[:, :, :1]), ("pages", c.pages.transpose(3, 4)),
                      ("scales", c.scales.double()), ("scales", c.scales[:, :3]), ("table", c.table.long()), ("table", c.table[0]),
                      ("lens", c.lens[:1]), ("refs", c.refs[:3])):
        with pytest.raises(ValueError):
            gdn.PagedCache(**{**good, name: bad})


def test_frequencies():
    f = gdn.gdn_rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and np.allclose(f, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    assert torch.equal(gdn.gdn_rope_frequencies(64, scaling="linear", factor=4.0, device="cpu"), f / 4)
    b = gdn.gdn_rope_frequencies(64, scaling="base", factor=8.0, device="cpu")
    assert b[0] == 1 and math.isclose(b[-1] * 8, f[-1], rel_tol=1e-12)
    p = gdn.gdn_rope_frequencies(64, scaling="parts", factor=8.0, original_len=4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(p[turns >= 32], f[turns >= 32]) and torch.equal(p[turns <= 1], f[turns <= 1] / 8)
    assert ((p <= f) & (p >= f / 8)).all() and gdn.gdn_rope_frequencies(0, device="cpu").shape == (0,)
    for bad in (dict(rotary_dim=24), dict(rotary_dim=64, scaling="x"), dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, base=0.0)):
        with pytest.raises(ValueError):
            gdn.gdn_rope_frequencies(device="cpu", **bad)
