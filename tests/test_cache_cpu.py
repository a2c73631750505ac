"""The paged cache's refusals and sizes: everything that is decided before a
launch, so no GPU is needed."""

import ctypes

import pytest
import torch

from coreset_attention_approximation_b200 import wildcat


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(wildcat.LIB_PATH):
        from coreset_attention_approximation_b200 import build

        build.build()
    return wildcat.lib()


def shape(**kw):
    base = dict(batch=2, hq=8, hkv=2, d=64, dv=64, dtype=wildcat.WC_BF16, page=16, n_pages=40, max_pages=10,
                scale=0.0, k_page=0, k_head=0, k_token=0, v_page=0, v_head=0, v_token=0)
    base.update(kw)
    return wildcat.WcCache(**base)


OK, ODD, BIG = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), 1 << 40
DENSE = dict(k_page=2048, k_head=1024, k_token=64, v_page=2048, v_head=1024, v_token=64)


def test_workspace_sizes(lib):
    n = lib.wc_cache_workspace_bytes(ctypes.byref(shape()), 0)
    a = lib.wc_cache_workspace_bytes(ctypes.byref(shape()), 1)
    assert n > 0 and n % 256 == 0 and a - n >= 4 * 2 * 8 * 160
    assert lib.wc_cache_workspace_bytes(ctypes.byref(shape(**DENSE)), 0) == n
    assert lib.wc_cache_workspace_bytes(ctypes.byref(shape()), 2) == 0
    assert lib.wc_cache_workspace_bytes(None, 0) == 0


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(hkv=0), dict(hq=3), dict(hq=0), dict(d=12), dict(d=0), dict(d=264),
    dict(dv=4), dict(dtype=2), dict(page=0), dict(page=65537), dict(n_pages=0), dict(max_pages=0),
    dict(max_pages=1 << 27), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(batch=65535, hq=512, hkv=2),
    dict(DENSE, k_token=60), dict(DENSE, k_token=32), dict(DENSE, k_head=0), dict(DENSE, v_page=8),
    dict(DENSE, v_token=-64), dict(DENSE, k_page=2052),
])
def test_invalid_caches_are_refused_by_every_call(lib, kw):
    s = shape(**kw)
    assert lib.wc_cache_workspace_bytes(ctypes.byref(s), 0) == 0
    r = wildcat.WcRowStrides(128, 64, 64)
    assert lib.wc_cache_append(ctypes.byref(s), 1, OK, ctypes.byref(r), OK, ctypes.byref(r), OK, OK, OK, OK, OK, OK,
                               OK, BIG, None) == 1
    assert lib.wc_cache_attend(ctypes.byref(s), OK, 512, 64, OK, OK, OK, OK, 0, None, None, None, OK, OK, OK, OK, BIG,
                               None) == 1
    assert lib.wc_cache_evict(ctypes.byref(s), 5, 0, 0, OK, OK, OK, None, OK, OK, None, OK, OK, OK, BIG, None) == 1


def test_strides_beyond_32_bits_are_unsupported(lib):
    for kw in (dict(k_page=1 << 31), dict(v_page=1 << 32), dict(k_token=1 << 31, k_head=64)):
        s = shape(**dict(DENSE, **kw))
        assert lib.wc_cache_workspace_bytes(ctypes.byref(s), 0) == 0
        assert lib.wc_cache_attend(ctypes.byref(s), OK, 512, 64, OK, OK, OK, OK, 0, None, None, None, OK, OK, OK, OK,
                                   BIG, None) == 4
    # heads may lie further apart
    s = shape(**dict(DENSE, k_head=1 << 33, v_head=1 << 33))
    assert lib.wc_cache_workspace_bytes(ctypes.byref(s), 0) > 0


def test_append_refusals(lib):
    s, r = shape(), wildcat.WcRowStrides(128, 64, 64)

    def call(t=1, K=OK, ks=r, V=OK, vs=r, pos=OK, count=None, k=OK, v=OK, table=OK, scores=OK, ws=OK, n=BIG):
        ref = lambda x: None if x is None else ctypes.byref(x)
        return lib.wc_cache_append(ctypes.byref(s), t, K, ref(ks), V, ref(vs), pos, count, k, v, table, scores, ws, n,
                                   None)

    assert call(t=-1) == 1 and call(t=(1 << 30) + 1) == 1
    for name in ("K", "ks", "V", "vs", "pos", "k", "v", "table", "ws"):
        assert call(**{name: None}) == 1, name
    for name in ("K", "V", "k", "v", "ws"):
        assert call(**{name: ODD}) == 1, name
    assert call(pos=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert call(ks=wildcat.WcRowStrides(128, 64, 63)) == 1 and call(vs=wildcat.WcRowStrides(4, 64, 64)) == 1
    assert call(n=256) == 5
    assert call(t=0) == 0                          # nothing to write: no launch


def test_attend_refusals(lib):
    s = shape()

    def call(Q=OK, k=OK, v=OK, table=OK, lens=OK, r=0, Ks=None, W=None, rank=None, out=OK, lse=None, scores=None,
             ws=OK, n=BIG):
        return lib.wc_cache_attend(ctypes.byref(s), Q, 512, 64, k, v, table, lens, r, Ks, W, rank, out, lse, scores,
                                   ws, n, None)

    for name in ("Q", "k", "v", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == 1, name
    for name in ("k", "v", "ws"):
        assert call(**{name: ODD}) == 1, name
    assert call(Q=ctypes.c_void_p((1 << 20) + 1)) == 1
    assert call(out=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert call(r=-1) == 1 and call(r=4097, Ks=OK, W=OK) == 1
    assert call(r=4, W=OK) == 1 and call(r=4, Ks=OK) == 1 and call(r=4, Ks=ODD, W=OK) == 1
    assert call(r=4, Ks=OK, W=ODD) == 1
    small = lib.wc_cache_workspace_bytes(ctypes.byref(s), 0)
    assert call(n=small - 1) == 5
    assert call(scores=OK, n=small) == 5           # accumulation needs the larger workspace


def test_evict_refusals(lib):
    s = shape()

    def call(keep=5, sink=0, recent=0, k=OK, v=OK, table=OK, into=None, lens=OK, scores=OK, to=None, idx=OK,
             lens_out=OK, ws=OK, n=BIG):
        return lib.wc_cache_evict(ctypes.byref(s), keep, sink, recent, k, v, table, into, lens, scores, to, idx,
                                  lens_out, ws, n, None)

    for kw in (dict(keep=0), dict(keep=161), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=3),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert call(**kw) == 1, kw
    for name in ("k", "v", "table", "lens", "scores", "idx", "lens_out", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(into=ctypes.c_void_p((1 << 20) + 1)) == 1
    assert call(n=1024) == 5


def test_the_binding_refuses_before_it_calls():
    B, hkv, page, d = 2, 2, 16, 64
    k = torch.zeros(8, hkv, page, d)
    table = torch.zeros(B, 4, dtype=torch.int32)
    new = lambda **kw: wildcat.PagedCache(**dict(dict(k_pages=k, v_pages=k, table=table, hq=4), **kw))
    scores = torch.zeros(B, hkv, 64)
    for kw in (dict(k_pages=k[0]), dict(v_pages=k[:7]), dict(table=table.long()), dict(table=table[0]),
               dict(k_pages=k.half(), v_pages=k.half()), dict(v_pages=k.bfloat16()), dict(table=table.t()),
               dict(k_pages=k.transpose(2, 3)), dict(hq=3), dict(scores=scores.double()), dict(scores=scores[:1]),
               dict(k_pages=k[..., :60], v_pages=k[..., :60]), dict(scale=-1.0),
               dict(k_pages=k[:1].expand(8, hkv, page, d))):
        with pytest.raises(wildcat.WildcatError):
            new(**kw)
    with pytest.raises(wildcat.WildcatError, match="on a GPU"):
        new(scores=scores)
