"""Host-side refusals of the long-context calls, before any launch (no GPU):
the C entry points with made-up addresses that no kernel ever sees, and the
binding's checks of tensors."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, build

BAD, UNS, WS = tl.TL_ERR_INVALID_ARG, tl.TL_ERR_UNSUPPORTED, tl.TL_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def caller(fn, order, base):
    def call(**kw):
        assert set(kw) <= set(base), kw
        a = dict(base, **kw)
        return fn(*(a[n] for n in order.split()))
    return call


def test_page_bounds_refusals(lib):
    base = dict(k=256, ks=512, bt=1024, maxp=8, fn=1280, cl=1536, bnd=2048, sc=4096, B=2, hkv=2,
                d=128, P=16, ps=16, dt=tl.TL_BF16, err=None, st=None)
    b = caller(lib.tl_kv_page_bounds, "k bt maxp fn cl bnd sc B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_page_bounds_int8, "k ks bt maxp fn cl bnd sc B hkv d P ps err st", base)
    for call in (b, i):
        for name in ("k", "bt", "cl", "bnd", "sc"):
            assert call(**{name: None}) == BAD, name
        for name in ("B", "hkv", "d", "P", "ps", "maxp"):
            assert call(**{name: 0}) == BAD and call(**{name: -1}) == BAD, name
        for name, off in (("k", 264), ("bnd", 2056), ("sc", 4104), ("bt", 1026), ("cl", 1537),
                          ("fn", 1282)):
            assert call(**{name: off}) == BAD, name
        assert call(d=96) == UNS and call(ps=257) == UNS
        assert call(P=1 << 28) == UNS and call(B=1 << 20, maxp=1 << 12) == UNS
    assert b(dt=tl.TL_INT8) == UNS and b(dt=7) == UNS and b(dt=-1) == UNS
    assert i(ks=None) == BAD and i(ks=520) == BAD


def test_page_select_refusals(lib):
    base = dict(q=256, qd=tl.TL_BF16, bnd=512, sc=768, bt=1024, maxp=8, cl=1280, n=4, first=1,
                last=1, pt=1536, pl=1792, B=2, hq=8, hkv=2, d=128, P=16, ps=16, ws=2048,
                wsb=1 << 20, err=None, st=None)
    s = caller(lib.tl_kv_page_select,
               "q qd bnd sc bt maxp cl n first last pt pl B hq hkv d P ps ws wsb err st", base)
    for name in ("q", "bnd", "sc", "bt", "cl", "pt", "pl"):
        assert s(**{name: None}) == BAD, name
    for name in ("B", "hq", "hkv", "d", "P", "ps", "maxp", "n"):
        assert s(**{name: 0}) == BAD and s(**{name: -3}) == BAD, name
    assert s(hq=7) == BAD
    assert s(last=0) == BAD and s(first=-1) == BAD and s(first=4, last=1) == BAD
    assert s(first=2**31 - 1, last=2**31 - 1) == BAD
    for name, off in (("q", 264), ("bnd", 520), ("sc", 772), ("bt", 1026), ("cl", 1281),
                      ("pt", 1540), ("pl", 1796)):
        assert s(**{name: off}) == BAD, name
    assert s(qd=tl.TL_FP8_E4M3) == UNS and s(d=256) == UNS and s(hq=34) == UNS
    assert s(ps=300) == UNS and s(B=1 << 20, maxp=1 << 12) == UNS and s(n=1 << 28) == UNS
    size = tl.tl_kv_page_select_workspace_size
    need = size(2, 8, 2, 128, 8)
    assert need == 256 + 256 + 2 * 8 * 128  # 2 x 2 x 8 scores, 2 x 8 scales, the codes
    assert s(ws=None) == WS and s(ws=2064) == WS and s(wsb=need - 1) == WS
    assert size(0, 8, 2, 128, 8) == 0 and size(2, 7, 2, 128, 8) == 0
    assert size(64, 32, 8, 128, 8192) == 64 * 8 * 8192 * 4 + 64 * 32 * 4 + 64 * 32 * 128


def test_decode_pages_refusals(lib):
    base = dict(q=256, k=512, v=768, ks=12288, vs=16384, pt=1024, n=4, pl=1280, out=1536, B=2,
                hq=8, hkv=2, d=128, P=8, ps=16, sc=0.1, dt=tl.TL_BF16, ws=4096, wsb=0, err=None,
                st=None)
    a = caller(lib.tl_paged_attn_decode_pages,
               "q k v pt n pl out B hq hkv d P ps sc dt ws wsb err st", base)
    i = caller(lib.tl_paged_attn_decode_pages_int8,
               "q k v ks vs pt n pl out B hq hkv d P ps sc ws wsb err st", base)
    for call in (a, i):
        for name in ("q", "k", "v", "pt", "pl", "out"):
            assert call(**{name: None}) == BAD, name
        for name in ("B", "hq", "hkv", "d", "P", "ps", "n"):
            assert call(**{name: 0}) == BAD, name
        assert call(hq=7) == BAD and call(q=264) == BAD and call(pt=1026) == BAD
        assert call(d=96) == UNS and call(hq=34) == UNS and call(ps=272) == UNS
        assert call() == WS and call(ws=None, wsb=1 << 30) == WS
    assert a(dt=tl.TL_INT8) == UNS and a(ps=12) == UNS and a(dt=tl.TL_FP8_E4M3, d=64) == UNS
    assert i(ks=None) == BAD and i(vs=16392) == BAD and i(ps=24) == UNS and i(d=64) == UNS


def test_decode_mass_refusals(lib):
    base = dict(q=256, k=512, v=768, ks=12288, vs=16384, bt=1024, maxp=4, cl=1280, out=1536,
                m=2048, ml=64, B=2, T=1, hq=8, hkv=2, d=128, P=8, ps=16, w=0, sc=0.1,
                dt=tl.TL_BF16, ws=4096, wsb=0, err=None, st=None)
    a = caller(lib.tl_paged_attn_decode_mass,
               "q k v bt maxp cl out m ml B T hq hkv d P ps w sc dt ws wsb err st", base)
    i = caller(lib.tl_paged_attn_decode_mass_int8,
               "q k v ks vs bt maxp cl out m ml B T hq hkv d P ps w sc ws wsb err st", base)
    for call in (a, i):
        for name in ("q", "k", "v", "bt", "cl", "out", "m"):
            assert call(**{name: None, "wsb": 1 << 30}) == BAD, name
        for name in ("B", "T", "hq", "hkv", "d", "P", "ps", "maxp", "ml"):
            assert call(**{name: 0, "wsb": 1 << 30}) == BAD, name
        assert call(m=2056) == BAD and call(w=-1) == BAD and call(hq=9) == BAD
        assert call(T=5) == UNS and call(hq=34) == UNS  # more than 16 rows a KV head
        assert call(d=96, wsb=1 << 30) == UNS and call(ml=2**31 - 1) == UNS
        need = tl.tl_paged_attn_decode_mass_workspace_size(2, 1, 8, 2, 128, 64)
        assert call() == WS and call(wsb=need - 1) == WS
        assert call(ws=4112, wsb=1 << 30) == WS and call(ws=None, wsb=1 << 30) == WS
    assert a(dt=tl.TL_F32, T=2, wsb=1 << 30) == UNS and a(dt=tl.TL_INT8, wsb=1 << 30) == UNS
    assert i(ks=None) == BAD and i(ps=24, wsb=1 << 30) == UNS
    size = tl.tl_paged_attn_decode_mass_workspace_size
    # the decode's, the rows' statistics, one f32 per row and place (rounded to 32)
    assert size(2, 1, 8, 2, 128, 70) == \
        tl.tl_paged_attn_decode_workspace_size(2, 8, 2, 128) + 256 + 2 * 8 * 96 * 4
    for args in ((0, 1, 8, 2, 128, 64), (2, 0, 8, 2, 128, 64), (2, 1, 7, 2, 128, 64),
                 (2, 5, 8, 2, 128, 64), (2, 1, 8, 2, 0, 64), (2, 1, 8, 2, 128, 0)):
        assert size(*args) == 0, args


def test_evict_select_refusals(lib):
    base = dict(m=256, ml=100, cl=512, n=8, first=1, last=2, keep=768, new=1024, B=2, hkv=2,
                err=None, st=None)
    e = caller(lib.tl_kv_evict_select, "m ml cl n first last keep new B hkv err st", base)
    for name in ("m", "cl", "keep", "new"):
        assert e(**{name: None}) == BAD, name
    for name in ("ml", "n", "B", "hkv"):
        assert e(**{name: 0}) == BAD, name
    assert e(first=-1) == BAD and e(last=-1) == BAD and e(first=7, last=2) == BAD
    for name, off in (("m", 264), ("cl", 513), ("keep", 772), ("new", 1032)):
        assert e(**{name: off}) == BAD, name
    assert e(ml=(1 << 30) + 1) == UNS and e(n=(1 << 30) + 1) == UNS and e(B=1 << 28) == UNS


def test_compact_refusals(lib):
    base = dict(k=256, v=512, ks=12288, vs=16384, bt=1024, maxp=8, cl=1280, keep=1536, n=8,
                new=1792, m=2048, ml=128, B=2, hkv=2, d=128, P=16, ps=16, dt=tl.TL_BF16, err=None,
                st=None)
    c = caller(lib.tl_kv_cache_compact,
               "k v bt maxp cl keep n new m ml B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_cache_compact_int8,
               "k v ks vs bt maxp cl keep n new m ml B hkv d P ps err st", base)
    for call in (c, i):
        for name in ("k", "v", "bt", "cl", "keep", "new"):
            assert call(**{name: None}) == BAD, name
        for name in ("maxp", "n", "B", "hkv", "d", "P", "ps", "ml"):
            assert call(**{name: 0}) == BAD, name
        for name, off in (("k", 264), ("v", 520), ("bt", 1026), ("cl", 1281), ("keep", 1540),
                          ("new", 1796), ("m", 2056)):
            assert call(**{name: off}) == BAD, name
        assert call(d=100) == BAD  # a row is not whole 16-byte vectors
        assert call(d=8192) == UNS and call(ps=257) == UNS and call(P=1 << 28) == UNS
    assert c(dt=tl.TL_INT8) == UNS and c(dt=9) == UNS
    assert i(ks=None) == BAD and i(vs=None) == BAD and i(ks=12290) == BAD


def test_compact_refuses_lists_past_its_counters(lib):
    ok = dict(k=256, v=512, bt=1024, maxp=8, cl=1280, keep=1536, n=(1 << 30) + 1, new=1792, m=None,
              ml=0, B=1, hkv=1, d=128, P=16, ps=16, dt=tl.TL_BF16, err=None, st=None)
    c = caller(lib.tl_kv_cache_compact,
               "k v bt maxp cl keep n new m ml B hkv d P ps dt err st", ok)
    assert c() == UNS and c(n=0) == BAD


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    b, s = torch.zeros(4, 2, 2, 128, dtype=torch.int8), torch.zeros(4, 2)
    m, q = torch.zeros(1, 2, 64), torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tl.tl_kv_page_bounds(x, t, n, b, s)
    with pytest.raises(TypeError):
        tl.tl_kv_page_select(q, b, s, t, n, 16, 2)
    with pytest.raises(TypeError):
        tl.tl_paged_attn_decode_pages(q, x, x, t.view(1, 1, 4), n, 0.1)
    with pytest.raises(TypeError):
        tl.tl_paged_attn_decode_mass(q[:, None], x, x, t, n, m, 0.1)
    with pytest.raises(TypeError):
        tl.tl_kv_evict_select(m, n, 8)
    with pytest.raises(TypeError):
        tl.tl_kv_cache_compact(x, x, t, n, torch.zeros(1, 2, 8, dtype=torch.int32), n)
