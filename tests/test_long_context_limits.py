"""Sizes of the long-context calls at which a 32-bit counter of a kernel would pass its range: refused
before any launch (no GPU; made-up addresses that no kernel ever sees)."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, build

UNS, WS = tl.TL_ERR_UNSUPPORTED, tl.TL_ERR_WORKSPACE
MOST = 1 << 30


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


def test_page_select_counts_places_and_blocks(lib):
    """Loops over places step by up to 8,192: with a page of one key, n_select just below 2^31
    would carry an index past it."""
    base = dict(q=256, qd=tl.TL_BF16, bnd=512, sc=768, bt=1024, maxp=8, cl=1280, n=4, first=1,
                last=1, pt=1536, pl=1792, B=1, hq=8, hkv=2, d=128, P=16, ps=1, ws=2048, wsb=0,
                err=None, st=None)
    s = caller(lib.tl_kv_page_select,
               "q qd bnd sc bt maxp cl n first last pt pl B hq hkv d P ps ws wsb err st", base)
    assert s(n=2**31 - 1) == UNS and s(n=2**31 - 8192) == UNS and s(n=MOST + 1) == UNS
    assert s(maxp=2**31 - 1) == UNS and s(maxp=MOST + 1) == UNS
    assert s(n=MOST) == WS and s(maxp=MOST) == WS  # the checks behind it: no workspace


def test_decode_mass_counts_positions(lib):
    """A warp of the adding kernel steps 128 positions at a time: past a length near 2^31 the next
    position would be negative."""
    base = dict(q=256, k=512, v=768, ks=12288, vs=16384, bt=1024, maxp=1 << 27, cl=1280, out=1536,
                m=2048, ml=64, B=1, T=1, hq=1, hkv=1, d=128, P=8, ps=16, w=0, sc=0.1,
                dt=tl.TL_BF16, ws=4096, wsb=2**62, err=None, st=None)
    a = caller(lib.tl_paged_attn_decode_mass,
               "q k v bt maxp cl out m ml B T hq hkv d P ps w sc dt ws wsb err st", base)
    i = caller(lib.tl_paged_attn_decode_mass_int8,
               "q k v ks vs bt maxp cl out m ml B T hq hkv d P ps w sc ws wsb err st", base)
    size = tl.tl_paged_attn_decode_mass_workspace_size
    for ml in (2**31 - 33, 2**31 - 130, MOST + 1):
        assert a(ml=ml) == UNS and i(ml=ml) == UNS, ml
        assert size(1, 1, 1, 1, 128, ml) == 0, ml
    assert a(ml=MOST, wsb=0) == WS and i(ml=MOST, wsb=0) == WS
    assert size(1, 1, 1, 1, 128, MOST) > 4 * MOST


def test_compact_counts_positions_of_the_mass(lib):
    """Zeroing the mass behind the kept rows steps up to 1,024 positions at a time up to the
    length, which mass_len bounds."""
    base = dict(k=1 << 20, v=1 << 21, ks=12288, vs=16384, bt=1024, maxp=1 << 27, cl=1280, keep=1536,
                n=8, new=1792, m=1 << 22, ml=128, B=1, hkv=1, d=128, P=16, ps=16, dt=tl.TL_INT8,
                err=None, st=None)
    c = caller(lib.tl_kv_cache_compact,
               "k v bt maxp cl keep n new m ml B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_cache_compact_int8,
               "k v ks vs bt maxp cl keep n new m ml B hkv d P ps err st", base)
    for ml in (2**31 - 1, 2**31 - 1024, MOST + 1):
        assert c(ml=ml, dt=tl.TL_BF16) == UNS and i(ml=ml) == UNS, ml
    # at the limit, and without a mass whatever the number, the checks pass: the launch itself
    # fails here, where there is no GPU
    if not torch.cuda.is_available():
        assert i(ml=MOST) == tl.TL_ERR_CUDA and i(m=None, ml=2**31 - 1) == tl.TL_ERR_CUDA
