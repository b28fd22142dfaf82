"""Sizes of the long-context calls at which a 32-bit counter of a kernel would pass its range: refused
before any launch (no GPU; made-up addresses that no kernel ever sees)."""
import pytest

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
