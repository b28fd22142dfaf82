"""Outputs that overlap what other blocks of the same launch still read: refused before any launch
(no GPU; made-up addresses that no kernel ever sees)."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, build

BAD = tl.TL_ERR_INVALID_ARG


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


def passes(status):
    """All checks passed; the launch itself fails where there is no GPU."""
    return status == tl.TL_ERR_CUDA


def test_evict_select_is_not_in_place(lib):
    """Each head's CTAs read the sequence's length; one of them writes the new one."""
    M = 1 << 20
    base = dict(m=1 * M, ml=100, cl=2 * M, n=8, first=1, last=2, keep=3 * M, new=4 * M, B=4, hkv=2,
                err=None, st=None)
    e = caller(lib.tl_kv_evict_select, "m ml cl n first last keep new B hkv err st", base)
    mass, keep, lens = 4 * 4 * 2 * 100, 4 * 4 * 2 * 8, 4 * 4
    assert e(new=base["cl"]) == BAD
    assert e(cl=4 * M + 12) == BAD and e(cl=4 * M - 12) == BAD  # one element in common
    assert e(keep=2 * M) == BAD and e(keep=2 * M - keep + 16) == BAD
    assert e(keep=4 * M) == BAD and e(new=3 * M + keep - 16) == BAD
    assert e(keep=1 * M) == BAD and e(keep=1 * M + mass - 16) == BAD and e(new=1 * M + 64) == BAD
    if not torch.cuda.is_available():
        for kw in (dict(), dict(cl=4 * M + lens), dict(cl=4 * M - lens), dict(new=3 * M + keep),
                   dict(keep=1 * M + mass), dict(keep=2 * M - keep)):
            assert passes(e(**kw)), kw


def test_page_select_is_not_in_place(lib):
    M = 1 << 20
    base = dict(q=1 * M, qd=tl.TL_BF16, bnd=2 * M, sc=3 * M, bt=4 * M, maxp=8, cl=5 * M, n=4,
                first=1, last=1, pt=6 * M, pl=7 * M, B=4, hq=8, hkv=2, d=128, P=16, ps=16,
                ws=8 * M, wsb=1 << 18, err=None, st=None)
    s = caller(lib.tl_kv_page_select,
               "q qd bnd sc bt maxp cl n first last pt pl B hq hkv d P ps ws wsb err st", base)
    table, block, lens = 4 * 4 * 2 * 4, 4 * 4 * 8, 4 * 4
    need = tl.tl_kv_page_select_workspace_size(4, 8, 2, 128, 8)
    assert s(pl=base["cl"]) == BAD and s(cl=7 * M - 4) == BAD and s(cl=7 * M + 12) == BAD
    assert s(pt=base["bt"]) == BAD and s(bt=6 * M + table - 4) == BAD
    assert s(pt=5 * M) == BAD and s(pl=4 * M + block - 16) == BAD
    assert s(pt=8 * M) == BAD and s(pl=8 * M + need - 16) == BAD
    assert s(pl=6 * M) == BAD and s(pl=6 * M + table - 16) == BAD
    if not torch.cuda.is_available():
        for kw in (dict(), dict(cl=7 * M + lens), dict(bt=6 * M + table), dict(pl=6 * M + table),
                   dict(pt=4 * M + block), dict(pl=8 * M + need)):
            assert passes(s(**kw)), kw


def test_compaction_moves_each_buffer_once(lib):
    """K and V in one pool: two CTAs would gather the same rows at the same time."""
    M = 1 << 20
    base = dict(k=1 * M, v=2 * M, ks=3 * M, vs=4 * M, bt=5 * M, maxp=8, cl=6 * M, keep=7 * M, n=8,
                new=8 * M, m=9 * M, ml=128, B=2, hkv=2, d=128, P=16, ps=16, dt=tl.TL_BF16,
                err=None, st=None)
    c = caller(lib.tl_kv_cache_compact,
               "k v bt maxp cl keep n new m ml B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_cache_compact_int8,
               "k v ks vs bt maxp cl keep n new m ml B hkv d P ps err st", base)
    slots = 16 * 16 * 2
    assert c(v=1 * M) == BAD and c(v=1 * M + slots * 256 - 16) == BAD
    assert i(v=1 * M) == BAD and i(v=1 * M + slots * 128 - 16) == BAD
    assert i(vs=3 * M) == BAD and i(ks=4 * M + slots * 4 - 16) == BAD and i(ks=1 * M) == BAD
    assert c(m=1 * M) == BAD and i(m=3 * M) == BAD
    if not torch.cuda.is_available():
        for call, kw in ((c, dict()), (i, dict()), (c, dict(v=1 * M + slots * 256)),
                         (i, dict(v=1 * M + slots * 128)), (i, dict(vs=3 * M + slots * 4)),
                         (c, dict(m=None)), (i, dict(m=None))):
            assert passes(call(**kw)), kw
