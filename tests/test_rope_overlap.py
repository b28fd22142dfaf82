"""The rotary calls refuse lists and tables that lie over what they write, before any launch (no
GPU; made-up addresses that no kernel ever sees)."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, build
from tests.test_rope_tables import caller

BAD = tl.TL_ERR_INVALID_ARG
M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def over(base, lists, written):
    """Places of each list (name, bytes, alignment) that have their first or last element in what
    is written (name, first byte, bytes), and places beside it."""
    for name, size, step in lists:
        for to, at, n in written:
            for place in (at, at + n - step, at - size + step):
                yield {name: place}, True
            for place in (at + n, at - size):
                yield {name: place}, False


def check(call, base, lists, written):
    for kw, hit in over(base, lists, written):
        if hit:
            assert call(**kw) == BAD, kw
        elif not torch.cuda.is_available():  # all checks passed; the launch fails without a GPU
            assert call(**kw) == tl.TL_ERR_CUDA, kw


def test_rows(lib):
    for dt, e in ((tl.TL_BF16, 2), (tl.TL_F32, 4)):
        base = dict(x=M, xs=2048, o=4 * M, os=1536, pos=256, f=8192, rot=64, il=0, m=1.0, n=40, h=8,
                    d=128, dt=dt, st=None)
        r = caller(lib.tl_rope, "x xs o os pos f rot il m n h d dt st", base)
        check(r, base, [("pos", 160, 4), ("f", 256, 8)], [("o", 4 * M, (39 * 1536 + 1024) * e)])
        one = caller(lib.tl_rope, "x xs o os pos f rot il m n h d dt st", dict(base, n=1, os=0))
        check(one, base, [("pos", 4, 4), ("f", 256, 8)], [("o", 4 * M, 1024 * e)])


def test_append(lib):
    base = dict(q=M, qs=1024, o=2 * M, os=1024, k=3 * M, ks=256, v=4 * M, vs=256, sd=tl.TL_BF16,
                kc=5 * M, vc=6 * M, ksc=7 * M, vsc=8 * M, sm=9 * M, pos=10 * M, f=11 * M, rot=128,
                il=0, m=1.0, n=3, P=16, ps=16, hq=8, hkv=2, d=128, dt=tl.TL_BF16, err=None,
                st=None)
    a = caller(lib.tl_kv_cache_write_rope,
               "q qs o os k ks v vs sd kc vc sm pos f rot il m n P ps hq hkv d dt err st", base)
    i = caller(lib.tl_kv_cache_write_rope_int8,
               "q qs o os k ks v vs sd kc vc ksc vsc sm pos f rot il m n P ps hq hkv d err st",
               base)
    lists = [("sm", 24, 8), ("pos", 12, 4), ("f", 512, 8)]
    slots = 16 * 16 * 2
    check(a, base, lists, [("o", 2 * M, 3 * 1024 * 2), ("kc", 5 * M, slots * 256),
                           ("vc", 6 * M, slots * 256)])
    check(i, base, lists, [("o", 2 * M, 3 * 1024 * 2), ("kc", 5 * M, slots * 128),
                           ("vc", 6 * M, slots * 128), ("ksc", 7 * M, slots * 4),
                           ("vsc", 8 * M, slots * 4)])


def test_compaction(lib):
    base = dict(k=M, v=2 * M, ks=3 * M, vs=4 * M, bt=5 * M, maxp=8, cl=6 * M, keep=7 * M, n=4,
                nl=8 * M, mass=9 * M, mlen=128, f=10 * M, rot=128, il=0, B=4, hkv=2, d=128, P=16,
                ps=16, dt=tl.TL_BF16, err=None, st=None)
    a = caller(lib.tl_kv_cache_compact_rope,
               "k v bt maxp cl keep n nl mass mlen f rot il B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_cache_compact_rope_int8,
               "k v ks vs bt maxp cl keep n nl mass mlen f rot il B hkv d P ps err st", base)
    lists = [("bt", 4 * 8 * 4, 4), ("cl", 16, 4), ("keep", 4 * 2 * 4 * 4, 16), ("nl", 16, 16),
             ("f", 512, 8)]
    slots, mass = 16 * 16 * 2, ("mass", 9 * M, 4 * 2 * 128 * 4)
    check(a, base, lists, [("k", M, slots * 256), ("v", 2 * M, slots * 256), mass])
    check(i, base, lists, [("k", M, slots * 128), ("v", 2 * M, slots * 128),
                           ("ks", 3 * M, slots * 4), ("vs", 4 * M, slots * 4), mass])


def test_step_workspace(lib):
    """The plan writes the workspace beside the warps that write the rows and scales."""
    B, hq, hkv, d = 3, 8, 2, 128
    need = tl.tl_paged_attn_decode_write_rope_workspace_size(B, hq, hkv, d)
    base = dict(q=M, qs=1024, k=3 * M, ks=256, v=4 * M, vs=256, sm=9 * M, pos=10 * M, f=11 * M,
                rot=128, il=0, m=1.0, kc=5 * M, vc=6 * M, ksc=7 * M, vsc=8 * M, bt=12 * M, maxp=8,
                cl=13 * M, out=14 * M, B=B, hq=hq, hkv=hkv, d=d, P=16, ps=16, w=0, sc=0.1,
                dt=tl.TL_BF16, ws=64 * M, wsb=need, err=None, st=None)
    a = caller(lib.tl_paged_attn_decode_write_rope,
               "q qs k ks v vs sm pos f rot il m kc vc bt maxp cl out B hq hkv d P ps w sc dt ws "
               "wsb err st", base)
    i = caller(lib.tl_paged_attn_decode_write_rope_int8,
               "q qs k ks v vs sm pos f rot il m kc vc ksc vsc bt maxp cl out B hq hkv d P ps w sc "
               "ws wsb err st", base)
    slots = 16 * 16 * hkv
    lists = [("sm", 24, 8), ("pos", 12, 4), ("f", 512, 8), ("k", 2 * 256 * 2 + 512, 2),
             ("q", 3 * 1024 * 2, 2)]
    for call, size, scales in ((a, 2, []), (i, 1, [("ksc", slots * 4, 16), ("vsc", slots * 4, 16)])):
        check(call, base, lists + scales + [("kc", slots * d * size, 16),
                                            ("vc", slots * d * size, 16)],
              [("ws", 64 * M, need)])
