"""Rotary tables (tl_rope_freqs) against their definitions, the arithmetic of an
angle's cosine and sine restated on the host against 64 bits, and the host-side
refusals of the rotary calls (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, api, build
from tests import rope_ref as ref

BAD, UNS, OK = tl.TL_ERR_INVALID_ARG, tl.TL_ERR_UNSUPPORTED, tl.TL_OK
WS = tl.TL_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


# ------------------------------------------------------------------ tables --

def turns(freqs):
    return np.array([(int(x) % 2 ** 64) / 2.0 ** 64 for x in freqs])


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (16, 10000.0), (128, 500000.0), (130, 1.5),
                                      (4096, 1e6)])
def test_plain_table(rot, base):
    freqs, scale = tl.tl_rope_freqs(rot, base, device="cpu")
    assert scale == 1.0 and freqs.shape == (rot // 2,) and freqs.dtype == torch.int64
    want = ref.inv_freq(rot, base) / (2 * math.pi)
    # pow, a division and the product by 2^64 (exact): within 2^-51, and half a 2^-64
    assert (np.abs(turns(freqs) - want) <= want * 2.0 ** -50 + 2.0 ** -65).all()


def test_stretched_tables():
    rot, base, L, k = 64, 10000.0, 8192.0, 8.0
    f = ref.inv_freq(rot, base)
    t = L * f / (2 * math.pi)

    def check(want, **kw):
        freqs, scale = tl.tl_rope_freqs(rot, base, device="cpu", **kw)
        want = np.asarray(want) / (2 * math.pi)
        assert (np.abs(turns(freqs) - want) <= want * 2.0 ** -45 + 2.0 ** -65).all()
        return scale

    assert check(f / k, scaling=tl.TL_ROPE_LINEAR, factor=k) == 1.0
    assert check(ref.inv_freq(rot, base * k ** (rot / (rot - 2))), scaling=tl.TL_ROPE_BASE,
                 factor=k) == 1.0
    keep = np.clip((t - 1.0) / 3.0, 0, 1)
    assert 0 < np.sum((keep > 0) & (keep < 1)) < 10
    assert check(f * keep + f / k * (1 - keep), scaling=tl.TL_ROPE_BANDS, factor=k, trained_len=L,
                 low=1.0, high=4.0) == 1.0

    def at(n):
        return rot * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    slow = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    scale = check(f / k * slow + f * (1 - slow), scaling=tl.TL_ROPE_RAMP, factor=k, trained_len=L,
                  low=1.0, high=32.0)
    assert scale == np.float32(0.1 * math.log(k) + 1)
    many = 1 + np.arange(rot // 2) / 7
    assert check(f / many, scaling=tl.TL_ROPE_FACTORS, factors=many) == 1.0


def test_tables_wrap_whole_turns():
    """f = 2 pi exactly is no turn at all: entries are taken modulo one turn."""
    n = 4
    freqs, _ = tl.tl_rope_freqs(2 * n, 10000.0, tl.TL_ROPE_FACTORS, device="cpu",
                                factors=[1e-3] * n)  # up to 159 turns a position
    want = ref.inv_freq(2 * n) / 1e-3 / (2 * math.pi) % 1.0
    assert np.abs(turns(freqs) - want).max() < 2.0 ** -44


def test_table_refusals(lib):
    out = (ctypes.c_uint64 * 2048)()
    scale = ctypes.c_float(7)

    def f(rot=8, base=1e4, kind=0, factor=2.0, L=100.0, low=1.0, high=4.0, factors=None,
          freqs=out, s=scale):
        return lib.tl_rope_freqs(rot, base, kind, factor, L, low, high, factors, freqs,
                                 None if s is None else ctypes.byref(s))
    assert f() == OK and f(factor=-1.0, L=-1.0, low=9.0) == OK  # a plain table reads none of them
    for rot in (0, -2, 1, 7, 4098):
        assert f(rot=rot) == BAD
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert f(base=base) == BAD
    for kind in (-1, 6):
        assert f(kind=kind) == UNS
    for kind in (tl.TL_ROPE_LINEAR, tl.TL_ROPE_BASE, tl.TL_ROPE_BANDS, tl.TL_ROPE_RAMP):
        for factor in (0.0, -1.0, math.inf, math.nan):
            assert f(kind=kind, factor=factor) == BAD
    for kind in (tl.TL_ROPE_BANDS, tl.TL_ROPE_RAMP):
        assert f(kind=kind, L=0.0) == BAD and f(kind=kind, L=math.nan) == BAD
        assert f(kind=kind, low=0.0) == BAD and f(kind=kind, low=4.0) == BAD
        assert f(kind=kind, high=math.inf) == BAD and f(kind=kind, high=math.nan) == BAD
    assert f(kind=tl.TL_ROPE_BASE, rot=2) == BAD and f(kind=tl.TL_ROPE_BASE, factor=1e-9) == BAD
    assert f(kind=tl.TL_ROPE_FACTORS) == BAD
    for bad in (0.0, -1.0, math.nan, math.inf):
        assert f(kind=tl.TL_ROPE_FACTORS, factors=(ctypes.c_double * 4)(1, 1, bad, 1)) == BAD
    assert f(freqs=None) == BAD and f(s=None) == BAD
    with pytest.raises(ValueError):
        tl.tl_rope_freqs(8, scaling=tl.TL_ROPE_FACTORS, factors=[1.0, 2.0], device="cpu")
    with pytest.raises(tl.TLError):
        tl.tl_rope_freqs(7, device="cpu")


# ------------------------------------------------------------------ angles --

def turn32(freq, pos):
    """Cosine and sine as the kernels compute them: the phase in integers, series in binary32
    (a fused multiply-add is a 64-bit product and sum rounded once more: within half a 2^-29 of
    the single rounding, which the bound below leaves room for)."""
    f = np.float32

    def fma(a, b, c):
        return (a.astype(np.float64) * b.astype(np.float64) + c).astype(np.float32)

    h = math.pi / 2
    phase = np.array([(int(p) * int(q)) % 2 ** 64 >> 32 for p, q in zip(pos, freq)], np.uint64)
    quarter = ((phase + 2 ** 29) % 2 ** 32 >> np.uint64(30)).astype(np.int64)
    r = phase.astype(np.int64) - (quarter << 30)
    r = np.where(r >= 2 ** 31, r - 2 ** 32, r)
    assert (np.abs(r) <= 2 ** 29).all()
    t = r.astype(np.float32) * f(2.0 ** -30)
    x = t * t
    one = np.ones_like(t)
    s = fma(x, one * f(h ** 9 / math.factorial(9)), -float(f(h ** 7 / math.factorial(7))))
    s = fma(x, s, float(f(h ** 5 / math.factorial(5))))
    s = fma(x, s, -float(f(h ** 3 / math.factorial(3))))
    s = fma(x, s, float(f(h - float(f(h)))))
    s = fma(t, one * f(h), (t * s).astype(np.float64))
    c = fma(x, one * -f(h ** 10 / math.factorial(10)), float(f(h ** 8 / math.factorial(8))))
    c = fma(x, c, -float(f(h ** 6 / math.factorial(6))))
    c = fma(x, c, float(f(h ** 4 / math.factorial(4))))
    c = fma(x, c, -float(f(h ** 2 / 2)))
    c = fma(x, c, 1.0)
    odd = (quarter & 1) == 1
    a, b = np.where(odd, s, c), np.where(odd, c, s)
    return np.where((quarter + 1) & 2, -a, a), np.where(quarter & 2, -b, b)


def test_cosine_and_sine_are_within_their_bound():
    g = np.random.default_rng(0)
    n = 200000
    freq = g.integers(0, 2 ** 64, n, dtype=np.uint64)
    pos = g.integers(0, 2 ** 31, n)
    # phases at and next to the borders of the quarters
    edges = [(k << 30) + (1 << 29) + e for k in range(4) for e in (-2, -1, 0, 1, 2)]
    edges += [(k << 30) + e for k in range(4) for e in (0, 1, 2, 3)]
    freq[:len(edges)] = np.array([(e % 2 ** 32) << 32 for e in edges], np.uint64)
    pos[:len(edges)] = 1
    pos[1000:2000] = 0
    pos[2000:3000] *= -1
    c, s = turn32(freq, pos)
    exact = np.array([(int(p) * int(q)) % 2 ** 64 / 2.0 ** 64 for p, q in zip(pos, freq)])
    a = 2 * math.pi * exact
    assert np.abs(c - np.cos(a)).max() < 2.0 ** -23
    assert np.abs(s - np.sin(a)).max() < 2.0 ** -23
    assert (c[1000:2000] == 1).all() and (s[1000:2000] == 0).all()


def test_far_positions_keep_their_angles():
    """What a binary32 product loses at a position near a million, the integer phase has."""
    f = ref.inv_freq(128)
    freq = np.array([int(x) for x in ref.table(f)], np.uint64)
    for p in (1, 999_983, 2 ** 31 - 1):
        c, _ = turn32(freq, np.full(64, p))
        # 64-bit products: 2^-52 of the angle; the table: 2^-53 of the frequency
        tol = 2.0 ** -23 + p * f * 2.0 ** -51
        assert (np.abs(c - np.cos(p * f)) <= tol).all()
    wrong = np.cos((np.float32(999_983) * f.astype(np.float32)).astype(np.float64))
    assert np.abs(wrong - np.cos(999_983 * f)).max() > 1e-3


# ---------------------------------------------------------------- refusals --

def caller(fn, order, base):
    def call(**kw):
        assert set(kw) <= set(base), kw
        a = dict(base, **kw)
        return fn(*(a[n] for n in order.split()))
    return call


def test_rope_refusals(lib):
    M = 1 << 20
    base = dict(x=M, xs=1024, o=4 * M, os=1024, pos=256, f=512, rot=64, il=0, m=1.0, n=3, h=8,
                d=128, dt=tl.TL_BF16, st=None)
    r = caller(lib.tl_rope, "x xs o os pos f rot il m n h d dt st", base)
    assert r(n=0) == OK and r(n=0, x=None, pos=None) == OK
    for name in ("x", "o", "pos", "f"):
        assert r(**{name: None}) == BAD, name
    for name in ("h", "d"):
        assert r(**{name: 0}) == BAD and r(**{name: -1}) == BAD
    assert r(n=-1) == BAD
    for rot in (0, 1, -2, 63, 130):
        assert r(rot=rot) == BAD
    assert r(pos=258) == BAD and r(f=516) == BAD and r(x=M + 1) == BAD and r(o=4 * M + 1) == BAD
    assert r(dt=tl.TL_F32, x=M + 2) == BAD
    assert r(dt=tl.TL_FP8_E4M3) == UNS and r(dt=tl.TL_INT8) == UNS and r(dt=9) == UNS
    assert r(d=4098) == UNS and r(h=1 << 24) == UNS
    assert r(xs=-1) == BAD and r(os=1023) == BAD and r(xs=1 << 31) == BAD and r(os=1 << 31) == BAD
    # outputs over inputs: one element is enough; in place is the same place and stride
    assert r(o=M + 2) == BAD and r(o=M - 2) == BAD and r(o=M, os=2048) == BAD
    assert r(o=M + 2 * (2 * 1024 + 1023), n=3) == BAD
    # rows of one stride that lie beside each other's elements are told apart, to the element
    assert r(xs=4096, os=4096, o=M + 2 * 1023) == BAD
    assert r(xs=4096, os=4096, o=M + 2 * 4096 - 2 * 1023) == BAD
    assert r(xs=4096, os=2048, o=M + 2 * 1024) == BAD  # of different strides by their ranges


def test_write_rope_refusals(lib):
    M = 1 << 24
    base = dict(q=M, qs=1024, o=2 * M, os=1024, k=3 * M, ks=256, v=4 * M, vs=256, sd=tl.TL_BF16,
                kc=5 * M, vc=6 * M, ksc=7 * M, vsc=8 * M, sm=9 * M, pos=10 * M, f=11 * M, rot=128,
                il=0, m=1.0, n=3, P=16, ps=16, hq=8, hkv=2, d=128, dt=tl.TL_BF16, err=None,
                st=None)
    a = caller(lib.tl_kv_cache_write_rope,
               "q qs o os k ks v vs sd kc vc sm pos f rot il m n P ps hq hkv d dt err st", base)
    i = caller(lib.tl_kv_cache_write_rope_int8,
               "q qs o os k ks v vs sd kc vc ksc vsc sm pos f rot il m n P ps hq hkv d err st",
               base)
    for call in (a, i):
        assert call(n=0) == OK and call(n=0, k=None) == OK
        for name in ("q", "o", "k", "v", "kc", "vc", "sm", "pos", "f"):
            assert call(**{name: None}) == BAD, name
        assert call(hq=0) == BAD  # queries given for no heads
        for name in ("P", "ps", "hkv", "d"):
            assert call(**{name: 0}) == BAD and call(**{name: -1}) == BAD, name
        assert call(n=-1) == BAD and call(hq=-1) == BAD
        for rot in (0, 3, 130, -4):
            assert call(rot=rot) == BAD
        for name, off in (("sm", 4), ("pos", 2), ("f", 4), ("q", 1), ("k", 1), ("v", 1), ("o", 1),
                          ("kc", 8), ("vc", 8)):
            assert call(**{name: base[name] + off}) == BAD, name
        for sd in (tl.TL_FP8_E4M3, tl.TL_INT8, 7):
            assert call(sd=sd) == UNS
        assert call(P=1 << 28) == UNS and call(hkv=1 << 23) == UNS
        for name in ("qs", "ks", "vs"):
            assert call(**{name: -1}) == BAD and call(**{name: 1 << 31}) == BAD
        assert call(os=1023) == BAD
        # what is written over anything else
        for name, other in (("o", "q"), ("o", "k"), ("o", "v"), ("o", "kc"), ("o", "vc"),
                            ("kc", "vc"), ("kc", "q"), ("vc", "k"), ("kc", "v")):
            at = base[other] + (2 if name == "o" else 16)
            assert call(**{name: at}) == BAD, (name, other)
    assert a(dt=tl.TL_F32) == UNS and a(dt=9) == UNS
    assert a(d=100, rot=100, hkv=1, hq=1) == BAD  # pool rows of 200 bytes
    assert i(ksc=None) == BAD and i(vsc=None) == BAD and i(ksc=7 * M + 2) == BAD
    assert i(d=1040, rot=2) == UNS
    assert i(ksc=8 * M) == BAD and i(ksc=5 * M + 64) == BAD and i(vsc=3 * M) == BAD


def test_step_refusals(lib):
    M = 1 << 24
    base = dict(q=M, qs=1024, k=3 * M, ks=256, v=4 * M, vs=256, sm=9 * M, pos=10 * M, f=11 * M,
                rot=128, il=0, m=1.0, kc=5 * M, vc=6 * M, ksc=7 * M, vsc=8 * M, bt=12 * M, maxp=8,
                cl=13 * M, out=14 * M, B=3, hq=8, hkv=2, d=128, P=16, ps=16, w=0, rp=8, sc=0.1,
                dt=tl.TL_BF16, ws=None, wsb=0, err=None, st=None)
    a = caller(lib.tl_paged_attn_decode_write_rope,
               "q qs k ks v vs sm pos f rot il m kc vc bt maxp cl out B hq hkv d P ps w sc dt ws "
               "wsb err st", base)
    i = caller(lib.tl_paged_attn_decode_write_rope_int8,
               "q qs k ks v vs sm pos f rot il m kc vc ksc vsc bt maxp cl out B hq hkv d P ps w sc "
               "ws wsb err st", base)
    g = caller(lib.tl_paged_attn_decode_write_rope_ring,
               "q qs k ks v vs sm pos f rot il m kc vc bt maxp cl out B hq hkv d P ps w rp sc dt "
               "ws wsb err st", dict(base, w=100))
    size = tl.tl_paged_attn_decode_write_rope_workspace_size
    need = size(3, 8, 2, 128)
    assert need >= tl.tl_paged_attn_decode_workspace_size(3, 8, 2, 128) + 4 * 3 * 8 * 128
    assert size(0, 8, 2, 128) == 0 and size(3, 7, 2, 128) == 0 and size(3, 8, 2, 0) == 0
    for call in (a, i, g):
        assert call() == WS and call(ws=1 << 30, wsb=need - 1) == WS
        assert call(ws=(1 << 30) + 128, wsb=need) == WS
        for name in ("q", "k", "v", "sm", "pos", "f", "kc", "vc", "bt", "cl", "out"):
            assert call(**{name: None}) == BAD, name
        for name in ("B", "hq", "hkv", "d", "P", "ps", "maxp"):
            assert call(**{name: 0}) == BAD and call(**{name: -1}) == BAD, name
        assert call(hq=7) == BAD and call(w=-1) == BAD
        for rot in (0, 3, 130):
            assert call(rot=rot) == BAD
        for name, off in (("sm", 4), ("pos", 2), ("f", 4), ("q", 1), ("k", 1), ("kc", 8),
                          ("out", 8), ("bt", 2), ("cl", 2)):
            assert call(**{name: base[name] + off}) == BAD, name
        for name in ("qs", "ks", "vs"):
            assert call(**{name: -1}) == BAD
        assert call(d=256, rot=128) == UNS and call(hq=34) == UNS and call(ps=257) == UNS
        assert call(d=96, rot=96) == UNS
        # the workspace over the rows or the pools
        assert call(ws=3 * M - 4096, wsb=need) == BAD and call(ws=5 * M, wsb=need) == BAD
    for call in (a, g):
        assert call(dt=tl.TL_INT8) == UNS and call(dt=9) == UNS
    assert i(ksc=None) == BAD and i(vsc=None) == BAD and i(ps=24) == UNS and i(ps=8) == UNS
    assert g(w=0) == BAD and g(rp=0) == BAD and g(rp=9) == BAD and g(w=129) == BAD


def test_compact_rope_refusals(lib):
    M = 1 << 24
    base = dict(k=M, v=2 * M, ks=3 * M, vs=4 * M, bt=5 * M, maxp=8, cl=6 * M, keep=7 * M, n=4,
                nl=8 * M, mass=9 * M, mlen=128, f=10 * M, rot=128, il=0, B=2, hkv=2, d=128, P=16,
                ps=16, dt=tl.TL_BF16, err=None, st=None)
    a = caller(lib.tl_kv_cache_compact_rope,
               "k v bt maxp cl keep n nl mass mlen f rot il B hkv d P ps dt err st", base)
    i = caller(lib.tl_kv_cache_compact_rope_int8,
               "k v ks vs bt maxp cl keep n nl mass mlen f rot il B hkv d P ps err st", base)
    for call in (a, i):
        for name in ("k", "v", "bt", "cl", "keep", "nl", "f"):
            assert call(**{name: None}) == BAD, name
        for name in ("B", "hkv", "d", "P", "ps", "maxp", "n", "mlen"):
            assert call(**{name: 0}) == BAD and call(**{name: -1}) == BAD, name
        for rot in (0, 1, -16, 144, 7):
            assert call(rot=rot) == BAD
        assert call(f=10 * M + 4) == BAD
        assert call(rot=24) == UNS and call(rot=2) == UNS
        assert call(ps=257) == UNS and call(P=1 << 28) == UNS
        assert call(k=2 * M) == BAD and call(mass=M) == BAD
    assert a(d=72, rot=16) == UNS  # rows of 144 bytes, not whole units
    assert a(dt=tl.TL_INT8) == UNS and a(dt=9) == UNS
    assert i(ks=None) == BAD and i(vs=None) == BAD
    assert i(d=48, rot=16) == UNS and i(d=1024, rot=16) == UNS


def test_binding_checks():
    """The binding's checks come before the library's; CPU tensors are refused."""
    bf = torch.bfloat16
    x = torch.zeros(4, 2, 8, dtype=bf)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    pool = torch.zeros(2, 4, 2, 8, dtype=bf)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        tl.tl_rope(x, pos, freqs)
    with pytest.raises(TypeError):
        tl.tl_kv_cache_write_rope(x, x, x, pool, pool, slots, pos, freqs)
    with pytest.raises(TypeError):
        tl.tl_kv_cache_compact_rope(pool, pool, pos, pos, pos, pos, freqs)


def test_binding_reads_rows_where_they_lie(monkeypatch):
    """Strides and shapes of rows, with the device checks replaced."""
    calls = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(api, "_run", lambda name, dev, stream, *a: calls.append((name, a)))
    monkeypatch.setattr(api, "_returned",
                        lambda shape, dtype, dev, stream: torch.empty(shape, dtype=dtype))

    class Dev:
        index = 0
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: Dev))
    bf = torch.bfloat16
    rows = torch.zeros(5, 8, 16, dtype=bf)
    q, k, v = rows.split([4, 2, 2], 1)
    pos, freqs = torch.zeros(5, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)
    pool = torch.zeros(2, 4, 2, 16, dtype=bf)
    slots = torch.zeros(5, dtype=torch.int64)
    out = tl.tl_kv_cache_write_rope(q, k, v, pool, pool.clone(), slots, pos, freqs, True, 1.5)
    name, a = calls.pop()
    assert name == "tl_kv_cache_write_rope" and out.shape == (5, 4, 16) and out.is_contiguous()
    assert a[0] == rows.data_ptr() and a[1] == 128 and a[3] == 64
    assert a[4] == rows.data_ptr() + 2 * 64 and a[5] == 128 and a[7] == 128
    assert a[14:17] == (16, 1, 1.5) and a[17:23] == (5, 2, 4, 4, 2, 16)
    assert tl.tl_kv_cache_write_rope(None, k, v, pool, pool.clone(), slots, pos, freqs) is None
    assert calls.pop()[1][:4] == (None, 0, None, 0)
    assert tl.tl_rope(q, pos, freqs[:3], out=q) is q
    assert calls.pop()[1][6] == 6
    for bad in (dict(k_new=k[:, :1]), dict(k_new=k.float()), dict(q=q[:4]), dict(q=q[..., ::2]),
                dict(q=q.transpose(0, 1)), dict(q=q[:, :0]), dict(positions=pos.long()),
                dict(positions=pos[:4]), dict(freqs=freqs.double()), dict(freqs=freqs[:0]),
                dict(freqs=torch.zeros(9, dtype=torch.int64)), dict(slot_mapping=slots.int()),
                dict(q_out=torch.zeros(5, 4, 16)), dict(q=None, q_out=q)):
        args = dict(q=q, k_new=k, v_new=v, k_cache=pool, v_cache=pool.clone(), slot_mapping=slots,
                    positions=pos, freqs=freqs)
        with pytest.raises((TypeError, ValueError)):
            tl.tl_kv_cache_write_rope(**dict(args, **bad))
        assert not calls
