"""Rotary rows and appends of many tokens, whose warps take two or four passes
over a token's heads (16 items an SM and more: 2,432 on 152 SMs), against the
same rows in small calls, which take one, bit for bit, and against the plain
64-bit implementations of tests/rope_ref.py."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import rope_ref as ref
from tests.test_gpu_rope import POOL_KINDS, Pools, check_rows, i32, positions, slots_of, table, view

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def lie(kind, x):
    """x [n, h, d] on the GPU, its rows as `kind` says: 'aligned', 'four' (on 4-byte boundaries
    only: words of two elements), 'off' (on an element's: no words at all, element by element)."""
    n, h, d = x.shape
    if kind == "off":
        t, _ = view("off", n, h, d, x.dtype)
    elif kind == "four":
        step = h * d + 2
        t = torch.zeros(n * step + 2, dtype=x.dtype, device="cuda")[2:].view(n, step)[:, :h * d]
        t = t.view(n, h, d)
    else:
        t = torch.empty(n, h, d, dtype=x.dtype, device="cuda")
    return t.copy_(x)


# Query heads that are an odd number of passes (d = 48: 10 heads a pass, 80: 6, 96: 5, 112: 4,
# 192: 2), so that a pass of queries alone comes before one with keys, and lanes are left over
# behind its last head; then whole warps of lanes, up to four passes.
SIZES = [(10, 1, 48, 48), (30, 2, 48, 16), (6, 1, 80, 80), (18, 2, 80, 32), (5, 1, 96, 96),
         (15, 3, 96, 48), (4, 1, 112, 112), (12, 2, 112, 64), (2, 1, 192, 192), (6, 2, 192, 48),
         (7, 2, 80, 80), (0, 4, 128, 128), (8, 2, 128, 128), (20, 4, 128, 64), (8, 2, 128, 120),
         (3, 1, 64, 64), (6, 3, 256, 256)]


def append_in_parts(pools, q, k, v, slots, pos, step, *args):
    out = []
    for a in range(0, k.shape[0], step):
        b = slice(a, a + step)
        out.append(pools.append(None if q is None else q[b], k[b], v[b], slots[b], pos[b], *args))
    return None if q is None else torch.cat(out)


@pytest.mark.parametrize("src,kind", POOL_KINDS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", SIZES)
def test_append_of_many_tokens(src, kind, inter, hq, hkv, d, rot):
    n, ps, m = 5003, 16, 1.25
    P = n // ps + 9
    T = ref.TYPES[src]
    freqs, f = table(rot, 500000.0)
    slots, pos = slots_of(n, P, ps, seed=1), positions(n, seed=2)
    pos = np.where((slots >= 0) & (pos < 0), 77, pos)
    rows = ref.randn((n, hq + 2 * hkv, d), T, seed=3)
    q, k, v = rows.split([hq, hkv, hkv], 1)
    dev = rows.cuda().split([hq, hkv, hkv], 1)
    at, p = torch.as_tensor(slots).cuda(), i32(pos)
    many, few = Pools(kind, P, ps, hkv, d, seed=4), Pools(kind, P, ps, hkv, d, seed=4)
    args = (freqs, inter, m)
    one = many.append(dev[0] if hq else None, dev[1], dev[2], at, p, *args)
    two = append_in_parts(few, dev[0] if hq else None, dev[1], dev[2], at, p, 100, *args)
    for name, x in many.t.items():
        assert torch.equal(ref.bits(x), ref.bits(few.t[name])), name
    some = np.r_[0:40, n // 2:n // 2 + 40, n - 40:n]
    if hq:
        assert torch.equal(ref.bits(one), ref.bits(two))
        check_rows(q[some], one.cpu()[some], pos[some], f, inter, m, "q")
    live = some[slots[some] >= 0]
    there = torch.as_tensor(slots[live]).cuda()
    kw, ke = ref.rotate(ref.as_values(k)[live], pos[live][:, None], f, inter, m)
    vw = ref.as_values(v)[live]
    for name, want, err in (("k", kw, ke), ("v", vw, np.zeros_like(vw))):
        got, scales = many.rows(name, there)
        if kind == "int8":
            ref.close_int8(got, scales, want, err, name)
        else:
            ref.close(got, want, err, name)


@pytest.mark.parametrize("src,kind", POOL_KINDS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("where", ["four", "off"])
def test_append_of_many_tokens_off_alignment(src, kind, inter, where):
    """Rows on 4-byte boundaries and off them: the same bits as aligned ones."""
    n, hq, hkv, d, ps = 5003, 8, 2, 128, 16
    P = n // ps + 9
    T = ref.TYPES[src]
    freqs, _ = table(128, 500000.0)
    slots, pos = slots_of(n, P, ps, seed=1), positions(n, seed=2)
    pos = np.where((slots >= 0) & (pos < 0), 77, pos)
    args = (torch.as_tensor(slots).cuda(), i32(pos), freqs, inter)
    rows = [ref.randn((n, h, d), T, seed=h) for h in (hq, hkv, hkv)]
    one, two = Pools(kind, P, ps, hkv, d, seed=4), Pools(kind, P, ps, hkv, d, seed=4)
    a = one.append(*(x.cuda() for x in rows), *args)
    b = two.append(*(lie(where, x) for x in rows), *args)
    assert torch.equal(ref.bits(a), ref.bits(b))
    for name, x in one.t.items():
        assert torch.equal(ref.bits(x), ref.bits(two.t[name])), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("h,d,rot", [(20, 128, 128), (33, 128, 64), (32, 80, 80), (13, 96, 96),
                                     (9, 192, 48), (5, 256, 256), (8, 128, 120), (40, 48, 20)])
@pytest.mark.parametrize("where", ["aligned", "four", "off"])
def test_rows_of_many_tokens(dtype, inter, h, d, rot, where):
    n, m = 2503, 1.25
    freqs, f = table(rot, 500000.0)
    pos = positions(n, seed=4)
    x = ref.randn((n, h, d), dtype, seed=5)
    rows = lie(where, x)
    p = i32(pos)
    out = tl.tl_rope(rows, p, freqs, inter, m)
    whole = x.cuda()
    small = torch.cat([tl.tl_rope(whole[a:a + 50], p[a:a + 50], freqs, inter, m)
                       for a in range(0, n, 50)])
    assert torch.equal(ref.bits(out), ref.bits(small))
    some = np.r_[0:40, n // 2:n // 2 + 40, n - 40:n]
    check_rows(x[some], out.cpu()[some], pos[some], f, inter, m, where)
    assert tl.tl_rope(rows, p, freqs, inter, m, out=rows) is rows  # in place: the same bits
    assert torch.equal(ref.bits(rows), ref.bits(out))
