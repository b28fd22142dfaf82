"""A decode step that rotates its queries and keys itself: the same outputs, pools and error bits
as the append that rotates and the decode behind it, bit for bit, for every pool, plan and layout."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as lref
from tests import rope_ref as ref
from tests.test_gpu_rope import Pools, i32, table, word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def decode(pools, q, tbl, lens, scale, window, ring, err, **kw):
    t = pools.t
    if pools.kind == "int8":
        return tl.tl_paged_attn_decode_int8(q, t["k"], t["v"], t["ks"], t["vs"], tbl, lens, scale,
                                            window=window, error_word=err, **kw)
    if ring:
        return tl.tl_paged_attn_decode_ring(q, t["k"], t["v"], tbl, lens, scale, window, ring,
                                            error_word=err, **kw)
    return tl.tl_paged_attn_decode(q, t["k"], t["v"], tbl, lens, scale, window=window,
                                   error_word=err, **kw)


def step(pools, rows, slots, pos, freqs, tbl, lens, scale, window, ring, inter, m, err, **kw):
    t = pools.t
    how = dict(interleaved=inter, rope_scale=m, error_word=err, **kw)
    if pools.kind == "int8":
        return tl.tl_paged_attn_decode_write_rope_int8(
            *rows, slots, pos, freqs, t["k"], t["v"], t["ks"], t["vs"], tbl, lens, scale,
            window=window, **how)
    if ring:
        return tl.tl_paged_attn_decode_write_rope_ring(
            *rows, slots, pos, freqs, t["k"], t["v"], tbl, lens, scale, window, ring, **how)
    return tl.tl_paged_attn_decode_write_rope(*rows, slots, pos, freqs, t["k"], t["v"], tbl, lens,
                                              scale, window=window, **how)


def case(kind, lens, group, hkv, d, ps, seed, ring=0):
    src = torch.float32 if kind == "f32" else torch.bfloat16
    B, hq = len(lens), group * hkv
    if ring:
        tbl, P = lref.tables([ring * ps] * B, ps, seed)
    else:
        tbl, P = lref.tables(lens, ps, seed)
    slots = np.full(B, -1, np.int64)
    for b, n in enumerate(lens):
        if n > 0:
            at = n - 1
            page = int(tbl[b, at // ps % ring if ring else at // ps])
            slots[b] = page * ps + at % ps
    rows = ref.randn((B, hq + 2 * hkv, d), src, seed + 1).cuda().split([hq, hkv, hkv], 1)
    return tbl.cuda(), P, torch.as_tensor(slots).cuda(), rows, i32([n - 1 for n in lens])


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("group,hkv,d,ps,rot,inter,window", [
    (4, 8, 128, 16, 128, False, 0), (4, 2, 128, 16, 64, True, 0), (1, 3, 128, 32, 128, True, 40),
    (16, 1, 128, 16, 96, False, 0), (5, 2, 128, 16, 20, False, 33), (2, 2, 64, 16, 64, False, 0),
    (2, 2, 64, 16, 6, True, 0),
])
@pytest.mark.parametrize("lens", [[700], [0, 1, 2, 16, 17, 333, 900, 48, 0],
                                  [1 + 7 * b % 300 for b in range(150)]])
def test_same_as_the_two_calls(kind, group, hkv, d, ps, rot, inter, window, lens):
    if kind in ("e4m3", "int8") and d != 128:
        pytest.skip("one-byte pools have heads of 128")
    tbl, P, slots, rows, pos = case(kind, lens, group, hkv, d, ps, seed=1)
    freqs, _ = table(rot, 500000.0)
    lens, scale, m = i32(lens), d ** -0.5, 1.25
    one, two = Pools(kind, P, ps, hkv, d, 3), Pools(kind, P, ps, hkv, d, 3)
    e1, e2 = word(), word()
    q = one.append(*rows, slots, pos, freqs, inter, m, err=e1)
    want = decode(one, q, tbl, lens, scale, window, 0, e1)
    got = step(two, rows, slots, pos, freqs, tbl, lens, scale, window, 0, inter, m, e2)
    assert int(e1.item()) == int(e2.item()) == 0
    assert torch.equal(got, want)
    for n, x in one.t.items():
        assert torch.equal(ref.bits(x), ref.bits(two.t[n])), n
    # against 64 bits too: the attention of the keys held, for a few sequences
    for b in [int(lens.argmax()), int(lens.argmin())]:
        n = int(lens[b])
        if n == 0:
            assert torch.all(got[b] == 0)


@pytest.mark.parametrize("kind", ["bf16", "f32", "int8"])
def test_a_large_batch(kind):
    """More sequences than a block of the plan has threads."""
    lens = [1 + 13 * b % 70 for b in range(1100)]
    tbl, P, slots, rows, pos = case(kind, lens, 2, 2, 128, 16, seed=1)
    freqs, _ = table(128)
    one, two = Pools(kind, P, 16, 2, 128, 3), Pools(kind, P, 16, 2, 128, 3)
    e1, e2 = word(), word()
    q = one.append(*rows, slots, pos, freqs, err=e1)
    want = decode(one, q, tbl, i32(lens), 0.1, 0, 0, e1)
    got = step(two, rows, slots, pos, freqs, tbl, i32(lens), 0.1, 0, 0, False, 1.0, e2)
    assert int(e1.item()) == int(e2.item()) == 0 and torch.equal(got, want)
    for n, x in one.t.items():
        assert torch.equal(ref.bits(x), ref.bits(two.t[n])), n


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_rings(kind):
    ps, ring, window = 16, 4, 50
    lens = [1, 40, 64, 65, 1000, 0]
    tbl, P, slots, rows, pos = case(kind, lens, 4, 2, 128, ps, seed=1, ring=ring)
    freqs, _ = table(128)
    one, two = Pools(kind, P, ps, 2, 128, 3), Pools(kind, P, ps, 2, 128, 3)
    e1, e2 = word(), word()
    q = one.append(*rows, slots, pos, freqs, err=e1)
    want = decode(one, q, tbl, i32(lens), 0.1, window, ring, e1)
    got = step(two, rows, slots, pos, freqs, tbl, i32(lens), 0.1, window, ring, False, 1.0, e2)
    assert int(e1.item()) == int(e2.item()) == 0 and torch.equal(got, want)
    assert torch.equal(ref.bits(one.t["k"]), ref.bits(two.t["k"]))


def test_rows_off_alignment_and_a_given_workspace():
    lens = [33, 700, 5]
    tbl, P, slots, rows, pos = case("bf16", lens, 4, 2, 128, 16, seed=1)
    freqs, _ = table(128)
    size = tl.tl_paged_attn_decode_write_rope_workspace_size(3, 8, 2, 128)
    buf = torch.full((size + 512,), 7, dtype=torch.uint8, device="cuda")
    one, two = Pools("bf16", P, 16, 2, 128, 3), Pools("bf16", P, 16, 2, 128, 3)
    want = step(one, rows, slots, pos, freqs, tbl, i32(lens), 0.1, 0, 0, False, 1.0, None)
    off = []
    for x in rows:
        y = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        off.append(y.copy_(x))
    got = step(two, off, slots, pos, freqs, tbl, i32(lens), 0.1, 0, 0, False, 1.0, None,
               workspace=buf[:size])
    assert torch.equal(got, want) and torch.equal(one.t["k"], two.t["k"])
    assert torch.all(buf[size:] == 7)


def test_errors_are_those_of_the_two_calls():
    lens = [33, 700, 5, 60]
    for kind in ("bf16", "int8"):
        for slot, p, n, bit in ((-7, 32, 33, tl.TL_DEVERR_SLOT_RANGE),
                                (0, -1, 33, tl.TL_DEVERR_CONTEXT_RANGE),
                                (None, 32, 5000, tl.TL_DEVERR_CONTEXT_RANGE)):
            tbl, P, slots, rows, pos = case(kind, lens, 4, 2, 128, 16, seed=1)
            freqs, _ = table(128)
            if slot is not None:
                slots[0] = slot
            pos[0] = p
            ln = i32([n] + lens[1:])
            one, two = Pools(kind, P, 16, 2, 128, 3), Pools(kind, P, 16, 2, 128, 3)
            e1, e2 = word(), word()
            q = one.append(*rows, slots, pos, freqs, err=e1)
            want = decode(one, q, tbl, ln, 0.1, 0, 0, e1)
            got = step(two, rows, slots, pos, freqs, tbl, ln, 0.1, 0, 0, False, 1.0, e2)
            assert int(e1.item()) == int(e2.item()) == bit
            assert torch.equal(got, want)
            assert torch.equal(ref.bits(one.t["k"]), ref.bits(two.t["k"]))


def test_two_captured_steps():
    """Two graphs of a step, replayed in turn over new rows."""
    lens = [33, 700, 5]
    tbl, P, slots, rows, pos = case("bf16", lens, 4, 2, 128, 16, seed=1)
    freqs, _ = table(128)
    ln = i32(lens)
    pools = Pools("bf16", P, 16, 2, 128, 3)

    def run():
        return step(pools, rows, slots, pos, freqs, tbl, ln, 0.1, 0, 0, False, 1.0, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(run())
    for seed in range(3):
        for g, got in zip(graphs, outs):
            for x in rows:
                x.copy_(ref.randn(x.shape, torch.bfloat16, seed))
            pos.copy_(ln - 1 - seed)
            g.replay()
            assert torch.equal(got, run())
