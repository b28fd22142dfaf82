"""Rotary positions on the GPU against the plain 64-bit implementations of
tests/rope_ref.py: rotated rows, the append that rotates queries and keys on
their way, and the compaction that turns kept keys to their new positions."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as lref
from tests import rope_ref as ref
from tests.parity import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def positions(n, seed, padding=True):
    """Far and near, the ends of the range, padding in between."""
    g = np.random.default_rng(seed)
    p = g.integers(0, 1 << 20, n)
    some = [0, 1, 2 ** 31 - 1, 999_983] + ([-1, -5, -2 ** 31] if padding else [])
    p[:min(n, len(some))] = some[:n]
    return g.permutation(p)


# --------------------------------------------------------------------- rows --

def check_rows(x, out, pos, f, inter, m, what):
    """x (CPU), out (CPU): [N, H, d] of one type."""
    pos = np.asarray(pos)
    live = pos >= 0
    # a far position's angle in 64 bits is off by 2^31 x 2^-53 only through its frequency: take
    # the frequencies that the table stands for
    want, err = ref.rotate(ref.as_values(x), np.where(live, pos, 0)[:, None], f, inter, m)
    ref.close(out[live], want[live], err[live], what)
    assert torch.equal(ref.bits(out[~live]), ref.bits(x[~live])), what
    assert torch.equal(ref.bits(out[..., 2 * len(f):]), ref.bits(x[..., 2 * len(f):])), what


def view(kind, n, h, d, dtype):
    """A CUDA tensor [n, h, d] whose tokens lie `kind` apart, and all of its storage."""
    if kind == "tight":
        t = torch.zeros(n, h, d, dtype=dtype, device="cuda")
        return t, t
    if kind == "part":  # some heads of wider rows
        t = torch.zeros(n, h + 3, d, dtype=dtype, device="cuda")
        return t[:, 2:2 + h], t
    # rows that start off a 16-byte boundary
    t = torch.zeros(n * (h * d + 3) + 1, dtype=dtype, device="cuda")
    return t[1:].view(n, h * d + 3)[:, :h * d].view(n, h, d), t


def table(rot, base=10000.0):
    t = ref.table(ref.inv_freq(rot, base))
    return t.cuda(), t.double().numpy() / 2.0 ** 64 * 2 * np.pi


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("h,d,rot,n", [
    (1, 128, 128, 1), (8, 128, 128, 37), (5, 128, 64, 3), (3, 64, 16, 130), (2, 80, 80, 19),
    (2, 80, 32, 19), (3, 96, 96, 7), (4, 256, 256, 9), (1, 192, 48, 33), (40, 128, 128, 65),
    (2, 6, 2, 5), (3, 34, 34, 11), (1, 512, 512, 3), (7, 128, 120, 4), (2, 1040, 1040, 2),
])
def test_rows(dtype, inter, h, d, rot, n):
    freqs, f = table(rot)
    pos = positions(n, seed=n)
    x = ref.randn((n, h, d), dtype, seed=d + n)
    m = 1.25
    for src, dst in (("tight", "tight"), ("part", "tight"), ("off", "part"), ("part", None),
                     ("off", None)):
        xs, xall = view(src, n, h, d, dtype)
        xs.copy_(x)
        before = xall.clone()
        if dst is None:  # in place
            out = tl.tl_rope(xs, i32(pos), freqs, inter, m, out=xs)
            assert out is xs
            kept = xall.clone()
            xs.zero_()
            w = before.clone()
            as_there = torch.as_strided(w, xs.shape, xs.stride(), xs.storage_offset())
            as_there.zero_()
            assert torch.equal(ref.bits(xall), ref.bits(w))  # nothing but its rows was written
            got = torch.as_strided(kept, xs.shape, xs.stride(), xs.storage_offset()).cpu()
        else:
            o, oall = view(dst, n, h, d, dtype)
            oall.fill_(7)
            o.fill_(9)
            tl.tl_rope(xs, i32(pos), freqs, inter, m, out=o)
            got = o.cpu()
            assert torch.equal(ref.bits(xall), ref.bits(before))
            o.fill_(9)
            assert ((oall == 9).sum() == n * h * d) and ((oall == 7).sum() == oall.numel() - n * h * d)
        check_rows(x, got, pos, f, inter, m, f"{src} -> {dst}")


def test_rows_by_default_and_none_at_all():
    freqs, f = table(128, 500000.0)
    x = ref.randn((33, 4, 128), torch.bfloat16, seed=1)
    pos = positions(33, seed=2, padding=False)
    out = tl.tl_rope(x.cuda(), i32(pos), freqs)
    check_rows(x, out.cpu(), pos, f, False, 1.0, "default")
    none = tl.tl_rope(x.cuda()[:0], i32([]), freqs)
    assert none.shape == (0, 4, 128)
    one = x.cuda()[:1].expand(33, 4, 128)  # one row at every position: tokens at stride 0
    out = tl.tl_rope(one, i32(pos), freqs)
    check_rows(x[:1].expand(33, 4, 128), out.cpu(), pos, f, False, 1.0, "expanded")


def test_many_rows():
    """More rows than a wave of blocks; equal to small calls bit for bit."""
    n, h, d = 9001, 33, 128
    freqs, f = table(d)
    pos = positions(n, seed=4)
    x = ref.randn((n, h, d), torch.bfloat16, seed=5).cuda()
    out = tl.tl_rope(x, i32(pos), freqs)
    for a, b in ((0, 1), (4000, 4007), (8990, 9001), (17, 320)):
        assert torch.equal(out[a:b], tl.tl_rope(x[a:b], i32(pos[a:b]), freqs))
    check_rows(x[:64].cpu(), out[:64].cpu(), pos[:64], f, False, 1.0, "head")
    check_rows(x[-64:].cpu(), out[-64:].cpu(), pos[-64:], f, False, 1.0, "tail")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 64), (80, 20)])
def test_negated_table_is_the_gradient(inter, d, rot):
    """The gradient of sum(w . rotation(x)) is the rotation of w by the negated table: against
    the formula, and against differences of it in 64 bits."""
    freqs, f = table(rot)
    n, h, m = 21, 3, 1.5
    pos = positions(n, seed=6)
    live = pos >= 0
    w = ref.randn((n, h, d), torch.float32, seed=8)
    dx = tl.tl_rope(w.cuda(), i32(pos), -freqs, inter, m).cpu()
    wn = w.double().numpy()
    lo, hi = ref.ends(rot, inter)
    a = np.where(live, pos, 0)[:, None, None] * f
    want = wn.copy()
    mm = np.where(live, m, 1.0)[:, None, None]
    want[..., lo] = mm * (wn[..., lo] * np.cos(a) + wn[..., hi] * np.sin(a))
    want[..., hi] = mm * (wn[..., hi] * np.cos(a) - wn[..., lo] * np.sin(a))
    _, err = ref.rotate(wn, np.where(live, pos, 0)[:, None], f, inter, m)
    ref.close(dx, want, err, "gradient")
    g = np.random.default_rng(9)
    x = g.standard_normal((n, h, d))

    def total(z):
        y, _ = ref.rotate(z, np.where(live, pos, 0)[:, None], f, inter, m)
        return (wn * np.where(live[:, None, None], y, z)).sum()
    for _ in range(6):  # the sum is linear: a difference has no truncation, only roundings
        v = g.standard_normal(x.shape)
        diff = (total(x + v) - total(x - v)) / 2
        scale = np.abs(wn).sum() * 4 * m
        assert abs(diff - (dx.double().numpy() * v).sum()) < \
            scale * 2.0 ** -22 + np.abs(v).sum() * 4 * 2.0 ** -22


def test_not_finite_values_stay_in_their_pair():
    freqs, f = table(64)
    for inter in (False, True):
        for dtype in (torch.bfloat16, torch.float32):
            x = ref.randn((3, 2, 128), dtype, seed=3)
            clean = tl.tl_rope(x.cuda(), i32([5, 6, 7]), freqs, inter).cpu()
            lo, hi = ref.ends(64, inter)
            x[0, 1, lo[9]] = float("nan")
            x[1, 0, hi[3]] = float("inf")
            x[2, 0, 100] = float("-inf")  # behind the rotated part: as it is
            out = tl.tl_rope(x.cuda(), i32([5, 6, 7]), freqs, inter).cpu()
            off = torch.zeros(3, 2, 128, dtype=torch.bool)
            for t, g, i in ((0, 1, 9), (1, 0, 3)):
                off[t, g, lo[i]] = off[t, g, hi[i]] = True
            assert not torch.isfinite(out[off].float()).any()
            assert out[2, 0, 100] == float("-inf")
            off[2, 0, 100] = True
            assert torch.equal(out[~off], clean[~off])


# ------------------------------------------------------------------- append --

POOL_KINDS = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3"),
              ("bf16", "int8"), ("f32", "int8")]


class Pools:
    """Pools of some content on the GPU, and that content."""

    def __init__(self, kind, P, ps, hkv, d, seed=0):
        self.kind, self.P, self.ps, self.hkv, self.d = kind, P, ps, hkv, d
        self.t = {}
        g = torch.Generator().manual_seed(seed)
        for n in ("k", "v"):
            if kind == "int8":
                self.t[n] = torch.randint(-127, 128, (P, ps, hkv, d), generator=g, dtype=torch.int8)
                self.t[n + "s"] = torch.rand((P, hkv, ps), generator=g) * 0.04 + 0.005
            else:
                self.t[n] = ref.randn((P, ps, hkv, d), ref.TYPES[kind], seed + 1)
        self.t = {n: x.cuda() for n, x in self.t.items()}
        self.before = {n: x.clone() for n, x in self.t.items()}

    def rows(self, n, slots):
        """(values or codes [N, hkv, d], scales [N, hkv] or None) at slots, on the CPU."""
        x = self.t[n].view(-1, self.hkv, self.d)[slots].cpu()
        if self.kind != "int8":
            return x, None
        s = self.t[n + "s"].transpose(1, 2).reshape(-1, self.hkv)[slots].cpu()
        return x, s

    def untouched_but(self, slots):
        """Every slot but these holds the bytes it held."""
        hit = torch.zeros(self.P * self.ps, dtype=torch.bool, device="cuda")
        hit[slots] = True
        for n, x in self.t.items():
            a, b = x, self.before[n]
            if n.endswith("s"):
                a, b = (y.transpose(1, 2).reshape(-1, self.hkv) for y in (a, b))
            else:
                a, b = (y.view(-1, self.hkv, self.d) for y in (a, b))
            assert torch.equal(ref.bits(a[~hit]), ref.bits(b[~hit])), n

    def append(self, q, k, v, slots, pos, freqs, inter=False, m=1.0, err=None, **kw):
        w = word() if err is None else err
        args = (slots, pos, freqs, inter, m)
        if self.kind == "int8":
            out = tl.tl_kv_cache_write_rope_int8(q, k, v, self.t["k"], self.t["v"], self.t["ks"],
                                                 self.t["vs"], *args, error_word=w, **kw)
        else:
            out = tl.tl_kv_cache_write_rope(q, k, v, self.t["k"], self.t["v"], *args,
                                            error_word=w, **kw)
        if err is None:
            assert int(w.item()) == 0
        return out

    def check(self, k, v, slots, pos, f, inter, m, what):
        """The rows at the live slots (numpy) of K rotated and of V."""
        live = slots >= 0
        at = torch.as_tensor(slots[live]).cuda()
        k, v = (ref.as_values(x)[live] for x in (k, v))
        kw, ke = ref.rotate(k, pos[live][:, None], f, inter, m)
        for n, want, err in (("k", kw, ke), ("v", v, np.zeros_like(v))):
            got, scales = self.rows(n, at)
            if self.kind == "int8":
                ref.close_int8(got, scales, want, err, f"{what} {n}")
            else:
                ref.close(got, want, err, f"{what} {n}")
        self.untouched_but(at)


def slots_of(n, P, ps, seed, skip=0.2):
    """Distinct slots, some tokens without one (numpy int64)."""
    g = np.random.default_rng(seed)
    s = g.permutation(P * ps)[:n].astype(np.int64)
    s[g.random(n) < skip] = -1
    return s


@pytest.mark.parametrize("src,kind", POOL_KINDS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot,ps,n", [
    (32, 8, 128, 128, 16, 1), (8, 2, 128, 128, 16, 70), (4, 4, 64, 32, 8, 33), (0, 3, 64, 64, 5, 20),
    (5, 1, 128, 96, 32, 9), (6, 2, 80, 80, 16, 21), (3, 1, 48, 20, 4, 6), (40, 8, 128, 64, 64, 131),
    (2, 2, 256, 256, 16, 5),
])
def test_append(src, kind, inter, hq, hkv, d, rot, ps, n):
    P = n // ps + 3
    freqs, f = table(rot, 500000.0)
    m = 1.25
    pools = Pools(kind, P, ps, hkv, d, seed=n)
    slots, pos = slots_of(n, P, ps, seed=1), positions(n, seed=2)
    pos = np.where((slots >= 0) & (pos < 0), 77, pos)
    T = ref.TYPES[src]
    rows = ref.randn((n, hq + 2 * hkv, d), T, seed=3)
    fused = rows.cuda()
    q, k, v = fused.split([hq, hkv, hkv], 1)
    args = (torch.as_tensor(slots).cuda(), i32(pos), freqs, inter, m)
    qc, kc, vc = rows.split([hq, hkv, hkv], 1)
    out = pools.append(q if hq else None, k, v, *args)
    if hq:
        assert out.shape == (n, hq, d) and out.dtype == T
        check_rows(qc, out.cpu(), pos, f, inter, m, "q")
    else:
        assert out is None
    assert torch.equal(ref.bits(fused), ref.bits(rows.cuda()))
    pools.check(kc, vc, slots, pos, f, inter, m, kind)
    # separate rows, q in place in the fused ones: the same bits
    again = Pools(kind, P, ps, hkv, d, seed=n)
    got = again.append(q if hq else None, k.contiguous(), v.contiguous(), *args,
                       q_out=q if hq else None)
    for name, x in pools.t.items():
        assert torch.equal(ref.bits(x), ref.bits(again.t[name])), name
    if hq:
        assert got is q and torch.equal(ref.bits(q), ref.bits(out))
        assert torch.equal(ref.bits(fused[:, hq:]), ref.bits(rows.cuda()[:, hq:]))


@pytest.mark.parametrize("src,kind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "int8"),
                                      ("bf16", "e4m3")])
def test_append_off_alignment(src, kind):
    """Rows off 16-byte boundaries: the same bits as aligned ones."""
    n, hq, hkv, d, ps = 23, 3, 2, 128, 16
    freqs, _ = table(128)
    T = ref.TYPES[src]
    slots, pos = slots_of(n, 4, ps, 1), positions(n, 2, padding=False)
    args = (torch.as_tensor(slots).cuda(), i32(pos), freqs)
    rows = {h: ref.randn((n, c, d), T, seed=c).cuda() for h, c in (("q", hq), ("k", hkv), ("v", hkv))}
    one, two = Pools(kind, 4, ps, hkv, d), Pools(kind, 4, ps, hkv, d)
    a = one.append(rows["q"], rows["k"], rows["v"], *args)
    off = {}
    for h, x in rows.items():
        off[h], _ = view("off", n, x.shape[1], d, T)
        off[h].copy_(x)
    b = two.append(off["q"], off["k"], off["v"], *args)
    assert torch.equal(a, b)
    for name, x in one.t.items():
        assert torch.equal(ref.bits(x), ref.bits(two.t[name])), name


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
def test_append_unrotated_rows_are_the_plain_write(kind):
    """At position 0 with rope_scale 1 keys are as they are: the bytes of the plain write, V's at
    any position (a NaN's payload too)."""
    n, hkv, d, ps, P = 37, 2, 128, 16, 5
    src = ref.TYPES[kind if kind in ("bf16", "f32") else "bf16"]
    k, v = ref.randn((n, hkv, d), src, 1).cuda(), ref.randn((n, hkv, d), src, 2).cuda()
    if kind != "int8":
        v.view(torch.int16 if src == torch.bfloat16 else torch.int32)[3, 1, 5] = -3
    slots = torch.as_tensor(slots_of(n, P, ps, 3)).cuda()
    freqs, _ = table(128)
    a, b = Pools(kind, P, ps, hkv, d), Pools(kind, P, ps, hkv, d)
    a.append(None, k, v, slots, i32([0] * n), freqs)
    write = {"int8": tl.tl_kv_cache_write_int8, "e4m3": tl.tl_kv_cache_write_fp8}.get(
        kind, tl.tl_kv_cache_write)
    write(k, v, *[b.t[x] for x in (("k", "v", "ks", "vs") if kind == "int8" else ("k", "v"))], slots)
    for name, x in a.t.items():
        assert torch.equal(ref.bits(x), ref.bits(b.t[name])), name


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_append_reports_and_skips_bad_rows(kind):
    n, hq, hkv, d, ps, P = 9, 4, 2, 128, 16, 2
    freqs, f = table(128)
    k, v = (ref.randn((n, hkv, d), torch.bfloat16, s).cuda() for s in (1, 2))
    q = ref.randn((n, hq, d), torch.bfloat16, 3)
    good = np.array([0, 1, 2, 3, -1, 5, 6, 7, 8])
    for bad, pos2, bit in ((32, 4, tl.TL_DEVERR_SLOT_RANGE), (-2, 4, tl.TL_DEVERR_SLOT_RANGE),
                           (2 ** 40, 4, tl.TL_DEVERR_SLOT_RANGE), (9, -1, tl.TL_DEVERR_CONTEXT_RANGE),
                           (9, -2 ** 31, tl.TL_DEVERR_CONTEXT_RANGE)):
        slots, pos = good.copy(), np.arange(n) + 100
        slots[5], pos[5] = bad, pos2
        pools, w = Pools(kind, P, ps, hkv, d), word()
        out = pools.append(q.cuda(), k, v, torch.as_tensor(slots).cuda(), i32(pos), freqs, err=w)
        assert int(w.item()) == bit
        slots[5] = -1
        pools.check(k, v, slots, pos, f, False, 1.0, kind)
        check_rows(q, out.cpu(), pos, f, False, 1.0, "q")


def test_append_int8_not_finite():
    n, hkv, d, ps = 4, 2, 128, 16
    freqs, _ = table(128)
    for bad in (float("nan"), float("inf"), float("-inf")):
        k, v = (ref.randn((n, hkv, d), torch.bfloat16, s) for s in (1, 2))
        clean, hurt, w = Pools("int8", 2, ps, hkv, d), Pools("int8", 2, ps, hkv, d), word()
        args = (torch.arange(4).cuda(), i32([3, 4, 5, 6]), freqs)
        k[2, 1, 7] = k[2, 1, 71] = 0.0
        clean.append(None, k.cuda(), v.cuda(), *args)
        k[2, 1, 7] = bad  # element 7 turns with element 71
        hurt.append(None, k.cuda(), v.cuda(), *args, err=w)
        assert int(w.item()) == tl.TL_DEVERR_VALUE_RANGE
        for name in clean.t:  # codes 0 for the pair, everything else as without it
            assert torch.equal(clean.t[name], hurt.t[name]), name


def test_append_e4m3_clamps_what_the_rotation_enlarges():
    """(440, 440) turned by an eighth of a turn is (0, 622): written as 448."""
    freqs = torch.tensor([1 << 61] * 64, dtype=torch.int64).cuda()
    k = torch.full((1, 1, 128), 440.0, dtype=torch.bfloat16)
    pools = Pools("e4m3", 1, 16, 1, 128)
    pools.append(None, k.cuda(), k.cuda(), torch.tensor([3]).cuda(), i32([1]), freqs)
    got = pools.t["k"].view(16, 128)[3].float().cpu()
    assert torch.all(got[:64].abs() < 1e-3) and torch.all(got[64:] == 448)


def test_append_of_nothing():
    pools = Pools("bf16", 2, 16, 2, 128)
    freqs, _ = table(128)
    z = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = pools.append(z, z[:, :2], z[:, :2], torch.zeros(0, dtype=torch.int64).cuda(), i32([]), freqs)
    assert out.shape == (0, 4, 128)
    pools.untouched_but(torch.zeros(0, dtype=torch.int64).cuda())


def test_append_far_slots():
    """Element offsets past 2^31 and 2^32 in a long pool, the last slot among them."""
    P, ps, hkv, d = 140_000, 32, 8, 128  # 4.6 x 10^9 elements
    k_pool, v_pool = (torch.zeros((P, ps, hkv, d), dtype=torch.float8_e4m3fn, device="cuda")
                      for _ in range(2))
    n = 6
    slots = torch.tensor([0, 2_097_151, 2_097_152, 4_194_304, 4_300_001, P * ps - 1])
    freqs, f = table(128)
    k, v = (ref.randn((n, hkv, d), torch.bfloat16, s) for s in (1, 2))
    pos = np.arange(n) * 1000
    w = word()
    tl.tl_kv_cache_write_rope(None, k.cuda(), v.cuda(), k_pool, v_pool, slots.cuda(), i32(pos),
                              freqs, error_word=w)
    assert int(w.item()) == 0
    want, err = ref.rotate(ref.as_values(k), pos[:, None], f, False)
    got = k_pool.view(-1, hkv, d)[slots.cuda()].cpu()
    ref.close(got, want, err, "k")
    ref.close(v_pool.view(-1, hkv, d)[slots.cuda()].cpu(), ref.as_values(v), np.zeros(v.shape), "v")


# --------------------------------------------------------------- compaction --

def keep_lists(lens, hkv, n, first, seed):
    g = np.random.default_rng(seed)
    keep = np.full((len(lens), hkv, n), -1, np.int32)
    for b, L in enumerate(lens):
        for h in range(hkv):
            m = min(L, n)
            f = min(first, m)
            rest = np.sort(g.permutation(np.arange(f, L))[:m - f])
            keep[b, h, :m] = np.concatenate([np.arange(f), rest])
    return keep, np.minimum(lens, n).astype(np.int32)


def run_compact(pools, tbl, lens, keep, new, freqs, inter, err=None, mass=None, **kw):
    w = word() if err is None else err
    args = (tbl.cuda(), i32(lens), i32(keep), i32(new), freqs, inter)
    if pools.kind == "int8":
        tl.tl_kv_cache_compact_rope_int8(pools.t["k"], pools.t["v"], pools.t["ks"], pools.t["vs"],
                                         *args, mass=mass, error_word=w, **kw)
    else:
        tl.tl_kv_cache_compact_rope(pools.t["k"], pools.t["v"], *args, mass=mass, error_word=w,
                                    **kw)
    if err is None:
        assert int(w.item()) == 0


def check_compact(pools, tbl, lens, keep, new, f, inter, skip=()):
    """Moved keys turned, V and rows that stay by their bytes, all else as it was; skip: (b, h, j)
    that the call was to leave."""
    ps, hkv, d = pools.ps, pools.hkv, pools.d
    e4m3 = pools.kind == "e4m3"  # by bytes: the CPU indexes no such type
    now, old = ({n: x.cpu().view(torch.uint8) if e4m3 else x.cpu() for n, x in y.items()}
                for y in (pools.t, pools.before))

    def typed(x):
        return x.contiguous().view(torch.float8_e4m3fn) if e4m3 else x
    flat = {n: (x.transpose(1, 2).reshape(-1, hkv) if n.endswith("s") else x.view(-1, hkv, d))
            for n, x in old.items()}
    got = {n: (x.transpose(1, 2).reshape(-1, hkv) if n.endswith("s") else x.view(-1, hkv, d))
           for n, x in now.items()}
    stay = {n: x.clone() for n, x in flat.items()}  # what everything but moved keys has to be
    for b, n in enumerate(new):
        for h in range(hkv):
            j = np.array([j for j in range(n) if keep[b, h, j] != j and (b, h, j) not in skip],
                         dtype=np.int64)
            if not len(j):
                continue
            i = keep[b, h, j].astype(np.int64)
            row = tbl[b].long().numpy()
            to, frm = row[j // ps] * ps + j % ps, row[i // ps] * ps + i % ps
            x = ref.as_values(typed(flat["k"][frm, h]))
            if pools.kind == "int8":
                x = (x.astype(np.float32) * flat["ks"][frm, h].numpy()[:, None]).astype(np.float64)
            want, err = ref.rotate(x, j - i, f, inter)
            if pools.kind == "int8":
                ref.close_int8(got["k"][to, h], got["ks"][to, h], want, err, f"b{b} h{h}")
                stay["ks"][to, h], stay["vs"][to, h] = got["ks"][to, h], flat["vs"][frm, h]
            else:
                ref.close(typed(got["k"][to, h]), want, err, f"b{b} h{h}")
                if 2 * len(f) < d:  # behind the rotated part
                    tail = slice(2 * len(f), d)
                    assert torch.equal(ref.bits(got["k"][to, h][:, tail]),
                                       ref.bits(flat["k"][frm, h][:, tail]))
            stay["k"][to, h], stay["v"][to, h] = got["k"][to, h], flat["v"][frm, h]
    for n in got:
        assert torch.equal(ref.bits(got[n]), ref.bits(stay[n])), n


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lens,n,first,hkv,d,rot,ps", [
    ([0, 1, 2, 16, 17, 333, 900, 48], 40, 4, 2, 128, 128, 16),  # few rows, shared by CTAs
    ([700], 650, 0, 1, 128, 64, 16), ([64, 100, 5], 100, 1, 3, 64, 16, 24),
    ([90 + 7 * b for b in range(40)], 77, 2, 4, 128, 128, 8),   # a CTA a row
    ([33] * 90, 20, 3, 4, 64, 64, 16), ([300, 40], 129, 0, 2, 256, 128, 5),
])
def test_compact(kind, inter, lens, n, first, hkv, d, rot, ps):
    tbl, P = lref.tables(lens, ps, seed=1)
    pools = Pools(kind, P, ps, hkv, d, seed=2)
    keep, new = keep_lists(lens, hkv, n, first, seed=3)
    freqs, f = table(rot)
    run_compact(pools, tbl, lens, keep, new, freqs, inter)
    check_compact(pools, tbl, lens, keep, new, f, inter)


def test_compact_with_mass_is_the_plain_one_but_for_keys():
    lens, n, hkv, d, ps = [200, 31, 90], 50, 2, 128, 16
    tbl, P = lref.tables(lens, ps, seed=1)
    keep, new = keep_lists(lens, hkv, n, 4, seed=3)
    freqs, f = table(128)
    for kind in ("bf16", "int8"):
        a, b = Pools(kind, P, ps, hkv, d, seed=2), Pools(kind, P, ps, hkv, d, seed=2)
        m0 = torch.rand((3, hkv, 207), generator=torch.Generator().manual_seed(4))
        ma, mb = m0.cuda(), m0.cuda()
        run_compact(a, tbl, lens, keep, new, freqs, False, mass=ma)
        args = (tbl.cuda(), i32(lens), i32(keep), i32(new))
        if kind == "int8":
            tl.tl_kv_cache_compact_int8(b.t["k"], b.t["v"], b.t["ks"], b.t["vs"], *args, mass=mb)
        else:
            tl.tl_kv_cache_compact(b.t["k"], b.t["v"], *args, mass=mb)
        assert torch.equal(ma, mb) and torch.equal(a.t["v"], b.t["v"])
        if kind == "int8":
            assert torch.equal(a.t["vs"], b.t["vs"])
        check_compact(a, tbl, lens, keep, new, f, False)
        # turns of nothing at all: the plain compaction's bytes
        c = Pools("bf16", P, ps, hkv, d, seed=2)
        e = Pools("bf16", P, ps, hkv, d, seed=2)
        run_compact(c, tbl, lens, keep, new, torch.zeros_like(freqs), False)
        tl.tl_kv_cache_compact(e.t["k"], e.t["v"], *args)
        assert torch.equal(ref.bits(c.t["k"]), ref.bits(e.t["k"]))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_compact_reports_and_skips(kind):
    lens, n, hkv, d, ps = [60, 50, 40, 30], 20, 2, 128, 16
    freqs, f = table(128)
    tbl, P = lref.tables(lens, ps, seed=1)
    keep, new = keep_lists(lens, hkv, n, 2, seed=3)
    # an entry behind the sequence, one before its own place, one far out
    skip = [(0, 1, 7), (1, 0, 9), (2, 0, 5)]
    for (b, h, j), bad in zip(skip, (60, 8, 2 ** 31 - 1)):
        keep[b, h, j] = bad
    pools, w = Pools(kind, P, ps, hkv, d, seed=2), word()
    run_compact(pools, tbl, lens, keep, new, freqs, False, err=w)
    assert int(w.item()) == tl.TL_DEVERR_CONTEXT_RANGE
    check_compact(pools, tbl, lens, keep, new, f, False, skip=set(skip))
    # new lengths out of range: the sequence stays; a page outside the pool: its rows stay
    keep, new = keep_lists(lens, hkv, n, 2, seed=3)
    for value in (-1, 21, 61):
        pools, w = Pools(kind, P, ps, hkv, d, seed=2), word()
        bad = new.copy()
        bad[0] = value
        run_compact(pools, tbl, lens, keep, bad, freqs, False, err=w)
        assert int(w.item()) == tl.TL_DEVERR_CONTEXT_RANGE
        bad[0] = 0
        check_compact(pools, tbl, lens, keep, bad, f, False)
    pools, w = Pools(kind, P, ps, hkv, d, seed=2), word()
    hurt = tbl.clone()
    hurt[1, 1] = P  # positions 16 .. 31 of sequence 1
    run_compact(pools, hurt, lens, keep, new, freqs, False, err=w)
    assert int(w.item()) == tl.TL_DEVERR_PAGE_RANGE
    gone = {(1, h, j) for h in range(hkv) for j in range(new[1])
            if 16 <= j < 32 or 16 <= keep[1, h, j] < 32}
    check_compact(pools, tbl, lens, keep, new, f, False, skip=gone)


def test_compact_twice_follows_the_positions():
    """Two cuts one behind the other: keys end within two roundings of one rotated at its place."""
    L, hkv, d, ps = 400, 2, 128, 16
    freqs, f = table(128, 500000.0)
    tbl, P = lref.tables([L], ps, seed=1)
    raw = ref.randn((L, hkv, d), torch.float32, seed=5)
    pools = Pools("f32", P, ps, hkv, d)
    slots = tbl[0, torch.arange(L) // ps].long() * ps + torch.arange(L) % ps
    pools.append(None, raw.cuda(), raw.cuda(), slots.cuda(), i32(np.arange(L)), freqs)
    ids = np.tile(np.arange(L), (hkv, 1))
    lens = [L]
    for n, seed in ((250, 1), (90, 2)):
        keep, new = keep_lists(lens, hkv, n, 4, seed)
        run_compact(pools, tbl, lens, keep, new, freqs, False)
        ids = np.stack([ids[h][keep[0, h]] for h in range(hkv)])
        lens = [n]
    got, _ = pools.rows("k", slots[:90].cuda())
    for h in range(hkv):
        x = raw[torch.as_tensor(ids[h]), h].double().numpy()
        want, err = ref.rotate(x, np.arange(90), f, False)
        # three rotations, each by at most the bound and a rounding of values up to |lo| + |hi|
        ref.close(got[:, h], want, 3 * err * 1.01 + 3 * 2.0 ** -24 * err / (2.6 * 2.0 ** -23), f"h{h}")


# ----------------------------------------------------------------- together --

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_a_conversation_cut_and_continued(kind):
    """A prompt is appended and attended, decode steps gather weights, the cache is cut with its
    positions closed up, and the steps behind it go on at the new length.  At every step the keys
    held are the raw keys rotated at the places they have now, to the roundings of their type, and
    the attention is that of the keys, values and queries held."""
    hq, hkv, d, ps, B, T, room = 8, 2, 128, 16, 3, 70, 100
    group = hq // hkv
    lens = [70, 41, 0]
    scale = d ** -0.5
    tbl, P = lref.tables([room] * B, ps, seed=1)
    freqs, f = table(128)
    rng = torch.Generator().manual_seed(7)
    pools = Pools(kind, P, ps, hkv, d)
    t = pools.t
    mass = torch.zeros(B, hkv, 112, device="cuda")
    raw = {n: np.zeros((B, room, hkv, d)) for n in "kv"}  # by token, in order of arrival
    came = list(lens)                                     # tokens of each sequence so far
    ids = [np.tile(np.arange(n), (hkv, 1)) for n in lens]  # the token at each place of a head
    cut = [0] * B                                         # places a cut may have moved

    def place(b, p):
        return int(tbl[b, p // ps]) * ps + p % ps

    def held(n, b):
        at = torch.tensor([place(b, p) for p in range(lens[b])]).cuda()
        x, s = pools.rows(n, at)
        x = ref.as_values(x)
        return x if s is None else x * s.double().numpy()[..., None]

    def check_cache(b):
        """A pair of keys (sum of magnitudes A, up to sqrt 2 A once rotated) is rounded when it is
        written, and turned and rounded once more if a cut moved it: each rounding is off by half
        a step r of a value, and a turn adds the pair's two errors.  int8: half a code, a 254th of
        the row's largest value."""
        k = held("k", b)
        for h in range(hkv):
            x = raw["k"][b, ids[b][h], h]
            want, err = ref.rotate(x, np.arange(lens[b]), f, False)
            lo, hi = ref.ends(128, False)
            A = np.concatenate([np.abs(x[:, lo]) + np.abs(x[:, hi])] * 2, 1)
            moved = (np.arange(lens[b]) < cut[b])[:, None]
            if kind == "int8":
                one = np.sqrt(2) * np.abs(x).max(1, keepdims=True) / 254 * 1.01
                tol = np.where(moved, 3 * one, one)
            else:
                r = ref.HALF_STEP[ref.TYPES[kind]]
                one = np.sqrt(2) * A * r * (1 + r) + (2.0 ** -10 if kind == "e4m3" else 0)
                tol = np.where(moved, 3 * one, one)
            assert (np.abs(k[:, h] - want) <= tol + 3 * err).all(), (b, h)

    def attention(q, b):
        """Of the rotated queries [hq, d] (as held) over the keys and values held."""
        k, v = held("k", b), held("v", b)
        out = np.zeros((hq, d))
        for h in range(hkv):
            z = q[h * group:(h + 1) * group] @ k[:, h].T * scale
            w = np.exp(z - z.max(1, keepdims=True))
            out[h * group:(h + 1) * group] = w / w.sum(1, keepdims=True) @ v[:, h]
        return out

    # the prompts, right-aligned
    x = torch.randn((B * T, hq + 2 * hkv, d), generator=rng).bfloat16()
    pos = np.array([[c - (T - n) if c >= T - n else -1 for c in range(T)] for n in lens])
    slots = np.array([[place(b, p) if p >= 0 else -1 for p in pos[b]] for b in range(B)])
    for b in range(B):
        for c in range(T):
            if pos[b, c] >= 0:
                raw["k"][b, pos[b, c]] = x[b * T + c, hq:hq + hkv].double()
                raw["v"][b, pos[b, c]] = x[b * T + c, hq + hkv:].double()
    q, k, v = x.cuda().split([hq, hkv, hkv], 1)
    qr = pools.append(q, k, v, torch.as_tensor(slots.ravel()).cuda(), i32(pos.ravel()), freqs)
    qr = qr.view(B, T, hq, d)
    if kind == "int8":
        pre = tl.tl_paged_attn_prefill_int8(qr, t["k"], t["v"], t["ks"], t["vs"], tbl.cuda(),
                                            i32(pos), scale)
    else:
        pre = tl.tl_paged_attn_prefill(qr, t["k"], t["v"], tbl.cuda(), i32(pos), scale)
    for b in range(B):
        if lens[b]:
            check_cache(b)
            assert_close(pre[b, T - 1], attention(qr[b, T - 1].cpu().double().numpy(), b), "prefill")

    def step():
        x = torch.randn((B, hq + 2 * hkv, d), generator=rng).bfloat16()
        live = [b for b in range(B) if lens[b] > 0]
        s = torch.tensor([place(b, lens[b]) if b in live else -1 for b in range(B)])
        p = [lens[b] if b in live else -1 for b in range(B)]
        q, k, v = x.cuda().split([hq, hkv, hkv], 1)
        qr = pools.append(q, k, v, s.cuda(), i32(p), freqs)
        for b in live:
            raw["k"][b, came[b]] = x[b, hq:hq + hkv].double()
            raw["v"][b, came[b]] = x[b, hq + hkv:].double()
            ids[b] = np.concatenate([ids[b], np.full((hkv, 1), came[b])], 1)
            came[b] += 1
            lens[b] += 1
        a = (tbl.cuda(), i32(lens), mass, scale)
        if kind == "int8":
            out = tl.tl_paged_attn_decode_mass_int8(qr[:, None], t["k"], t["v"], t["ks"], t["vs"], *a)
        else:
            out = tl.tl_paged_attn_decode_mass(qr[:, None], t["k"], t["v"], *a)
        for b in range(B):
            if lens[b] == 0:
                assert torch.all(out[b] == 0)
                continue
            check_cache(b)
            assert_close(out[b, 0], attention(qr[b].cpu().double().numpy(), b), f"step b{b}")

    for _ in range(3):
        step()
    keep, new = tl.tl_kv_evict_select(mass, i32(lens), 32, keep_first=2, keep_last=8)
    args = (tbl.cuda(), i32(lens), keep, new, freqs)
    if kind == "int8":
        tl.tl_kv_cache_compact_rope_int8(t["k"], t["v"], t["ks"], t["vs"], *args, mass=mass)
    else:
        tl.tl_kv_cache_compact_rope(t["k"], t["v"], *args, mass=mass)
    kp = keep.cpu().numpy()
    lens = new.tolist()
    assert lens == [32, 32, 0]
    for b in range(2):
        ids[b] = np.stack([ids[b][h][kp[b, h]] for h in range(hkv)])
        cut[b] = 32
        check_cache(b)
    for _ in range(3):
        step()


def test_a_captured_step_replayed():
    """Append, compaction and rows captured into a graph and replayed over new values; two
    graphs of the same calls beside each other."""
    n, hq, hkv, d, ps = 5, 8, 2, 128, 16
    freqs, _ = table(128)
    lens = [60, 33]
    tbl, P = lref.tables(lens, ps, seed=1)
    keep, new = keep_lists(lens, hkv, 30, 2, seed=3)
    pools = Pools("bf16", P, ps, hkv, d)
    rows = torch.zeros(n, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    q, k, v = rows.split([hq, hkv, hkv], 1)
    slots, pos = torch.arange(n).cuda() * 3, i32([0] * n)
    c = [x.cuda() for x in (tbl, torch.tensor(lens, dtype=torch.int32), torch.as_tensor(keep),
                            torch.as_tensor(new))]

    def step():
        out = tl.tl_kv_cache_write_rope(q, k, v, pools.t["k"], pools.t["v"], slots, pos, freqs)
        tl.tl_kv_cache_compact_rope(pools.t["k"], pools.t["v"], *c, freqs)
        return out, tl.tl_rope(out, pos, freqs, True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    for seed in range(3):
        for g, got in zip(graphs, outs):
            for x, b in pools.t.items():
                b.copy_(pools.before[x])
            rows.copy_(ref.randn(rows.shape, torch.bfloat16, seed))
            pos.copy_(torch.arange(n) * 1000 + seed)
            g.replay()
            torch.cuda.synchronize()
            held = {x: b.clone() for x, b in pools.t.items()}
            for x, b in pools.t.items():
                b.copy_(pools.before[x])
            want = step()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            for x, b in pools.t.items():
                assert torch.equal(b, held[x]), x


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_compact_lists_in_any_order(kind):
    """Entries at or behind their place, in no order and some of them twice; many heads and few."""
    for lens, hkv in (([500, 300], 1), ([400] * 60, 3)):
        n, d, ps = 120, 128, 16
        tbl, P = lref.tables(lens, ps, seed=1)
        g = np.random.default_rng(5)
        keep = np.stack([[np.array([g.integers(j, L) for j in range(n)]) for _ in range(hkv)]
                         for L in lens]).astype(np.int32)
        keep[:, :, 7] = keep[:, :, 3] = 40
        keep[:, :, ::10] = np.arange(0, n, 10)
        new = np.full(len(lens), n, np.int32)
        freqs, f = table(128)
        pools = Pools(kind, P, ps, hkv, d, seed=2)
        run_compact(pools, tbl, lens, keep, new, freqs, False)
        check_compact(pools, tbl, lens, keep, new, f, False)


def test_compact_by_the_largest_shift():
    """The last of 200,000 keys moved to the front: 199,999 positions back."""
    L, hkv, d, ps = 200_000, 1, 128, 64
    tbl, P = lref.tables([L], ps, seed=1)
    pools = Pools("bf16", P, ps, hkv, d, seed=2)
    keep, new = np.array([[[L - 1, 1, L - 2]]], np.int32), np.array([3], np.int32)
    freqs, f = table(128, 500000.0)
    run_compact(pools, tbl, [L], keep, new, freqs, True)
    check_compact(pools, tbl, [L], keep, new, f, True)


def test_compact_of_nothing():
    """No length, or nothing that moves: every byte stays."""
    tbl, P = lref.tables([40, 30], 16, seed=1)
    pools = Pools("bf16", P, 16, 2, 128, seed=2)
    freqs, f = table(128)
    keep = np.tile(np.arange(30, dtype=np.int32), (2, 2, 1))
    for lens, new in (([40, 30], [30, 30]), ([0, 0], [0, 0]), ([40, 30], [0, 0]),
                      ([-3, 30], [0, 30])):
        run_compact(pools, tbl, lens, keep, new, freqs, False)
        check_compact(pools, tbl, lens, keep, new, f, False)


def test_appends_on_two_streams_at_once():
    """Disjoint slots of one pool, written by two streams' calls that overlap."""
    n, hq, hkv, d, ps = 2048, 8, 2, 128, 16
    freqs, f = table(128)
    pools = Pools("bf16", 2 * n // ps, ps, hkv, d)
    halves = []
    for i in range(2):
        rows = ref.randn((n, hq + 2 * hkv, d), torch.bfloat16, i).cuda()
        halves.append((rows, torch.arange(i, 2 * n, 2).cuda(), i32(np.arange(n) * 3 + i)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    w = word()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (rows, slots, pos) in zip(streams, halves):
            with torch.cuda.stream(s):
                q, k, v = rows.split([hq, hkv, hkv], 1)
                pools.append(q, k, v, slots, pos, freqs, err=w)
    torch.cuda.synchronize()
    assert int(w.item()) == 0
    k = torch.empty(2 * n, hkv, d, dtype=torch.bfloat16)
    v = torch.empty_like(k)
    pos = np.empty(2 * n, np.int64)
    for i, (rows, slots, p) in enumerate(halves):
        k[i::2], v[i::2] = rows[:, hq:hq + hkv].cpu(), rows[:, hq + hkv:].cpu()
        pos[i::2] = p.cpu().numpy()
    pools.check(k, v, np.arange(2 * n), pos, f, False, 1.0, "two streams")


def test_compact_far_pages():
    """Element offsets past 2^31 and 2^32: a sequence on the last pages of a long pool."""
    P, ps, hkv, d = 140_000, 32, 8, 128  # 4.6 x 10^9 elements
    pages = [139_999, 66_000, 5, 131_072]
    n = 100
    small = ref.randn((len(pages), ps, hkv, d), torch.float8_e4m3fn, 1)
    pools = [torch.zeros((P, ps, hkv, d), dtype=torch.float8_e4m3fn, device="cuda")
             for _ in range(2)]
    at = torch.tensor(pages).cuda()
    for x in pools:
        x.view(torch.uint8)[at] = small.view(torch.uint8).cuda()
    keep = np.tile(np.arange(0, n, 2, dtype=np.int32), (1, hkv, 1))
    freqs, f = table(128)
    w = word()
    tl.tl_kv_cache_compact_rope(*pools, i32([pages]), i32([n]), i32(keep), i32([n // 2]), freqs,
                                error_word=w)
    assert int(w.item()) == 0
    rows = ref.as_values(small).reshape(-1, hkv, d)
    j = np.arange(1, n // 2)
    got = [x.view(torch.uint8)[at].cpu().view(torch.float8_e4m3fn).reshape(-1, hkv, d)
           for x in pools]
    want, err = ref.rotate(rows[2 * j], -j[:, None], f, False)
    ref.close(got[0][1:n // 2], want, err, "k")
    assert np.array_equal(ref.as_values(got[1][1:n // 2]), rows[2 * j])
    # nothing else of the long pools was written
    for x in pools:
        x.view(torch.uint8)[at] = 0
        assert not bool(x.view(torch.int32).any())


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("B,hkv,n", [(1, 1, 700), (1, 8, 700), (1, 10, 300), (5, 3, 300), (8, 8, 200),
                                     (16, 8, 150), (19, 8, 90), (25, 4, 90)])
def test_compact_shared_by_clusters_of_every_size(kind, B, hkv, n):
    """From few rows, each shared by many CTAs, to as many as there are places."""
    lens = [n + 37 * b % 400 for b in range(B)]
    tbl, P = lref.tables(lens, 16, seed=1)
    pools = Pools(kind, P, 16, hkv, 128, seed=2)
    keep, new = keep_lists(lens, hkv, n * 2 // 3, 3, seed=3)
    freqs, f = table(64)
    mass = torch.rand((B, hkv, 1200), generator=torch.Generator().manual_seed(1))
    m = mass.cuda()
    run_compact(pools, tbl, lens, keep, new, freqs, True, mass=m)
    check_compact(pools, tbl, lens, keep, new, f, True)
    for b in range(B):
        for h in range(hkv):
            want = mass[b, h].clone()
            want[:new[b]] = mass[b, h][torch.as_tensor(keep[b, h, :new[b]]).long()]
            want[new[b]:lens[b]] = 0
            assert torch.equal(m[b, h].cpu(), want)
