"""Attention that gathers each key's weight, the selection of the keys that
stay and the in-place compaction, against the plain implementations of
tests/long_context_ref.py: selections and moved bytes equal bit for bit,
attention and masses within derived tolerances."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


# -------------------------------------------------------------------- mass --

def run_mass(pools, q, table, lens, mass, scale, window=0, err=None, p=None, **kw):
    p = pools.gpu() if p is None else p
    w = word() if err is None else err
    args = (table.cuda(), i32(lens), mass, scale)
    if pools.kind == "int8":
        out = tl.tl_paged_attn_decode_mass_int8(q.cuda(), p["k"], p["v"], p["ks"], p["vs"], *args,
                                                window=window, error_word=w, **kw)
    else:
        out = tl.tl_paged_attn_decode_mass(q.cuda(), p["k"], p["v"], *args, window=window,
                                           error_word=w, **kw)
    if err is None:
        assert int(w.item()) == 0
    return out


def check_mass(out, mass, mass0, pools, q, table, lens, scale, window, what):
    k, v = pools.values("k").double().numpy(), pools.values("v").double().numpy()
    hkv, ps, d = pools.hkv, pools.ps, pools.d
    units = pools.units("v").numpy()
    B, T, hq, _ = q.shape
    group = hq // hkv
    qn = q.double().numpy()
    mass, mass0 = mass.cpu().double().numpy(), mass0.double().numpy()
    for b, n in enumerate(lens):
        if n <= 0:
            assert torch.all(out[b] == 0) and np.array_equal(mass[b], mass0[b])
            continue
        pg = table[b, :-(-n // ps)].long().numpy()
        for g in range(hkv):
            kk = k[pg][:, :, g].reshape(-1, d)[:n]
            vv = v[pg][:, :, g].reshape(-1, d)[:n]
            flat = units[pg][:, :, g].reshape(-1, d)[:n].sum(0)
            add = np.zeros(n)
            seen = np.zeros(n, bool)
            es = 0.0
            for t in range(T):
                rows = slice(g * group, (g + 1) * group)
                pos = n - T + t
                key = np.arange(n)
                sees = key <= pos
                if window > 0:
                    sees &= key > pos - window
                w, o, mag = ref.attend(qn[b, t, rows], kk, vv, scale,
                                       np.broadcast_to(sees, (group, n)))
                tol = ref.out_tolerance(pools.kind, qn[b, t, rows], kk, mag, scale, n, flat)
                ref.assert_within(out[b, t, rows], o, tol, f"{what} out b{b} t{t} g{g}")
                add += w.sum(0)
                seen |= sees
                es = max(es, ref.score_error(qn[b, t, rows], kk, scale))
            # a weight: its score's error and its sum's, 2^-21 of the exponentials, the sums'
            # roundings; then the additions to the mass
            rel = 2 * es + 2 * 2.0 ** -21 + (n + T * group + 8) * 2.0 ** -23
            want = mass0[b, g, :n] + add
            tol = rel * add + 2.0 ** -23 * (np.abs(mass0[b, g, :n]) + add) + 1e-12
            bad = np.abs(mass[b, g, :n] - want) > tol
            assert not bad.any(), f"{what} mass b{b} g{g}: {bad.sum()} off"
            # keys no token sees, and everything behind the sequence, as they were
            assert np.array_equal(mass[b, g, :n][~seen], mass0[b, g, :n][~seen])
            assert np.array_equal(mass[b, g, n:], mass0[b, g, n:])


@pytest.mark.parametrize("kind,d,ps,hkv,group,T,window", [
    ("bf16", 128, 16, 8, 4, 1, 0), ("bf16", 128, 16, 2, 5, 1, 0), ("bf16", 64, 8, 3, 1, 1, 40),
    ("bf16", 128, 16, 2, 4, 4, 0), ("bf16", 64, 24, 2, 2, 8, 33), ("bf16", 128, 16, 1, 16, 1, 0),
    ("f32", 128, 16, 2, 4, 1, 0), ("f32", 64, 5, 3, 3, 1, 20), ("e4m3", 128, 16, 8, 4, 1, 0),
    ("e4m3", 128, 16, 2, 8, 1, 50), ("e4m3", 128, 8, 2, 3, 5, 0), ("e4m3", 128, 16, 2, 1, 7, 9),
    ("int8", 128, 16, 4, 4, 1, 0), ("int8", 128, 32, 2, 4, 2, 0), ("int8", 128, 16, 1, 5, 3, 64),
])
def test_mass_and_output(kind, d, ps, hkv, group, T, window):
    lens = [0, 1, 2, ps, ps + 1, 333, 900, 17 * ps - 1]
    table, P = ref.tables(lens, ps, seed=1)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=2)
    pools.poison(ref.used_slots(table, lens, P, ps))
    g = torch.Generator().manual_seed(3)
    q = torch.randn((len(lens), T, hkv * group, d), generator=g)
    q = q if kind == "f32" else q.bfloat16()
    mass_len = table.shape[1] * ps + 3  # odd row lengths: unaligned rows
    mass0 = torch.rand((len(lens), hkv, mass_len), generator=g)
    mass = mass0.cuda()
    scale = ref.default_scale(d)
    out = run_mass(pools, q, table, lens, mass, scale, window)
    check_mass(out, mass, mass0, pools, q, table, lens, scale, window, kind)


def test_mass_shorter_than_the_table_and_refusal_past_it():
    lens = [100, 101, 60]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    q = torch.randn((3, 1, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass0 = torch.rand((3, 2, 100), generator=torch.Generator().manual_seed(4))
    mass = mass0.cuda()
    err = word()
    out = run_mass(pools, q, table, lens, mass, 0.09, err=err)
    assert int(err.item()) == tl.TL_DEVERR_CONTEXT_RANGE
    check_mass(out, mass, mass0, pools, q, table, [100, 0, 60], 0.09, 0, "refused")


def test_mass_of_a_long_sequence_and_of_many():
    for lens, hkv, group in (([20000], 1, 8), ([(53 * b) % 500 for b in range(140)], 2, 2)):
        table, P = ref.tables(lens, 16, seed=1)
        pools = ref.Pools("bf16", P, 16, hkv, 128, seed=2)
        q = torch.randn((len(lens), 1, hkv * group, 128),
                        generator=torch.Generator().manual_seed(3)).bfloat16()
        mass0 = torch.zeros((len(lens), hkv, table.shape[1] * 16))
        mass = mass0.cuda()
        out = run_mass(pools, q, table, lens, mass, 0.09)
        check_mass(out, mass, mass0, pools, q, table, lens, 0.09, 0, f"b{len(lens)}")
        again = mass0.cuda()
        assert torch.equal(out, run_mass(pools, q, table, lens, again, 0.09))
        assert torch.equal(mass, again)  # the same bits
        # every row's weights sum to 1
        total = mass.double().sum(2).cpu()
        want = torch.tensor([[float(group if n > 0 else 0)] * hkv for n in lens])
        assert torch.allclose(total, want.double(), rtol=0, atol=group * 1e-4)


def test_mass_matches_the_multi_token_decode():
    lens = [700, 64, 9]
    table, P = ref.tables(lens, 16, seed=1)
    for kind in ("bf16", "e4m3"):
        pools = ref.Pools(kind, P, 16, 2, 128, seed=2)
        p = pools.gpu()
        q = torch.randn((3, 3, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
        mass = torch.zeros((3, 2, 720), device="cuda")
        out = run_mass(pools, q, table, lens, mass, 0.09, p=p)
        same = tl.tl_paged_attn_decode_multi(q.cuda(), p["k"], p["v"], table.cuda(), i32(lens), 0.09)
        assert torch.allclose(out, same, rtol=0, atol=1e-4)


def test_a_bad_page_gathers_nothing():
    lens = [64]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 1, 128, seed=2)
    bad = table.clone()
    bad[0, 1] = P + 5
    q = torch.randn((1, 1, 4, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass = torch.zeros((1, 1, 64), device="cuda")
    err = word()
    run_mass(pools, q, bad, lens, mass, 0.09, err=err)
    assert int(err.item()) == tl.TL_DEVERR_PAGE_RANGE
    m = mass.cpu()[0, 0]
    assert torch.all(m[16:32] == 0) and abs(float(m.sum()) - 4) < 1e-3


# --------------------------------------------------------------- selection --

def check_evict(mass, lens, n, first, last, err_bits=0):
    err = word()
    keep, new = tl.tl_kv_evict_select(mass.cuda(), i32(lens), n, keep_first=first, keep_last=last,
                                      error_word=err)
    assert int(err.item()) == err_bits
    B, hkv, N = mass.shape
    want = np.full((B, hkv, n), -1, np.int32)
    ln = []
    for b, L in enumerate(lens):
        L = L if 0 < L <= N else 0
        ln.append(min(L, n))
        for g in range(hkv):
            got = ref.largest(mass[b, g, :L].numpy(), n, first, last)
            want[b, g, :len(got)] = got
    assert new.cpu().tolist() == ln
    assert torch.equal(keep.cpu(), torch.from_numpy(want))
    return keep, new


def weights(shape, seed, zeros=0.05):
    g = torch.Generator().manual_seed(seed)
    m = torch.exp(3 * torch.randn(shape, generator=g)) * 1e-3
    return torch.where(torch.rand(shape, generator=g) < zeros, torch.zeros(()), m)


@pytest.mark.parametrize("n,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 0, 0), (64, 4, 16),
                                          (64, 40, 24), (200, 4, 100), (1000, 0, 3)])
def test_evict_select_is_exact(n, first, last):
    lens = [0, 1, 63, 64, 65, 300, 999, 1000, -2]
    check_evict(weights((9, 3, 1000), 5), lens, n, first, last)


@pytest.mark.parametrize("N", [3000, 4097, 8200, 33000, 140000, 300000])
@pytest.mark.parametrize("what", ["spread", "equal", "few", "zeros"])
def test_evict_select_long_rows(N, what):
    """One CTA to clusters of eight, and rows past their registers; rows of few distinct values."""
    g = torch.Generator().manual_seed(N)
    m = {"spread": lambda: weights((1, 1, N), N), "equal": lambda: torch.full((1, 1, N), 0.25),
         "few": lambda: torch.randint(0, 3, (1, 1, N), generator=g).float(),
         "zeros": lambda: weights((1, 1, N), N, zeros=0.9)}[what]()
    for n in (5, N // 2, N - 1):
        check_evict(m, [N], n, 2, 3)
        check_evict(m, [N - 7], n, 0, 0)


def test_evict_select_orders_every_float():
    x = torch.tensor([0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, float("inf"), float("-inf"),
                      float("nan"), 1.0, -1.0, float("nan"), 0.0, -0.0])
    for n in range(1, 14):
        check_evict(x.view(1, 1, -1), [14], n, 0, 0)
    check_evict(torch.full((1, 2, 40), float("nan")), [40], 7, 1, 2)


def test_evict_select_reports_a_length_past_the_mass():
    check_evict(weights((2, 2, 50), 1), [51, 50], 8, 0, 0, tl.TL_DEVERR_CONTEXT_RANGE)


# -------------------------------------------------------------- compaction --

def compact_ref(pools, table, lens, keep, new, mass):
    """The pools and mass after the call (new tensors)."""
    data = {n: x.clone() for n, x in pools.data.items()}
    scales = {n: x.clone() for n, x in pools.scales.items()}
    m = None if mass is None else mass.clone()
    ps = pools.ps
    for b, n in enumerate(new):
        for g in range(pools.hkv):
            for j in range(n):
                s = int(keep[b, g, j])
                if s < j or s >= lens[b]:
                    continue
                pd, pf = int(table[b, j // ps]), int(table[b, s // ps])
                for name in data:
                    data[name][pd, j % ps, g] = pools.data[name][pf, s % ps, g]
                    if scales:
                        scales[name][pd, g, j % ps] = pools.scales[name][pf, g, s % ps]
                if m is not None:
                    m[b, g, j] = mass[b, g, s]
            if m is not None:
                m[b, g, n:max(lens[b], n)] = 0
    return data, scales, m


def run_compact(pools, table, lens, keep, new, mass, err=None):
    p = pools.gpu()
    w = word() if err is None else err
    args = (table.cuda(), i32(lens), keep.cuda(), i32(new))
    m = None if mass is None else mass.cuda()
    if pools.kind == "int8":
        tl.tl_kv_cache_compact_int8(p["k"], p["v"], p["ks"], p["vs"], *args, mass=m, error_word=w)
    else:
        tl.tl_kv_cache_compact(p["k"], p["v"], *args, mass=m, error_word=w)
    if err is None:
        assert int(w.item()) == 0
    return p, m


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check_compact(pools, table, lens, keep, new, mass, err=None):
    p, m = run_compact(pools, table, lens, keep, new, mass, err)
    data, scales, want = compact_ref(pools, table, lens, keep, new, mass)
    for n in data:
        assert same(p[n], data[n]), n
        if scales:
            assert same(p[n + "s"], scales[n]), n + " scales"
    if mass is not None:
        assert torch.equal(m.cpu(), want)


def random_keep(lens, hkv, n, seed):
    rng = np.random.default_rng(seed)
    keep = np.full((len(lens), hkv, n), -1, np.int32)
    new = [min(max(L, 0), n) for L in lens]
    for b, L in enumerate(lens):
        for g in range(hkv):
            keep[b, g, :new[b]] = np.sort(rng.permutation(max(L, 0))[:new[b]])
    return torch.from_numpy(keep), new


@pytest.mark.parametrize("kind,d,ps,hkv,with_mass", [
    ("bf16", 128, 16, 8, True), ("bf16", 64, 8, 2, False), ("bf16", 96, 16, 3, True),
    ("bf16", 8, 5, 1, True), ("f32", 128, 16, 2, True), ("f32", 64, 3, 5, False),
    ("e4m3", 128, 16, 4, True), ("e4m3", 16, 32, 2, False), ("int8", 128, 16, 4, True),
    ("int8", 48, 24, 3, True), ("int8", 16, 16, 2, False), ("f32", 1024, 4, 40, False),
])
@pytest.mark.parametrize("n", [1, 70, 400])
def test_compact_moves_the_rows(kind, d, ps, hkv, with_mass, n):
    lens = [0, 1, 69, 70, 71, 500, 399, 1300]
    table, P = ref.tables(lens, ps, seed=1)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=2)
    keep, new = random_keep(lens, hkv, n, seed=n)
    mass = torch.rand((8, hkv, 1305), generator=torch.Generator().manual_seed(3)) if with_mass else None
    check_compact(pools, table, lens, keep, new, mass)


def test_compact_of_one_long_sequence_is_split():
    """Few rows: several CTAs share each row; lists that keep almost everything, whose sources
    and places overlap in every batch."""
    lens = [6000]
    table, P = ref.tables(lens, 16, seed=1)
    for n in (5990, 2000):
        for kind in ("bf16", "int8"):
            pools = ref.Pools(kind, P, 16, 1, 128, seed=2)
            keep, new = random_keep(lens, 1, n, seed=n)
            check_compact(pools, table, lens, keep, new, torch.rand((1, 1, 6000)))


def test_compact_follows_any_list_that_looks_ahead():
    """keep[j] >= j is all that is asked: repeated and unordered entries gather the rows as they
    were before the call; entries below j or past the length are skipped and reported."""
    lens = [800, 800, 800]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    rng = np.random.default_rng(3)
    n = 600
    j = np.arange(n)
    keep = np.stack([np.stack([rng.integers(j, 800) for _ in range(2)]) for _ in range(3)])
    keep[1] = 799  # one row everywhere
    keep[2, 0, 100], keep[2, 0, 101], keep[2, 1, 5], keep[2, 1, 6] = 99, -1, 800, 1 << 30
    keep = torch.from_numpy(keep.astype(np.int32))
    err = word()
    check_compact(pools, table, lens, keep, [n, n, n], torch.rand((3, 2, 800)), err)
    assert int(err.item()) == tl.TL_DEVERR_CONTEXT_RANGE


def test_compact_refuses_lengths_and_pages_on_the_device():
    lens = [100, 16 * 8 + 1, 100, 100, 90]
    table, P = ref.tables([100, 128, 100, 100, 90], 16, seed=1, width=8)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    keep, new = random_keep(lens, 2, 50, seed=3)
    mass = torch.rand((5, 2, 130), generator=torch.Generator().manual_seed(3))
    # too many kept, past the table, negative: left alone
    given = [51, 50, -1, 50, 50]
    err = word()
    p, m = run_compact(pools, table, lens, keep, given, mass, err)
    assert int(err.item()) == tl.TL_DEVERR_CONTEXT_RANGE
    data, _, want = compact_ref(pools, table, lens, keep, [0, 0, 0, 50, 50], mass)
    want[:3] = mass[:3]
    assert same(p["k"], data["k"]) and same(p["v"], data["v"]) and torch.equal(m.cpu(), want)
    # a bad page: its rows stay, and are reported
    bad = table.clone()
    bad[3, 2] = P
    err = word()
    p, _ = run_compact(pools, bad, [0, 0, 0, 100, 0], keep, [0, 0, 0, 50, 0], None, err)
    assert int(err.item()) == tl.TL_DEVERR_PAGE_RANGE
    some = keep.clone()
    row = torch.arange(50)
    for g in range(2):
        dead = ((some[3, g] // 16) == 2) | ((row // 16) == 2)
        some[3, g][dead] = -1  # compact_ref skips them
    data, _, _ = compact_ref(pools, table, [0, 0, 0, 100, 0], some, [0, 0, 0, 50, 0], None)
    assert same(p["k"], data["k"]) and same(p["v"], data["v"])


# ---------------------------------------------------------------- together --

def test_gather_evict_compact_and_go_on():
    """Steps that gather weights, an eviction, and a step over the smaller cache: the kept keys
    answer as the same keys did where they were; a second eviction on the moved masses."""
    hkv, group, d, ps = 2, 4, 128, 16
    lens = [300, 40, 555]
    table, P = ref.tables([n + 8 for n in lens], ps, seed=41)
    pools = ref.Pools("bf16", P, ps, hkv, d, seed=42)
    p = pools.gpu()
    g = torch.Generator().manual_seed(43)
    mass = torch.zeros((3, hkv, table.shape[1] * ps), device="cuda")
    scale = ref.default_scale(d)
    lens_now = list(lens)
    for round_ in range(2):
        for _ in range(2):
            q = torch.randn((3, 1, hkv * group, d), generator=g).bfloat16()
            before = mass.cpu()
            out = run_mass(pools, q, table, lens_now, mass, scale, p=p)
            check_mass(out, mass, before, pools, q, table, lens_now, scale, 0, f"round {round_}")
        keep, new = check_evict(mass.cpu(), lens_now, 96, 4, 16)
        data, _, want = compact_ref(pools, table, lens_now, keep.cpu(), new.cpu().tolist(),
                                    mass.cpu())
        tl.tl_kv_cache_compact(p["k"], p["v"], table.cuda(), i32(lens_now), keep, new, mass=mass)
        pools.data = data
        assert same(p["k"], data["k"]) and same(p["v"], data["v"])
        assert torch.equal(mass.cpu(), want)
        lens_now = new.cpu().tolist()
        # the next token goes behind the kept ones
        rows = torch.randn((2, 3, hkv, d), generator=g).bfloat16()
        slots = [int(table[b, L // ps]) * ps + L % ps for b, L in enumerate(lens_now)]
        tl.tl_kv_cache_write(rows[0].cuda(), rows[1].cuda(), p["k"], p["v"],
                             torch.tensor(slots, device="cuda"))
        pools.data = {n: p[n].cpu() for n in ("k", "v")}
        lens_now = [n + 1 for n in lens_now]


def test_an_eviction_captured_in_a_graph():
    lens = [200, 90]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    p = pools.gpu()
    mass = torch.zeros((2, 2, 208), device="cuda")
    q = torch.randn((2, 1, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out = torch.empty((2, 1, 8, 128), device="cuda")
    ws = tl.alloc_workspace(
        tl.tl_paged_attn_decode_mass_workspace_size(2, 1, 8, 2, 128, 208), "cuda")
    keep = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    tb, ln = table.cuda(), i32(lens)

    def step():
        tl.tl_paged_attn_decode_mass(q, p["k"], p["v"], tb, ln, mass, 0.09, out=out, workspace=ws)
        tl.tl_kv_evict_select(mass, ln, 64, keep_first=1, keep_last=8, keep=keep, new_lens=new)
        tl.tl_kv_cache_compact(p["k"], p["v"], tb, ln, keep, new, mass=mass)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # capture ran nothing
    assert not mass.any()
    graph.replay()
    torch.cuda.synchronize()
    first_out = out.clone()
    ref_mass = torch.zeros((2, 2, 208), device="cuda")
    want = run_mass(pools, q, table, lens, ref_mass, 0.09)
    assert torch.equal(first_out, want)
    k2, n2 = check_evict(ref_mass.cpu(), lens, 64, 1, 8)
    assert torch.equal(keep, k2) and torch.equal(new, n2)
    data, _, wm = compact_ref(pools, table, lens, k2.cpu(), n2.cpu().tolist(), ref_mass.cpu())
    assert same(p["k"], data["k"]) and torch.equal(mass.cpu(), wm)


# ------------------------------------------------------------------- edges --

def test_mass_and_compaction_past_32_bit_offsets():
    """Pools of more than 2^32 elements, only their last pages filled; a mass of as many places
    a row as the longest of contexts."""
    P, ps, hkv, d = 270000, 16, 8, 128
    lens = [500, 90]
    small, n = ref.tables(lens, ps, seed=1, spare=0)
    table = torch.where(small >= 0, P - 1 - small, -1).int()
    pools = ref.Pools("bf16", n, ps, hkv, d, seed=2)
    k = torch.empty((P, ps, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    far = (P - 1 - torch.arange(n)).cuda()
    k[far], v[far] = pools.data["k"].cuda(), pools.data["v"].cuda()
    q = torch.randn((2, 1, 32, d), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass0 = torch.rand((2, hkv, 500), generator=torch.Generator().manual_seed(4))
    mass = mass0.cuda()
    err = word()
    out = tl.tl_paged_attn_decode_mass(q.cuda(), k, v, table.cuda(), i32(lens), mass, 0.09,
                                       error_word=err)
    check_mass(out, mass, mass0, pools, q, small, lens, 0.09, 0, "far")
    keep, new = check_evict(mass.cpu(), lens, 200, 2, 20)
    data, _, want = compact_ref(pools, small, lens, keep.cpu(), new.cpu().tolist(), mass.cpu())
    tl.tl_kv_cache_compact(k, v, table.cuda(), i32(lens), keep, new, mass=mass, error_word=err)
    assert int(err.item()) == 0
    assert same(k[far], data["k"]) and same(v[far], data["v"]) and torch.equal(mass.cpu(), want)


def test_mass_of_several_calls_adds_up_and_two_streams():
    lens = [800, 30]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    p = pools.gpu()
    tb, ln = table.cuda(), i32(lens)
    g = torch.Generator().manual_seed(3)
    qs = [torch.randn((2, 1, 8, 128), generator=g).bfloat16().cuda() for _ in range(2)]
    masses = [torch.zeros((2, 2, 800), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                tl.tl_paged_attn_decode_mass(qs[i], p["k"], p["v"], tb, ln, masses[i], 0.09,
                                             stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        once = torch.zeros((2, 2, 800), device="cuda")
        tl.tl_paged_attn_decode_mass(qs[i], p["k"], p["v"], tb, ln, once, 0.09)
        want = once.clone()
        for _ in range(9):
            want += once  # the same additions in the same order
        assert torch.equal(masses[i], want)


def test_a_verify_step_longer_than_the_sequence():
    """Tokens before the sequence's first position see nothing: output 0, no weight."""
    lens = [1, 2, 3, 40]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=2)
    q = torch.randn((4, 4, 4, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass0 = torch.zeros((4, 2, 40))
    mass = mass0.cuda()
    out = run_mass(pools, q, table, lens, mass, 0.09)
    check_mass(out, mass, mass0, pools, q, table, lens, 0.09, 0, "short")
    assert torch.all(out[0, :3] == 0) and torch.all(out[1, :2] == 0)


def test_compact_twice_over_the_same_list():
    """A second call gathers from the moved rows: every call reads the pools as they are."""
    lens = [300, 300]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("int8", P, 16, 2, 128, seed=2)
    keep, new = random_keep(lens, 2, 120, seed=3)
    p = pools.gpu()
    args = (table.cuda(), i32(lens), keep.cuda(), i32(new))
    for _ in range(2):
        tl.tl_kv_cache_compact_int8(p["k"], p["v"], p["ks"], p["vs"], *args)
        data, scales, _ = compact_ref(pools, table, lens, keep, new, None)
        pools.data, pools.scales = data, scales
    assert all(same(p[n], data[n]) and same(p[n + "s"], scales[n]) for n in data)


def test_keeping_as_much_as_there_is_moves_nothing():
    lens = [64, 100]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("bf16", P, 16, 1, 64, seed=2)
    mass = weights((2, 1, 100), 3)
    keep, new = check_evict(mass, lens, 128, 0, 0)
    assert new.cpu().tolist() == lens
    p, m = run_compact(pools, table, lens, keep.cpu(), new.cpu().tolist(), mass)
    assert same(p["k"], pools.data["k"]) and torch.equal(m.cpu(), mass)


def test_threads_calling_with_different_sizes_at_once():
    """Each host thread's calls ask for another amount of shared memory (rows of 100 and 30,000
    values; 1 and 4 query heads a KV head), on a stream of its own."""
    import threading

    def make(n, hkv, group, seed):
        lens = [n, n // 2]
        table, P = ref.tables(lens, 16, seed=seed)
        p = ref.Pools("bf16", P, 16, hkv, 64, seed=seed).gpu()
        q = torch.randn((2, 1, hkv * group, 64), generator=torch.Generator().manual_seed(seed))
        return dict(p=p, q=q.bfloat16().cuda(), table=table.cuda(), lens=i32(lens),
                    mass=weights((2, hkv, n), seed).cuda(), n=n)

    def calls(c, stream):
        bounds = torch.empty((c["p"]["k"].shape[0], c["p"]["k"].shape[2], 2, 64),
                             dtype=torch.int8, device="cuda")
        scales = torch.empty(bounds.shape[:2], device="cuda")
        mass = c["mass"].clone()
        tl.tl_kv_page_bounds(c["p"]["k"], c["table"], c["lens"], bounds, scales, stream=stream)
        pages, lens = tl.tl_kv_page_select(c["q"][:, 0], bounds, scales, c["table"], c["lens"],
                                           16, 4, stream=stream)
        out = tl.tl_paged_attn_decode_mass(c["q"], c["p"]["k"], c["p"]["v"], c["table"],
                                           c["lens"], mass, 0.1, stream=stream)
        keep, new = tl.tl_kv_evict_select(mass, c["lens"], c["n"] // 3, stream=stream)
        return [pages, lens, out, mass, keep, new]

    cases = [make(100, 8, 1, 1), make(30000, 1, 4, 2)]
    want = [calls(c, None) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(40):
                    got = calls(cases[i], stream)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(f"case {i} differs")
        except Exception as e:  # reported by the main thread
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1, 0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("kind", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("B", [1, 16, 17, 130])
def test_a_batch_with_nothing_to_read(kind, B):
    """Every place of the batch is padding (length 0): zeros, empty lists, and all else as it was."""
    pools = ref.Pools(kind, 4, 16, 2, 128, seed=2)
    p = pools.gpu()
    q = torch.randn((B, 4, 128), generator=torch.Generator().manual_seed(3))
    q = (q if kind == "f32" else q.bfloat16()).cuda()
    table, lens = torch.full((B, 3), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
    mass = torch.rand((B, 2, 48), generator=torch.Generator().manual_seed(4)).cuda()
    before, w, int8 = mass.clone(), word(), kind == "int8"
    scales = (p["ks"], p["vs"]) if int8 else ()
    bounds = torch.full((4, 2, 2, 128), 5, dtype=torch.int8, device="cuda")
    bscales = torch.full((4, 2), 0.5, device="cuda")
    if int8:
        tl.tl_kv_page_bounds_int8(p["k"], p["ks"], table, lens, bounds, bscales, error_word=w)
    else:
        tl.tl_kv_page_bounds(p["k"], table, lens, bounds, bscales, error_word=w)
    assert torch.all(bounds == 5) and torch.all(bscales == 0.5)
    pages, page_lens = tl.tl_kv_page_select(q, bounds, bscales, table, lens, 16, 2, error_word=w)
    assert torch.all(pages == -1) and torch.all(page_lens == 0)
    attend = tl.tl_paged_attn_decode_pages_int8 if int8 else tl.tl_paged_attn_decode_pages
    out = torch.full((B, 4, 128), 7.0, device="cuda")
    attend(q, p["k"], p["v"], *scales, pages, page_lens, 0.1, out=out, error_word=w)
    assert torch.all(out == 0)
    gather = tl.tl_paged_attn_decode_mass_int8 if int8 else tl.tl_paged_attn_decode_mass
    out = torch.full((B, 1, 4, 128), 7.0, device="cuda")
    gather(q[:, None], p["k"], p["v"], *scales, table, lens, mass, 0.1, out=out, error_word=w)
    assert torch.all(out == 0) and torch.equal(mass, before)
    keep, new = tl.tl_kv_evict_select(mass, lens, 8, error_word=w)
    assert torch.all(keep == -1) and torch.all(new == 0)
    compact = tl.tl_kv_cache_compact_int8 if int8 else tl.tl_kv_cache_compact
    compact(p["k"], p["v"], *scales, table, lens, keep, new, mass=mass, error_word=w)
    assert torch.equal(mass, before) and int(w.item()) == 0
    assert all(same(p[n], pools.data[n]) for n in pools.data)


@pytest.mark.parametrize("group,T", [(4, 1), (4, 4), (16, 1)])
def test_v_scales_of_any_size(group, T):
    """Weights times V scales go through 16-bit parts: a power of two in every scale of a pool
    multiplies the outputs and changes no bit, and scales 10^6 apart in one sequence, rising or
    falling along it, keep the outputs within their tolerance."""
    lens = [700, 40, 1500]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("int8", P, 16, 2, 128, seed=2)
    q = torch.randn((3, T, 2 * group, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass0 = torch.zeros((3, 2, 1500))
    base = pools.scales["v"]
    outs = []
    for f in (1.0, 2.0 ** -60, 2.0 ** 40):
        pools.scales["v"] = base * f
        mass = mass0.cuda()
        outs.append(run_mass(pools, q, table, lens, mass, 0.09) / f)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    position = torch.zeros((P, 16))
    for b, n in enumerate(lens):
        blocks = -(-n // 16)
        place = torch.arange(blocks * 16).view(blocks, 16) / max(lens)
        position[table[b, :blocks].long()] = place
    for sign in (1.0, -1.0):
        pools.scales["v"] = base * torch.exp2(sign * 20 * (position - 0.5))[:, None, :]
        mass = mass0.cuda()
        out = run_mass(pools, q, table, lens, mass, 0.09)
        check_mass(out, mass, mass0, pools, q, table, lens, 0.09, 0, f"scales {sign}")


@pytest.mark.parametrize("kind,B,T", [("bf16", 3, 4), ("e4m3", 40, 3), ("bf16", 700, 4),
                                      ("bf16", 700, 1)])
def test_mass_of_pieces_in_parts(kind, B, T):
    """Fewer pieces than the warps that add the weights up: each piece goes in parts.  One long
    sequence (its pieces' sizes differ from the others'), short ones and empty ones."""
    lens = [(53 * b) % 90 for b in range(B)]
    lens[1] = 9000
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools(kind, P, 16, 1, 128, seed=2)
    q = torch.randn((B, T, 4, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    mass0 = torch.rand((B, 1, 9000), generator=torch.Generator().manual_seed(4))
    mass = mass0.cuda()
    out = run_mass(pools, q, table, lens, mass, 0.09)
    check_mass(out, mass, mass0, pools, q, table, lens, 0.09, 0, f"{kind} b{B}")
