"""Page bounds, page selection and the attention over the selected pages,
against the plain implementations of tests/long_context_ref.py: codes, scales
and selections equal bit for bit, attention within derived tolerances."""
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


def run_bounds(kind, pools, table, lens, first, b0, s0, err=None):
    bnd, sc = b0.cuda(), s0.cuda()
    w = word() if err is None else err
    f = None if first is None else i32(first)
    p = pools.gpu()
    if kind == "int8":
        tl.tl_kv_page_bounds_int8(p["k"], p["ks"], table.cuda(), i32(lens), bnd, sc, first_new=f,
                                  error_word=w)
    else:
        tl.tl_kv_page_bounds(p["k"], table.cuda(), i32(lens), bnd, sc, first_new=f, error_word=w)
    if err is None:
        assert int(w.item()) == 0
    return bnd.cpu(), sc.cpu()


def start_bounds(P, hkv, d, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-127, 128, (P, hkv, 2, d), generator=g, dtype=torch.int8),
            torch.rand((P, hkv), generator=g))


# ------------------------------------------------------------------ bounds --

@pytest.mark.parametrize("kind,d,ps,hkv,lens,first", [
    ("bf16", 128, 16, 8, [0, 1, 15, 16, 17, 100], None),
    ("bf16", 128, 16, 3, [33, 48, 49, 5], [32, 47, 0, 5]),
    ("bf16", 64, 8, 1, [7, 8, 9, 1000], [3, 0, 8, 500]),
    ("bf16", 64, 1, 2, [1, 5], None),
    ("bf16", 128, 256, 2, [255, 256, 300], [250, 0, 257]),
    ("f32", 128, 16, 2, [1, 31, 64], None),
    ("f32", 64, 24, 5, [23, 24, 25, 70], [0, 24, 24, 50]),
    ("e4m3", 128, 16, 8, [3, 16, 90], [2, 0, 80]),
    ("e4m3", 64, 32, 2, [3, 33], None),
    ("int8", 128, 16, 4, [1, 20, 47], None),
    ("int8", 64, 48, 2, [1, 50, 97], [0, -3, 96]),
])
def test_bounds_are_exact(kind, d, ps, hkv, lens, first):
    table, P = ref.tables(lens, ps, seed=3)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=5, only_k=True)
    pools.poison(ref.used_slots(table, lens, P, ps))
    b0, s0 = start_bounds(P, hkv, d)
    got_b, got_s = run_bounds(kind, pools, table, lens, first, b0, s0)
    want_b, want_s = ref.bounds(pools.values("k"), table, lens, first, ps, b0, s0)
    assert torch.equal(got_s, want_s)
    assert torch.equal(got_b, want_b)


def test_bounds_of_more_sequences_than_a_round():
    lens = [(7 * b) % 40 for b in range(2500)]
    first = [(3 * b) % 30 for b in range(2500)]
    table, P = ref.tables(lens, 8, seed=2)
    pools = ref.Pools("bf16", P, 8, 1, 64, seed=6, only_k=True)
    b0, s0 = start_bounds(P, 1, 64)
    got_b, got_s = run_bounds("bf16", pools, table, lens, first, b0, s0)
    want_b, want_s = ref.bounds(pools.values("k"), table, lens, first, 8, b0, s0)
    assert torch.equal(got_s, want_s) and torch.equal(got_b, want_b)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_non_finite_key_counts_as_zero_and_is_reported(kind):
    lens = [20, 40]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools(kind, P, 16, 2, 128, only_k=True)
    k = pools.data["k"]
    k[table[0, 0], 3, 1, 7] = float("nan")
    k[table[1, 1], 0, 0, 0] = float("inf")
    k[table[1, 2], :, 0, :] = float("-inf")
    b0, s0 = start_bounds(P, 2, 128)
    err = word()
    got_b, got_s = run_bounds(kind, pools, table, lens, None, b0, s0, err)
    want_b, want_s = ref.bounds(pools.values("k"), table, lens, None, 16, b0, s0)
    assert torch.equal(got_s, want_s) and torch.equal(got_b, want_b)
    assert int(err.item()) == tl.TL_DEVERR_VALUE_RANGE


def test_zero_keys_give_zero_codes_and_scale():
    table, P = ref.tables([16], 16)
    pools = ref.Pools("bf16", P, 16, 1, 128, only_k=True)
    pools.data["k"].zero_()
    got_b, got_s = run_bounds("bf16", pools, table, [16], None, *start_bounds(P, 1, 128))
    page = int(table[0, 0])
    assert not got_b[page].any() and float(got_s[page, 0]) == 0.0


def test_bounds_report_bad_pages_and_lengths_and_leave_them():
    lens = [40, 33, 16 * 3 + 1]
    table, P = ref.tables([40, 33, 48], 16, width=3)
    good = table.clone()
    table[0, 1], table[1, 2] = P, -1
    pools = ref.Pools("bf16", P, 16, 2, 128, only_k=True)
    b0, s0 = start_bounds(P, 2, 128)
    err = word()
    got_b, got_s = run_bounds("bf16", pools, table, lens, None, b0, s0, err)
    assert int(err.item()) == tl.TL_DEVERR_PAGE_RANGE | tl.TL_DEVERR_CONTEXT_RANGE
    want_b, want_s = ref.bounds(pools.values("k"), good, [40, 33, 0], None, 16, b0, s0)
    for page in (int(good[0, 1]), int(good[1, 2])):
        want_b[page], want_s[page] = b0[page], s0[page]
    assert torch.equal(got_b, want_b) and torch.equal(got_s, want_s)


# --------------------------------------------------------------- selection --

def random_bounds(P, hkv, d, seed, levels=None):
    g = torch.Generator().manual_seed(seed)
    hi = torch.randint(0, 128, (P, hkv, d), generator=g)
    lo = -torch.randint(0, 128, (P, hkv, d), generator=g)
    sc = (1 + torch.rand((P, hkv), generator=g)).bfloat16().float() / 127
    if levels:  # few distinct pages: many equal scores
        pick = torch.randint(0, levels, (P,), generator=g)
        hi, lo, sc = hi[pick], lo[pick], sc[pick]
    return torch.stack((hi, lo), 2).to(torch.int8), sc


def check_select(q, bnd, sc, table, lens, ps, n, first, last, err_bits=0):
    P = bnd.shape[0]
    err = word()
    got_t, got_l = tl.tl_kv_page_select(q.cuda(), bnd.cuda(), sc.cuda(), table.cuda(), i32(lens),
                                        ps, n, keep_first=first, keep_last=last, error_word=err)
    assert int(err.item()) == err_bits
    want_t, want_l = ref.page_select(q, bnd, sc, table, lens, ps, n, first, last, P)
    assert torch.equal(got_l.cpu(), want_l)
    assert torch.equal(got_t.cpu(), want_t)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group", [(8, 4), (1, 1), (2, 8), (3, 5), (12, 2), (16, 16), (5, 3)])
def test_selection_is_exact(hkv, group, d):
    lens = [0, 1, 16, 17, 300, 1999, 2000, 640]
    table, P = ref.tables(lens, 16, seed=7)
    bnd, sc = random_bounds(P, hkv, d, seed=8)
    q = torch.randn((len(lens), hkv * group, d), generator=torch.Generator().manual_seed(9))
    check_select(q.bfloat16(), bnd, sc, table, lens, 16, 9, 1, 2)
    check_select(q, bnd, sc, table, lens, 16, 40, 0, 1)


@pytest.mark.parametrize("n,first,last", [(1, 0, 1), (2, 1, 1), (3, 1, 2), (5, 4, 1), (124, 0, 1),
                                          (125, 3, 3), (126, 0, 1), (500, 7, 9)])
def test_selection_at_the_edges_of_n(n, first, last):
    lens = [125 * 8, 125 * 8 - 3, 9, 3 * 8]
    table, P = ref.tables(lens, 8, seed=1)
    bnd, sc = random_bounds(P, 2, 64, seed=2)
    q = torch.randn((4, 4, 64), generator=torch.Generator().manual_seed(3)).bfloat16()
    check_select(q, bnd, sc, table, lens, 8, n, first, last)


@pytest.mark.parametrize("blocks", [4000, 5000, 9000, 20000, 70000, 140000])
@pytest.mark.parametrize("levels", [3, None])
def test_long_rows_and_equal_scores(blocks, levels):
    """Rows of one CTA, of clusters of 2 to 8 and past their registers; a table that names few
    distinct pages, so most scores are equal and go by the index."""
    P, hkv = 600, 1
    bnd, sc = random_bounds(P, hkv, 64, seed=blocks, levels=levels)
    g = torch.Generator().manual_seed(blocks + 1)
    table = torch.randint(0, P, (2, blocks), generator=g, dtype=torch.int32)
    q = torch.randn((2, 2, 64), generator=g).bfloat16()
    for n in (7, blocks // 3, blocks - 1):
        check_select(q, bnd, sc, table, [blocks * 4, blocks * 4 - 5], 4, n, 2, 3)


def test_a_zero_query_selects_the_lowest_blocks():
    lens = [400]
    table, P = ref.tables(lens, 16, seed=4)
    bnd, sc = random_bounds(P, 2, 128, seed=5)
    check_select(torch.zeros(1, 4, 128, dtype=torch.bfloat16), bnd, sc, table, lens, 16, 6, 0, 1)


def test_selection_reports_what_it_cannot_read():
    lens = [320, 16 * 20 + 1, -4]
    table, P = ref.tables([320, 320, 0], 16, seed=4, width=20)
    table[0, 3], table[0, 9] = P, -7
    bnd, sc = random_bounds(P, 2, 128, seed=5)
    q = torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    q[0, 1, 5] = float("nan")
    q[0, 2, 6] = float("inf")
    check_select(q, bnd, sc, table, lens, 16, 8, 1, 1,
                 tl.TL_DEVERR_PAGE_RANGE | tl.TL_DEVERR_CONTEXT_RANGE | tl.TL_DEVERR_VALUE_RANGE)


# --------------------------------------------------------------- attention --

def head_pages(table, lens, hkv, n, ps, seed):
    """Random ascending pages per head, the last block always among them."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    pages = np.full((B, hkv, n), -1, np.int32)
    ln = np.zeros(B, np.int32)
    for b, L in enumerate(lens):
        nb = -(-L // ps) if L > 0 else 0
        if nb == 0:
            continue
        m = min(n, nb)
        ln[b] = L if nb <= n else (n - 1) * ps + (L - 1) % ps + 1
        for g in range(hkv):
            pick = np.sort(np.append(rng.permutation(nb - 1)[:m - 1], nb - 1))
            pages[b, g, :m] = table[b].numpy()[pick]
    return torch.from_numpy(pages), torch.from_numpy(ln)


def run_pages(pools, q, pages, ln, scale, err=None, **kw):
    p = pools.gpu()
    w = word() if err is None else err
    if pools.kind == "int8":
        out = tl.tl_paged_attn_decode_pages_int8(q.cuda(), p["k"], p["v"], p["ks"], p["vs"],
                                                 pages.cuda(), ln.cuda(), scale, error_word=w, **kw)
    else:
        out = tl.tl_paged_attn_decode_pages(q.cuda(), p["k"], p["v"], pages.cuda(), ln.cuda(),
                                            scale, error_word=w, **kw)
    if err is None:
        assert int(w.item()) == 0
    return out


def check_pages(out, pools, q, pages, ln, scale, what):
    k, v = pools.values("k").double().numpy(), pools.values("v").double().numpy()
    hkv, ps, d = pools.hkv, pools.ps, pools.d
    units = pools.units("v").numpy()
    group = q.shape[1] // hkv
    qn = q.double().numpy()
    for b in range(q.shape[0]):
        n = int(ln[b])
        for g in range(hkv):
            rows = slice(g * group, (g + 1) * group)
            pg = pages[b, g, :-(-n // ps)].long().numpy()
            kk = k[pg][:, :, g].reshape(-1, d)[:n]
            vv = v[pg][:, :, g].reshape(-1, d)[:n]
            if n == 0:
                assert torch.all(out[b, rows] == 0)
                continue
            _, o, mag = ref.attend(qn[b, rows], kk, vv, scale, np.ones((group, n), bool))
            tol = ref.out_tolerance(pools.kind, qn[b, rows], kk, mag, scale, n,
                                    units[pg][:, :, g].reshape(-1, d)[:n].sum(0))
            ref.assert_within(out[b, rows], o, tol, f"{what} b{b} g{g}")


@pytest.mark.parametrize("kind,d,ps,hkv,group", [
    ("bf16", 128, 16, 8, 4), ("bf16", 128, 16, 2, 5), ("bf16", 64, 8, 4, 1), ("bf16", 128, 24, 1, 16),
    ("bf16", 64, 128, 2, 12), ("f32", 128, 16, 2, 4), ("f32", 64, 5, 3, 2), ("e4m3", 128, 16, 8, 4),
    ("e4m3", 128, 8, 2, 8), ("e4m3", 128, 32, 1, 16), ("int8", 128, 16, 4, 4), ("int8", 128, 48, 2, 7),
    ("int8", 128, 16, 1, 16),
])
def test_attention_over_a_table_per_head(kind, d, ps, hkv, group):
    lens = [0, 1, ps, ps + 1, 40 * ps - 1, 7 * ps + 3, 300]
    table, P = ref.tables(lens, ps, seed=11)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=12)
    pools.poison(ref.used_slots(table, lens, P, ps))
    q = torch.randn((len(lens), hkv * group, d), generator=torch.Generator().manual_seed(13))
    q = q if kind == "f32" else q.bfloat16()
    scale = ref.default_scale(d)
    for n in (1, 6, 50):
        pages, ln = head_pages(table, lens, hkv, n, ps, seed=n)
        out = run_pages(pools, q, pages, ln, scale)
        check_pages(out, pools, q, pages, ln, scale, f"{kind} n{n}")


def test_attention_over_pages_of_a_large_batch():
    """More sequences than the one-warp plan takes, ragged."""
    lens = [(37 * b) % 700 for b in range(150)]
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=4)
    q = torch.randn((150, 8, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    pages, ln = head_pages(table, lens, 2, 12, 16, seed=6)
    out = run_pages(pools, q, pages, ln, 0.09)
    check_pages(out, pools, q, pages, ln, 0.09, "b150")


def test_one_long_sequence_in_many_pieces():
    lens = [30000]
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools("bf16", P, 16, 1, 128, seed=4)
    q = torch.randn((1, 8, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    pages, ln = head_pages(table, lens, 1, 1500, 16, seed=6)
    out = run_pages(pools, q, pages, ln, 0.09)
    check_pages(out, pools, q, pages, ln, 0.09, "one")
    assert torch.equal(out, run_pages(pools, q, pages, ln, 0.09))  # the same bits again


def test_pages_errors_are_reported():
    lens = [64, 64, 200]
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=4)
    q = torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    pages, ln = head_pages(table, lens, 2, 4, 16, seed=6)
    pages[0, 1, 2] = P  # one head's bad page: its keys count as masked
    ln[1] = 4 * 16 + 1  # longer than the table: nothing is read
    err = word()
    out = run_pages(pools, q, pages, ln, 0.09, err=err)
    assert int(err.item()) == tl.TL_DEVERR_PAGE_RANGE | tl.TL_DEVERR_CONTEXT_RANGE
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out))
    ln[1] = 0
    good = pages.clone()
    good[0, 1, 2] = 0
    want = run_pages(pools, q, good, ln, 0.09)
    assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[2], want[2])


# ---------------------------------------------------------------- together --

def test_a_step_selects_and_attends(kind="bf16"):
    """Three decode steps as a server runs them: write, bounds of the touched pages, selection,
    attention; with every page selected it is tl_paged_attn_decode."""
    hkv, group, d, ps = 2, 4, 128, 16
    lens = [500, 33, 1200]
    table, P = ref.tables([n + 3 for n in lens], ps, seed=21)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=22)
    p = pools.gpu()
    g = torch.Generator().manual_seed(23)
    bnd = torch.zeros((P, hkv, 2, d), dtype=torch.int8, device="cuda")
    sc = torch.zeros((P, hkv), device="cuda")
    tb = table.cuda()
    tl.tl_kv_page_bounds(p["k"], tb, i32(lens), bnd, sc)
    scale = ref.default_scale(d)
    for step in range(3):
        before = [n + step for n in lens]
        after = [n + 1 for n in before]
        new = torch.randn((2, 3, hkv, d), generator=g).bfloat16()
        slots = [int(table[b, L // ps]) * ps + L % ps for b, L in enumerate(before)]
        tl.tl_kv_cache_write(new[0].cuda(), new[1].cuda(), p["k"], p["v"],
                             torch.tensor(slots, device="cuda"))
        tl.tl_kv_page_bounds(p["k"], tb, i32(after), bnd, sc, first_new=i32(before))
        pools.data["k"], pools.data["v"] = p["k"].cpu(), p["v"].cpu()
        want_b, want_s = ref.bounds(pools.values("k"), table, after, None, ps,
                                    torch.zeros_like(bnd, device="cpu"),
                                    torch.zeros_like(sc, device="cpu"))
        assert torch.equal(bnd.cpu(), want_b) and torch.equal(sc.cpu(), want_s)
        q = torch.randn((3, hkv * group, d), generator=g).bfloat16()
        pages, ln = tl.tl_kv_page_select(q.cuda(), bnd, sc, tb, i32(after), ps, 8, keep_first=1)
        want_t, want_l = ref.page_select(q, want_b, want_s, table, after, ps, 8, 1, 1, P)
        assert torch.equal(pages.cpu(), want_t) and torch.equal(ln.cpu(), want_l)
        out = tl.tl_paged_attn_decode_pages(q.cuda(), p["k"], p["v"], pages, ln, scale)
        check_pages(out, pools, q, want_t, want_l, scale, f"step {step}")
        pages, ln = tl.tl_kv_page_select(q.cuda(), bnd, sc, tb, i32(after), ps, 80)
        assert ln.cpu().tolist() == after
        every = tl.tl_paged_attn_decode_pages(q.cuda(), p["k"], p["v"], pages, ln, scale)
        whole = tl.tl_paged_attn_decode(q.cuda(), p["k"], p["v"], tb, i32(after), scale)
        assert torch.allclose(every, whole, rtol=0, atol=1e-4)


def test_a_step_captured_in_a_graph_and_on_another_stream():
    hkv, group, d, ps = 2, 4, 128, 16
    lens = [500, 33, 1200]
    table, P = ref.tables(lens, ps, seed=31)
    pools = ref.Pools("bf16", P, ps, hkv, d, seed=32)
    p = pools.gpu()
    bnd = torch.zeros((P, hkv, 2, d), dtype=torch.int8, device="cuda")
    sc = torch.zeros((P, hkv), device="cuda")
    tb, ln_in = table.cuda(), i32(lens)
    q = torch.zeros((3, hkv * group, d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((3, hkv * group, d), device="cuda")
    pages = torch.empty((3, hkv, 8), dtype=torch.int32, device="cuda")
    ln = torch.empty(3, dtype=torch.int32, device="cuda")
    ws1 = tl.alloc_workspace(tl.tl_kv_page_select_workspace_size(3, hkv * group, hkv, d, tb.shape[1]), "cuda")
    ws2 = tl.alloc_workspace(tl.tl_paged_attn_decode_workspace_size(3, hkv * group, hkv, d), "cuda")

    def step():
        tl.tl_kv_page_bounds(p["k"], tb, ln_in, bnd, sc)
        tl.tl_kv_page_select(q, bnd, sc, tb, ln_in, ps, 8, page_table=pages, page_lens=ln,
                             workspace=ws1)
        tl.tl_paged_attn_decode_pages(q, p["k"], p["v"], pages, ln, 0.09, out=out, workspace=ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        qn = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).bfloat16()
        q.copy_(qn)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want_b, want_s = ref.bounds(pools.values("k"), table, lens, None, ps,
                                    torch.zeros_like(bnd, device="cpu"),
                                    torch.zeros_like(sc, device="cpu"))
        want_t, want_l = ref.page_select(qn, want_b, want_s, table, lens, ps, 8, 0, 1, P)
        assert torch.equal(pages.cpu(), want_t)
        check_pages(out, pools, qn, want_t, want_l, 0.09, f"replay {seed}")


# ------------------------------------------------------------------- edges --

def test_scores_at_the_largest_codes():
    """Every code and query at +-127: the sums' largest magnitudes, whole numbers all the same."""
    P, hkv = 40, 2
    bnd = torch.full((P, hkv, 2, 128), 127, dtype=torch.int8)
    bnd[:, :, 1] = -127
    bnd[::3, 0, 0, 5], bnd[1::3, 1, 1, 77] = 126, -126
    sc = torch.full((P, hkv), 0.03)
    sc[7::11] = 0.030000001
    q = torch.ones(1, 16, 128)
    q[0, 1::2, ::2] = -1
    table = torch.randperm(P, generator=torch.Generator().manual_seed(1)).int().view(1, P)
    for n in (1, 11, 39):
        check_select(q, bnd, sc, table, [P * 16], 16, n, 0, 1)
        check_select(q.bfloat16(), bnd, sc, table, [P * 16 - 9], 16, n, 0, 1)


def test_query_scales_out_of_the_ordinary():
    """Rows whose scale is subnormal, tiny, huge or zero: the codes are those of the division."""
    P = 50
    bnd, sc = random_bounds(P, 4, 64, seed=3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn((4, 4, 64), generator=g)
    mul = torch.tensor([1e-42, 1e-36, 1e35, 0.0]).view(1, 4, 1)
    table = torch.stack([torch.randperm(P, generator=g).int() for _ in range(4)])
    check_select(q * mul, bnd, sc, table, [P * 16] * 4, 16, 9, 0, 1)


@pytest.mark.parametrize("mul", [1e-44, 1e-37, 3e37])
def test_bounds_of_keys_of_extreme_size(mul):
    lens = [37]
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools("f32", P, 16, 2, 64, seed=2, only_k=True)
    pools.data["k"].mul_(mul / 10)
    b0, s0 = start_bounds(P, 2, 64)
    got_b, got_s = run_bounds("f32", pools, table, lens, None, b0, s0)
    want_b, want_s = ref.bounds(pools.values("k"), table, lens, None, 16, b0, s0)
    assert torch.equal(got_s, want_s) and torch.equal(got_b, want_b)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_halves_round_to_even(kind):
    """Keys whose quotients fall on halves (few bits, small multiples of the largest)."""
    table, P = ref.tables([16 * 40], 16, seed=1)
    pools = ref.Pools("f32", P, 16, 1, 128, seed=2, only_k=True)
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-254, 255, (P, 16, 1, 128), generator=g) * 0.5
    x[:, 0, 0, 0] = 127.0 if kind == "bf16" else 112.0
    pools.kind, pools.data["k"] = kind, x.clamp(-127, 127).to(ref.TYPES[kind])
    b0, s0 = start_bounds(P, 1, 128)
    got_b, got_s = run_bounds(kind, pools, table, [16 * 40], None, b0, s0)
    want_b, want_s = ref.bounds(pools.values("k"), table, [16 * 40], None, 16, b0, s0)
    assert torch.equal(got_s, want_s) and torch.equal(got_b, want_b)


def test_more_sequences_than_a_round_select():
    lens = [(11 * b) % 90 for b in range(1100)]
    table, P = ref.tables(lens, 8, seed=1)
    bnd, sc = random_bounds(P, 1, 64, seed=2)
    q = torch.randn((1100, 2, 64), generator=torch.Generator().manual_seed(3)).bfloat16()
    check_select(q, bnd, sc, table, lens, 8, 4, 1, 1)


def test_calls_on_two_streams_at_once():
    """Two steps at once, each with its own workspaces and outputs."""
    lens = [3000, 900]
    table, P = ref.tables(lens, 16, seed=31)
    pools = ref.Pools("bf16", P, 16, 2, 128, seed=32)
    p = pools.gpu()
    bnd = torch.zeros((P, 2, 2, 128), dtype=torch.int8, device="cuda")
    sc = torch.zeros((P, 2), device="cuda")
    tb, ln_in = table.cuda(), i32(lens)
    tl.tl_kv_page_bounds(p["k"], tb, ln_in, bnd, sc)
    g = torch.Generator().manual_seed(33)
    qs = [torch.randn((2, 8, 128), generator=g).bfloat16() for _ in range(2)]
    dq = [q.cuda() for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                pages, ln = tl.tl_kv_page_select(dq[i], bnd, sc, tb, ln_in, 16, 20, stream=s)
                o = tl.tl_paged_attn_decode_pages(dq[i], p["k"], p["v"], pages, ln, 0.09, stream=s)
                out[i].append((pages, o))
    torch.cuda.synchronize()
    for i in range(2):
        want_t, want_l = ref.page_select(qs[i], bnd.cpu(), sc.cpu(), table, lens, 16, 20, 0, 1, P)
        check_pages(out[i][0][1], pools, qs[i], want_t, want_l, 0.09, f"stream {i}")
        for pages, o in out[i]:
            assert torch.equal(pages.cpu(), want_t) and torch.equal(o, out[i][0][1])


def test_pages_past_32_bit_offsets():
    """Pools of more than 2^32 elements, only their last pages filled."""
    P, ps, hkv, d = 270000, 16, 8, 128  # 4.4e9 elements a pool
    lens = [700, 333]
    need = [-(-n // ps) for n in lens]
    table = torch.full((2, max(need)), -1, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1))
    small = torch.full((2, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        small[b, :n] = order[at:at + n].int()
        table[b, :n] = P - 1 - small[b, :n]
        at += n
    n = sum(need)
    pools = ref.Pools("bf16", n, ps, hkv, d, seed=2)
    k = torch.empty((P, ps, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    bnd = torch.empty((P, hkv, 2, d), dtype=torch.int8, device="cuda")
    sc = torch.empty((P, hkv), device="cuda")
    far = P - 1 - torch.arange(n)
    k[far.cuda()], v[far.cuda()] = pools.data["k"].cuda(), pools.data["v"].cuda()
    tl.tl_kv_page_bounds(k, table.cuda(), i32(lens), bnd, sc)
    want_b, want_s = ref.bounds(pools.values("k"), small, lens, None, ps,
                                torch.zeros((n, hkv, 2, d), dtype=torch.int8), torch.zeros((n, hkv)))
    assert torch.equal(bnd[far.cuda()].cpu(), want_b) and torch.equal(sc[far.cuda()].cpu(), want_s)
    q = torch.randn((2, 32, d), generator=torch.Generator().manual_seed(3)).bfloat16()
    pages, ln = tl.tl_kv_page_select(q.cuda(), bnd, sc, table.cuda(), i32(lens), ps, 10)
    want_t, want_l = ref.page_select(q, want_b, want_s, small, lens, ps, 10, 0, 1, n)
    assert torch.equal(pages.cpu(), torch.where(want_t >= 0, P - 1 - want_t, -1))
    out = tl.tl_paged_attn_decode_pages(q.cuda(), k, v, pages, ln, 0.09)
    check_pages(out, pools, q, want_t, want_l, 0.09, "far")


@pytest.mark.parametrize("kind,B,hkv,group", [
    ("bf16", 31, 2, 4), ("bf16", 32, 4, 2), ("bf16", 33, 2, 1), ("e4m3", 32, 2, 4),
    ("e4m3", 33, 2, 8), ("int8", 64, 2, 4), ("int8", 65, 1, 4), ("e4m3", 64, 1, 16),
    # more heads and sequences than warps: a piece of each sequence is no longer one item a warp
    ("bf16", 30, 64, 1), ("e4m3", 61, 48, 1), ("int8", 2, 300, 1),
])
def test_attention_over_pages_of_any_batch(kind, B, hkv, group):
    """Batches on both sides of the call's own planning, one sequence much longer than the rest,
    some empty."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(1, 120, B)]
    lens[B // 2], lens[0], lens[-1] = 2000, 0, 16
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools(kind, P, 16, hkv, 128, seed=4)
    q = torch.randn((B, hkv * group, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    pages, ln = head_pages(table, lens, hkv, 110, 16, seed=6)
    out = run_pages(pools, q, pages, ln, 0.09)
    check_pages(out, pools, q, pages, ln, 0.09, f"{kind} b{B}")
    assert torch.equal(out, run_pages(pools, q, pages, ln, 0.09))


@pytest.mark.parametrize("kind,group", [("bf16", 4), ("e4m3", 4), ("e4m3", 6), ("int8", 4),
                                        ("int8", 5), ("int8", 12), ("f32", 3)])
def test_a_nan_in_one_head_leaves_the_others(kind, group):
    lens = [500, 33]
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools(kind, P, 16, 2, 128, seed=4)
    pools.poison(ref.used_slots(table, lens, P, 16))
    q = torch.randn((2, 2 * group, 128), generator=torch.Generator().manual_seed(5))
    q = q if kind == "f32" else q.bfloat16()
    pages, ln = head_pages(table, lens, 2, 20, 16, seed=6)
    want = run_pages(pools, q, pages, ln, 0.09)
    bad = q.clone()
    bad[:, 1, 7] = float("nan")
    p, w = pools.gpu(), word()
    attend = tl.tl_paged_attn_decode_pages_int8 if kind == "int8" else tl.tl_paged_attn_decode_pages
    scales = (p["ks"], p["vs"]) if kind == "int8" else ()
    got = attend(bad.cuda(), p["k"], p["v"], *scales, pages.cuda(), i32(ln), 0.09, error_word=w)
    heads = [h for h in range(2 * group) if h != 1]
    assert torch.equal(got[:, heads], want[:, heads])


@pytest.mark.parametrize("kind,group,T", [("int8", 3, 2), ("int8", 1, 7), ("e4m3", 3, 2)])
def test_weights_with_columns_left_over(kind, group, T):
    """Tokens times heads that leave columns of the keys-as-rows form empty, over pools whose
    unread slots hold NaN."""
    lens = [9, 100, 1000]
    table, P = ref.tables(lens, 16, seed=3)
    pools = ref.Pools(kind, P, 16, 2, 128, seed=4)
    clean = ref.Pools(kind, P, 16, 2, 128, seed=4)
    pools.poison(ref.used_slots(table, lens, P, 16))
    q = torch.randn((3, T, 2 * group, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    res = []
    for x in (pools, clean):
        p, w, mass = x.gpu(), word(), torch.zeros((3, 2, 1000), device="cuda")
        gather = tl.tl_paged_attn_decode_mass_int8 if kind == "int8" else tl.tl_paged_attn_decode_mass
        scales = (p["ks"], p["vs"]) if kind == "int8" else ()
        out = gather(q.cuda(), p["k"], p["v"], *scales, table.cuda(), i32(lens), mass, 0.09,
                     error_word=w)
        assert int(w.item()) == 0 and torch.isfinite(out).all() and torch.isfinite(mass).all()
        res.append((out, mass))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
