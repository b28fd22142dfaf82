"""Operators that bound what a long sequence's decode step reads, for measurement.

Two ways over the paged KV cache: reading only the pages a cheap score selects
for the step's query (bounds of every page, selection, attention over the
selected pages), and evicting the keys that gathered the least attention
weight (attention that accumulates it, selection of the keys to keep, in-place
compaction).  Each case names one operator; run() computes it in plain torch
where `own` is false and through the package's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
POOL_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
              "int8": torch.int8}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step of 64 sequences: only each sequence's last page changes
        dict(name="bounds step b64", op="bounds", B=64, lo=17, hi=512, new=1, Hkv=8, d=128, ps=16,
             dtype="bf16"),
        # a batch of eight prompts of up to 8,192 tokens, every page
        dict(name="bounds prompts b8", op="bounds", B=8, lo=6144, hi=8192, new=8192, Hkv=8, d=128,
             ps=16, dtype="bf16"),
        # one user at 128K tokens: 8,192 pages a head, 256 of them read
        dict(name="select b1 128k", op="select", B=1, lo=131072, hi=131072, n_select=256, first=1,
             last=2, Hq=64, Hkv=8, d=128, ps=16, qdtype="bf16"),
        # a ragged batch of long sequences, 128 pages (2,048 keys) each
        dict(name="select b64 1k-32k", op="select", B=64, lo=1024, hi=32768, n_select=128, first=1,
             last=2, Hq=40, Hkv=8, d=128, ps=16, qdtype="bf16"),
        # the attention of the one long sequence: 4,096 of its keys
        dict(name="attend b1 256 pages", op="attend", B=1, lo=131072, hi=131072, n_select=256,
             Hq=64, Hkv=8, d=128, ps=16, dtype="bf16"),
        # the attention of the batch; its shortest sequences have fewer pages than the budget
        dict(name="attend b64 128 pages", op="attend", B=64, lo=1024, hi=16384, n_select=128,
             Hq=40, Hkv=8, d=128, ps=16, dtype="bf16"),
        # one long conversation's decode step that gathers the weights
        dict(name="mass b1 32k", op="mass", B=1, lo=32768, hi=32768, q_len=1, Hq=32, Hkv=8, d=128,
             ps=16, dtype="bf16", window=0),
        # the same for a batch of 64 over e4m3 pools
        dict(name="mass b64 e4m3", op="mass", B=64, lo=512, hi=8192, q_len=1, Hq=32, Hkv=8, d=128,
             ps=16, dtype="e4m3", window=0),
        # 128K keys cut to 8,192, the first 4 and the last 256 protected
        dict(name="evict b1 128k", op="evict", B=1, lo=131072, hi=131072, n_keep=8192, first=4,
             last=256, Hkv=8, ps=16),
        # a batch cut to 2,048 keys each
        dict(name="evict b64 1k-32k", op="evict", B=64, lo=1024, hi=32768, n_keep=2048, first=4,
             last=128, Hkv=8, ps=16),
        # the rows of one sequence moved to the front of its pages
        dict(name="compact b1 32k", op="compact", B=1, lo=32768, hi=32768, n_keep=8192, first=4,
             Hkv=8, d=128, ps=16, dtype="bf16"),
        # a batch; sequences within the budget move nothing
        dict(name="compact b64 8k", op="compact", B=64, lo=512, hi=8192, n_keep=2048, first=4,
             Hkv=8, d=128, ps=16, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "attend", "mass", "evict", "compact"])
    B = _spread(rng, 1, 96)
    # keys of the whole batch, within the largest listed case of the operator
    most = dict(bounds=57344, select=900000, attend=500000, mass=270000, evict=900000,
                compact=270000)[op]
    hi = _spread(rng, 1 if B > 1 else 16, max(64, min(131072, most // B)))
    lo = rng.choice([0, 1, hi // 8, hi // 2, hi]) if B > 1 else hi
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, B=B, lo=min(lo, hi), hi=hi, Hkv=Hkv, ps=rng.choice([8, 16, 16, 32, 64]))
    if op != "evict":
        c["d"] = rng.choice([64, 128, 128])
    if op in ("select", "attend", "mass"):
        group = rng.choice([1, 2, 4, 5, 8])
        c["Hq"] = Hkv * group
    if op == "bounds":
        c["new"] = rng.choice([1, 1, rng.randint(2, 300), hi])
        c["new"] = max(1, min(c["new"], hi))
    if op == "select":
        c["qdtype"] = rng.choice(["bf16", "f32"])
    if op in ("select", "attend"):
        c["n_select"] = _spread(rng, 3, 384)
    if op == "select":
        c["first"] = rng.randint(0, 1)
        c["last"] = rng.randint(1, 2)
    if op == "mass":
        c["q_len"] = rng.choice([1, 1, 2, 3]) if group <= 5 else 1
        c["window"] = rng.choice([0, 0, max(1, hi // 2)])
    if op in ("evict", "compact"):
        c["n_keep"] = _spread(rng, 8, max(16, hi))
        c["first"] = rng.randint(0, 4)
    if op == "evict":
        c["last"] = rng.randint(0, min(4, c["n_keep"] - c["first"]))
    if op in ("bounds", "attend", "mass"):
        c["dtype"] = rng.choice(["bf16", "bf16", "f32", "e4m3", "int8"])
        if c["dtype"] == "f32" and op == "mass":
            c["q_len"] = 1
        if c["dtype"] in ("e4m3", "int8"):
            c["d"] = 128
        if c["dtype"] == "int8":
            c["ps"] = max(16, c["ps"])
    if op == "compact":
        c["dtype"] = rng.choice(["bf16", "f32"])
    return c


# ------------------------------------------------------------------ inputs --

def _lens(case):
    """The batch's lengths, evenly spread over lo .. hi (their order goes by the seed)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _randn(shape, dtype, g):
    """N(0,1) with 1% of the values times 8, rounded once to the type."""
    x = torch.randn(shape, device=DEV, dtype=torch.bfloat16 if dtype != torch.float32 else dtype,
                    generator=g)
    hit = torch.rand(shape, device=DEV, dtype=torch.float16, generator=g) < 0.01
    return torch.where(hit, x * 8, x).to(dtype)


def _pool(s, case, P, g, names):
    """Pools of P pages and one spare that no table names, so that plain scatters have a place
    for entries that are not there; the framework gets the first P."""
    ps, Hkv, d = case["ps"], case["Hkv"], case["d"]
    for n in names:
        if case["dtype"] == "int8":
            s[n + "_all"] = torch.randint(-127, 128, (P + 1, ps, Hkv, d), device=DEV,
                                          dtype=torch.int8, generator=g)
            s[n + "_scales"] = torch.rand((P + 1, Hkv, ps), device=DEV, generator=g) * 0.045 + 0.005
        else:
            s[n + "_all"] = _randn((P + 1, ps, Hkv, d), POOL_TYPES[case["dtype"]], g)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, B, ps, Hkv = case["op"], case["B"], case["ps"], case["Hkv"]
    lens = torch.tensor(_lens(case), device=DEV, dtype=torch.int32)
    lens = lens[torch.randperm(B, device=DEV, generator=g)].contiguous()
    blocks = [-(-n // ps) for n in lens.tolist()]
    W = max(1, max(blocks))
    P = max(1, sum(blocks)) + 3
    order = torch.randperm(P, device=DEV, generator=g).int()
    table = torch.full((B, W), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case=dict(case), op=op, lens=lens, table=table, W=W, P=P, N=W * ps)
    nb = (lens + ps - 1) // ps
    if op == "bounds":
        _pool(s, case, P, g, ("k",))
        d = case["d"]
        s["first_new"] = (lens - case["new"]).clamp(min=0).int()
        s["most"] = min(W, -(-case["new"] // ps) + 1)
        s["bounds_all"] = torch.randint(-127, 128, (P + 1, Hkv, 2, d), device=DEV,
                                        dtype=torch.int8, generator=g)
        s["bscales_all"] = torch.rand((P + 1, Hkv), device=DEV, generator=g) * 0.04
    if op == "select":
        d = case["d"]
        hi = torch.randint(8, 128, (P, Hkv, d), device=DEV, generator=g)
        low = -torch.randint(8, 128, (P, Hkv, d), device=DEV, generator=g)
        s["bounds"] = torch.stack((hi, low), 2).to(torch.int8)
        s["bscales"] = (2 + 4 * torch.rand((P, Hkv), device=DEV, generator=g)).bfloat16().float() / 127
        s["q"] = _randn((B, case["Hq"], d), POOL_TYPES[case["qdtype"]], g)
    if op in ("attend", "mass"):
        _pool(s, case, P, g, ("k", "v"))
        shape = (B, case["Hq"], case["d"])
        if op == "mass":
            shape = (B, case["q_len"]) + shape[1:]
        s["q"] = _randn(shape, torch.float32 if case["dtype"] == "f32" else torch.bfloat16, g)
        s["scale"] = 1.0 / math.sqrt(case["d"])
    if op == "attend":
        n = case["n_select"]
        # each head's own random pages, the sequence's last one always among them
        r = torch.rand((B, Hkv, W), device=DEV, generator=g)
        i = torch.arange(W, device=DEV)
        r = torch.where(i == (nb - 1)[:, None, None], -1.0, r)
        r = torch.where(i < nb[:, None, None], r, 2.0)
        pick = r.argsort(-1)[..., :n]
        pick = torch.where(pick < nb[:, None, None], pick, W).sort(-1).values
        got = torch.gather(table[:, None].expand(B, Hkv, W), 2, pick.clamp(max=W - 1))
        pages = torch.full((B, Hkv, n), -1, device=DEV, dtype=torch.int32)
        pages[..., :pick.shape[-1]] = torch.where(pick < W, got, -1)
        s["pages"] = pages
        s["page_lens"] = torch.where(nb > n, (n - 1) * ps + (lens - 1) % ps + 1, lens).int()
    if op in ("mass", "evict", "compact"):
        # weights as steps gather them: heavy-tailed, some keys (the newest) with none at all;
        # for the step that adds to them, those of a few steps before it
        tail = 1 if op == "mass" else 3
        m = torch.exp(tail * torch.randn((B, Hkv, s["N"]), device=DEV, generator=g))
        m = m * (4.0 / max(case["hi"], 1))
        m = torch.where(torch.rand(m.shape, device=DEV, generator=g) < 0.02, 0.0, m)
        s["mass"] = torch.where(torch.arange(s["N"], device=DEV) < lens[:, None, None], m, 0.0)
    if op == "compact":
        _pool(s, case, P, g, ("k", "v"))
        n = case["n_keep"]
        j = torch.arange(s["N"], device=DEV)
        r = torch.where(j < case["first"], -1.0, torch.rand(m.shape, device=DEV, generator=g))
        r = torch.where(j < lens[:, None, None], r, 2.0)
        pick = r.argsort(-1)[..., :n]
        pick = torch.where(pick < lens[:, None, None], pick, s["N"]).sort(-1).values
        keep = torch.full((B, Hkv, n), -1, device=DEV, dtype=torch.int32)
        keep[..., :pick.shape[-1]] = torch.where(pick < s["N"], pick, -1).int()
        s["keep"] = keep
        s["new_lens"] = lens.clamp(max=n).int()
    return s


# --------------------------------------------------------------- the passes --

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _values(s, name, pages):
    """Pages of a pool as float32 values [..., ps, Hkv, d]."""
    x = s[name + "_all"][pages].float()
    if s["case"]["dtype"] == "int8":
        x = x * s[name + "_scales"][pages].transpose(-1, -2).unsqueeze(-1)
    return x


def _div(x, y):
    """x / y and 0 where y is 0; y is a tensor, so that the quotient is rounded once."""
    return torch.where(y > 0, x / torch.where(y > 0, y, 1.0), 0.0)


def _codes(x, s):
    return torch.round(_div(x, s)).clamp(-127, 127)


def _plain_bounds(s):
    c, ps, P = s["case"], s["case"]["ps"], s["P"]
    nb = (s["lens"].long() + ps - 1) // ps
    blk = (s["first_new"].long() // ps)[:, None] + torch.arange(s["most"], device=DEV)
    live = blk < nb[:, None]
    page = torch.gather(s["table"], 1, blk.clamp(max=s["W"] - 1)).long()
    page = torch.where(live, page, P)
    k = _values(s, "k", page)  # [B, most, ps, Hkv, d]
    key = blk[..., None] * ps + torch.arange(ps, device=DEV)
    here = (key < s["lens"][:, None, None])[..., None, None]
    top = torch.where(here, k, -math.inf).amax(2)
    low = torch.where(here, k, math.inf).amin(2)
    both = torch.stack((top, low), 3)  # [B, most, Hkv, 2, d]
    both = torch.where(live[..., None, None, None], both, 0.0)
    m127 = torch.full((), 127.0, device=DEV)
    scale = both.abs().amax((3, 4)) / m127
    s["bounds_all"][page] = _codes(both, scale[..., None, None]).to(torch.int8)
    s["bscales_all"][page] = scale
    return s["bounds_all"][:P] * s["bscales_all"][:P, :, None, None]


def _top(score, n, count, N):
    """The n of largest score of each row in ascending order (ties: the lowest index), the rest
    of the n being N; entries at or past `count` are none."""
    pick = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    pick = torch.where(pick < count, pick, N).sort(-1).values
    if pick.shape[-1] < n:
        pick = torch.nn.functional.pad(pick, (0, n - pick.shape[-1]), value=N)
    return pick


def _plain_select(s):
    c, ps, W = s["case"], s["case"]["ps"], s["W"]
    B, Hkv, d, n = c["B"], c["Hkv"], c["d"], c["n_select"]
    nb = (s["lens"].long() + ps - 1) // ps
    m127 = torch.full((), 127.0, device=DEV)
    q = s["q"].float().view(B, Hkv, -1, d)
    t = q.abs().amax(-1, keepdim=True) / m127
    a = _codes(q, t)
    a = torch.cat((a.clamp(min=0), a.clamp(max=0)), -1)
    page = s["table"].long().clamp(min=0)
    both = s["bounds"][page].float().flatten(3)  # [B, W, Hkv, 2 d]
    dots = torch.einsum("bgrd,bwgd->bgrw", a, both)  # whole numbers below 2^24: exact
    dots = dots * s["bscales"][page].transpose(1, 2)[:, :, None]
    score = (dots * t).amax(2)
    i = torch.arange(W, device=DEV)
    forced = (i < c["first"]) | (i >= (nb - c["last"])[:, None, None])
    score = torch.where(forced, math.inf, score)
    score = torch.where(i < nb[:, None, None], score, -math.inf)
    pick = _top(score, n, nb[:, None, None], W)
    got = torch.gather(s["table"][:, None].expand(B, Hkv, W), 2, pick.clamp(max=W - 1))
    lens = torch.where(nb > n, (n - 1) * ps + (s["lens"].long() - 1) % ps + 1, s["lens"].long())
    return torch.where(pick < W, got, -1), lens.int()


def _softmax(x, live):
    """Rows of x over their live places; 0 where a row has none."""
    x = torch.where(live, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_attend(s):
    c, ps = s["case"], s["case"]["ps"]
    B, Hkv, d, n = c["B"], c["Hkv"], c["d"], c["n_select"]
    page = s["pages"].long().clamp(min=0)
    head = torch.arange(Hkv, device=DEV)[:, None]

    def rows(name):
        x = s[name + "_all"].transpose(1, 2)[page, head].float()  # [B, Hkv, n, ps, d]
        if c["dtype"] == "int8":
            x = x * s[name + "_scales"][page, head].unsqueeze(-1)
        return x.flatten(2, 3)

    q = s["q"].float().view(B, Hkv, -1, d)
    x = torch.einsum("bgrd,bgkd->bgrk", q, rows("k")) * s["scale"]
    live = torch.arange(n * ps, device=DEV) < s["page_lens"][:, None, None, None]
    p = _softmax(x, live)
    return torch.einsum("bgrk,bgkd->bgrd", p, rows("v")).reshape(B, c["Hq"], d)


def _plain_mass(s):
    c, N = s["case"], s["N"]
    B, Hkv, d, T = c["B"], c["Hkv"], c["d"], c["q_len"]
    page = s["table"].long().clamp(min=0)
    k = _values(s, "k", page).flatten(1, 2)  # [B, N, Hkv, d]
    q = s["q"].float().view(B, T, Hkv, -1, d)
    x = torch.einsum("btgrd,bkgd->btgrk", q, k) * s["scale"]
    del k
    j = torch.arange(N, device=DEV)
    pos = (s["lens"].long()[:, None] - T + torch.arange(T, device=DEV))[:, :, None]
    live = j <= pos
    if c["window"] > 0:
        live = live & (j > pos - c["window"])
    p = _softmax(x, live[:, :, None, None])
    del x
    s["mass"] += p.sum((1, 3))
    v = _values(s, "v", page).flatten(1, 2)
    # unlisted pages of a shorter row stand for nothing: their weights are 0
    out = torch.einsum("btgrk,bkgd->btgrd", p, v).reshape(B, T, c["Hq"], d)
    return out, s["mass"]


def _plain_evict(s):
    c, N, n = s["case"], s["N"], s["case"]["n_keep"]
    L = s["lens"].long()[:, None, None]
    j = torch.arange(N, device=DEV)
    forced = (j < c["first"]) | (j >= L - c["last"])
    score = torch.where(forced, math.inf, s["mass"])
    score = torch.where(j < L, score, -math.inf)
    pick = _top(score, n, L, N)
    return torch.where(pick < N, pick, -1).int(), s["lens"].clamp(max=n)


def _plain_compact(s):
    c, ps, P, n, N = s["case"], s["case"]["ps"], s["P"], s["case"]["n_keep"], s["N"]
    B, Hkv = c["B"], c["Hkv"]
    j = torch.arange(n, device=DEV).expand(B, Hkv, n)
    live = j < s["new_lens"][:, None, None]
    src = torch.where(live, s["keep"].long(), 0)
    table = s["table"].long()[:, None].expand(B, Hkv, s["W"])

    def place(i):
        page = torch.gather(table, 2, (i // ps).clamp(max=s["W"] - 1))
        return torch.where(live, page, P), torch.where(live, i % ps, 0)

    head = torch.arange(Hkv, device=DEV)[:, None].expand(B, Hkv, n)
    (pd, od), (pf, of) = place(j), place(src)
    for name in ("k", "v"):
        pool = s[name + "_all"]
        pool[pd, od, head] = pool[pf, of, head]
    i = torch.arange(N, device=DEV)
    m = torch.gather(s["mass"], 2, src)
    new = torch.where(i < s["lens"][:, None, None], 0.0, s["mass"])
    new[..., :min(n, N)] = torch.where(live, m, torch.nn.functional.pad(
        new, (0, max(0, n - N)))[..., :n])[..., :N]
    s["mass"].copy_(new)
    return s["k_all"][:P], s["v_all"][:P], s["mass"]


_plain = dict(bounds=_plain_bounds, select=_plain_select, attend=_plain_attend, mass=_plain_mass,
              evict=_plain_evict, compact=_plain_compact)


def _tl():
    import paged_kv_attention_cache_gb300 as tl
    return tl


def _own_bounds(s):
    P = s["P"]
    if s["case"]["dtype"] == "int8":
        _tl().tl_kv_page_bounds_int8(s["k_all"][:P], s["k_scales"][:P], s["table"], s["lens"],
                                     s["bounds_all"][:P], s["bscales_all"][:P],
                                     first_new=s["first_new"])
    else:
        _tl().tl_kv_page_bounds(s["k_all"][:P], s["table"], s["lens"], s["bounds_all"][:P],
                                s["bscales_all"][:P], first_new=s["first_new"])
    return s["bounds_all"][:P] * s["bscales_all"][:P, :, None, None]


def _own_select(s):
    c = s["case"]
    return _tl().tl_kv_page_select(s["q"], s["bounds"], s["bscales"], s["table"], s["lens"],
                                   c["ps"], c["n_select"], keep_first=c["first"],
                                   keep_last=c["last"])


def _own_attend(s):
    P = s["P"]
    if s["case"]["dtype"] == "int8":
        return _tl().tl_paged_attn_decode_pages_int8(
            s["q"], s["k_all"][:P], s["v_all"][:P], s["k_scales"][:P], s["v_scales"][:P],
            s["pages"], s["page_lens"], s["scale"])
    return _tl().tl_paged_attn_decode_pages(s["q"], s["k_all"][:P], s["v_all"][:P], s["pages"],
                                            s["page_lens"], s["scale"])


def _own_mass(s):
    P, w = s["P"], s["case"]["window"]
    if s["case"]["dtype"] == "int8":
        out = _tl().tl_paged_attn_decode_mass_int8(
            s["q"], s["k_all"][:P], s["v_all"][:P], s["k_scales"][:P], s["v_scales"][:P],
            s["table"], s["lens"], s["mass"], s["scale"], window=w)
    else:
        out = _tl().tl_paged_attn_decode_mass(s["q"], s["k_all"][:P], s["v_all"][:P], s["table"],
                                              s["lens"], s["mass"], s["scale"], window=w)
    return out, s["mass"]


def _own_evict(s):
    c = s["case"]
    return _tl().tl_kv_evict_select(s["mass"], s["lens"], c["n_keep"], keep_first=c["first"],
                                    keep_last=c["last"])


def _own_compact(s):
    P = s["P"]
    _tl().tl_kv_cache_compact(s["k_all"][:P], s["v_all"][:P], s["table"], s["lens"], s["keep"],
                              s["new_lens"], mass=s["mass"])
    return s["k_all"][:P], s["v_all"][:P], s["mass"]


_own = dict(bounds=_own_bounds, select=_own_select, attend=_own_attend, mass=_own_mass,
            evict=_own_evict, compact=_own_compact)


# -------------------------------------------------------------------- work --

def work(case):
    op, B, ps, Hkv = case["op"], case["B"], case["ps"], case["Hkv"]
    lens = _lens(case)
    e = dict(bf16=2, f32=4, e4m3=1, int8=1)[case.get("dtype", "bf16")]
    row = case.get("d", 0) * e + (4 if case.get("dtype") == "int8" else 0)
    d = case.get("d", 0)
    if op == "bounds":
        keys = pages = 0
        for n in lens:
            first = max(0, n - case["new"]) // ps
            keys += n - first * ps
            pages += -(-n // ps) - first
        # the values stand for int8 codes: a pass writes codes and scales
        return dict(bytes=Hkv * (keys * row + pages * (2 * d + 4)) + 4 * pages + 8 * B,
                    flops=2 * Hkv * keys * d)
    if op == "select":
        nb = [-(-n // ps) for n in lens]
        qb = 2 if case["qdtype"] == "bf16" else 4
        return dict(bytes=sum(nb) * (Hkv * (2 * d + 4) + 4) + B * (case["Hq"] * d * qb + 8)
                    + 4 * B * Hkv * case["n_select"],
                    flops=4 * sum(nb) * case["Hq"] * d)
    if op == "attend":
        keys = sum(min(n, case["n_select"] * ps) for n in lens)
        return dict(bytes=2 * Hkv * keys * row + 4 * Hkv * sum(
            min(-(-n // ps), case["n_select"]) for n in lens) + B * case["Hq"] * d * 6,
            flops=4 * keys * case["Hq"] * d)
    if op == "mass":
        T, w = case["q_len"], case["window"]
        keys = sum(min(n, w + T - 1) if w > 0 else n for n in lens)
        return dict(bytes=Hkv * keys * (2 * row + 8) + 4 * sum(-(-n // ps) for n in lens)
                    + B * T * case["Hq"] * d * 6, flops=4 * keys * T * case["Hq"] * d)
    if op == "evict":
        return dict(bytes=4 * Hkv * (sum(lens) + sum(min(n, case["n_keep"]) for n in lens)),
                    flops=2 * Hkv * sum(lens))
    kept = sum(min(n, case["n_keep"]) for n in lens)
    moved = sum(max(0, case["n_keep"] - case["first"]) for n in lens if n > case["n_keep"])
    return dict(bytes=Hkv * (4 * moved * row + 8 * kept + 4 * sum(lens)), flops=0)


# ------------------------------------------------------------------- exact --

def _pool64(s, name):
    x = s[name + "_all"]
    x = x.float().double() if x.dtype == torch.float8_e4m3fn else x.double()
    if s["case"]["dtype"] == "int8":
        x = x * s[name + "_scales"].double().permute(0, 2, 1)[..., None]
        if s["op"] == "bounds":  # a key's value there is the 32-bit product
            x = x.float().double()
    return x


def _attend64(q, k, v, scale, sees):
    """softmax(scale q k^T) v in float64 for rows q [R, d] over keys [n, d]; sees [R, n]."""
    z = (q.double() @ k.T) * scale
    z = z.masked_fill(~sees, -math.inf)
    e = torch.exp(z - z.max(1, keepdim=True).values.clamp(min=-1e300))
    tot = e.sum(1, keepdim=True)
    w = e / tot.masked_fill(tot == 0, 1)
    return w, w @ v


def exact(case, seed):
    s = prepare(case, seed)
    op, B, ps, Hkv = case["op"], case["B"], case["ps"], case["Hkv"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if op == "bounds":
        k = _pool64(s, "k")
        first = s["first_new"].tolist()
        out = s["bounds_all"][:s["P"]].double() * s["bscales_all"][:s["P"]].double()[..., None, None]
        pages, counts = [], []
        for b, n in enumerate(lens):
            for i in range(first[b] // ps, -(-n // ps)):
                pages.append(table[b][i])
                counts.append(min(ps, n - i * ps))
        if pages:
            at = torch.tensor(pages, device=DEV)
            dead = torch.arange(ps, device=DEV) >= torch.tensor(counts, device=DEV)[:, None]
            dead = dead[..., None, None]
            hi = k[at].masked_fill(dead, -math.inf).max(1).values
            lo = k[at].masked_fill(dead, math.inf).min(1).values
            x = torch.stack((hi, lo), 2)
            # the scale is a 32-bit number, and a code is the 32-bit quotient's nearest whole
            # number: with few bits in the keys, quotients fall on halves often
            step = (x.abs().flatten(2).max(2).values / 127).float().double()[..., None, None]
            codes = (x / step.masked_fill(step == 0, 1)).float().double().round()
            out[at] = codes.clamp(-127, 127) * step
        return out
    if op == "select":
        picked = []
        totals = []
        n = case["n_select"]
        for b, L in enumerate(lens):
            nb = -(-L // ps)
            totals.append(L if nb <= n else (n - 1) * ps + (L - 1) % ps + 1)
            pages = torch.tensor(table[b][:nb], device=DEV, dtype=torch.long)
            q = s["q"][b].double().view(Hkv, -1, case["d"])
            t = (q.float().abs().amax(-1, keepdim=True).double() / 127).float().double()
            a = torch.round((q / t).float()).clamp(-127, 127).double()
            x = s["bounds"][pages].double()
            big = torch.einsum("grd,pgd->grp", a * (a >= 0), x[:, :, 0]) + \
                torch.einsum("grd,pgd->grp", a * (a < 0), x[:, :, 1])
            z = (big.float() * s["bscales"][pages].T[:, None]) * t.float()
            z = z.amax(1).double()
            if nb:
                z[:, :min(case["first"], nb)] = math.inf
                z[:, max(0, nb - case["last"]):] = math.inf
            order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :n].sort(1).values
            row = torch.full((Hkv, n), -1, device=DEV, dtype=torch.int32)
            row[:, :order.shape[1]] = pages.int()[order] if nb else row[:, :0]
            picked.append(row)
        return torch.stack(picked), torch.tensor(totals, device=DEV, dtype=torch.int32)
    if op == "attend":
        k, v = s["k_all"], s["v_all"]
        out = torch.zeros((B, case["Hq"], case["d"]), device=DEV, dtype=torch.float64)
        group = case["Hq"] // Hkv
        if case["dtype"] == "int8":
            k, v = _pool64(s, "k"), _pool64(s, "v")
        for b, n in enumerate(s["page_lens"].tolist()):
            for g in range(Hkv):
                pages = s["pages"][b, g, :-(-n // ps)].long()
                kk, vv = (x[pages, :, g].float().double() if case["dtype"] == "e4m3"
                          else x[pages, :, g].double() for x in (k, v))
                kk, vv = (x.reshape(-1, case["d"])[:n] for x in (kk, vv))
                rows = slice(g * group, (g + 1) * group)
                if n:
                    sees = torch.ones((group, n), device=DEV, dtype=torch.bool)
                    out[b, rows] = _attend64(s["q"][b, rows], kk, vv, s["scale"], sees)[1]
        return out
    if op == "mass":
        k, v = _pool64(s, "k"), _pool64(s, "v")
        T, group, d = case["q_len"], case["Hq"] // Hkv, case["d"]
        out = torch.zeros((B, T, case["Hq"], d), device=DEV, dtype=torch.float64)
        mass = s["mass"].double()
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = torch.tensor(table[b][:-(-n // ps)], device=DEV)
            kb, vb = (x[pages].flatten(0, 1)[:n] for x in (k, v))
            key = torch.arange(n, device=DEV)
            for t in range(T):
                p = n - T + t
                sees = key <= p
                if case["window"] > 0:
                    sees &= key >= p - case["window"] + 1
                for g in range(Hkv):
                    rows = slice(g * group, (g + 1) * group)
                    w, o = _attend64(s["q"][b, t, rows], kb[:, g], vb[:, g], s["scale"],
                                     sees.expand(group, n))
                    out[b, t, rows] = o
                    mass[b, g, :n] += w.sum(0)
        return out, mass
    if op == "evict":
        n = case["n_keep"]
        keep = torch.full((B, Hkv, n), -1, device=DEV, dtype=torch.int32)
        for b, L in enumerate(lens):
            z = s["mass"][b, :, :L].double()
            z[:, :case["first"]] = math.inf
            z[:, max(0, L - case["last"]):] = math.inf
            got = torch.argsort(z, dim=1, descending=True, stable=True)[:, :n].sort(1).values
            keep[b, :, :got.shape[1]] = got.int()
        return keep, torch.tensor([min(L, n) for L in lens], device=DEV, dtype=torch.int32)
    # compaction moves values and computes none
    return None
