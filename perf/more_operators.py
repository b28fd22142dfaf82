"""Rotary positions around a paged KV cache, for measurement.

Three operators: the rotation of query or key rows at their positions; the
append of a step's or a prompt's keys and values to the pages, with queries and
keys rotated on the way; and the compaction of an evicted cache whose kept keys
are turned to the positions they move to.  Each case names one operator; run()
computes it in plain torch where `own` is false and through the package's entry
points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's decode step: the queries of one token far into a conversation
        dict(name="rope b1 step", op="rope", N=1, H=32, d=128, rot=128, inter=False, dtype="bf16",
             fused=0, far=30000, base=500000.0, scaling="none"),
        # a prompt chunk's queries, read where the fused projection left them (8 KV heads
        # beside them), frequencies scaled in bands for long contexts
        dict(name="rope 16k of qkv", op="rope", N=16384, H=32, d=128, rot=128, inter=False,
             dtype="bf16", fused=16, far=100000, base=500000.0, scaling="bands"),
        # interleaved pairs over half of the head, float32 activations
        dict(name="rope 4k f32 half head", op="rope", N=4096, H=32, d=128, rot=64, inter=True,
             dtype="f32", fused=0, far=4096, base=10000.0, scaling="none"),
        # an odd number of tokens of short heads whose rotated part is a quarter, positions
        # near a million, interpolated
        dict(name="rope 2777 far", op="rope", N=2777, H=12, d=64, rot=16, inter=False,
             dtype="bf16", fused=0, far=1000000, base=10000.0, scaling="linear"),
        # one decode step of one sequence, rows of the fused projection
        dict(name="append b1 step", op="append", B=1, T=1, lo=1, past=32768, Hq=32, Hkv=8, d=128,
             ps=16, rot=128, inter=False, dtype="bf16", src="bf16", fused=True, base=500000.0,
             scaling="none"),
        # one decode step of 64 sequences
        dict(name="append b64 step", op="append", B=64, T=1, lo=1, past=8192, Hq=32, Hkv=8, d=128,
             ps=16, rot=128, inter=False, dtype="bf16", src="bf16", fused=True, base=500000.0,
             scaling="none"),
        # a right-aligned batch of eight prompts of 1,024 to 2,048 tokens
        dict(name="append prompts 16k", op="append", B=8, T=2048, lo=1024, past=512, Hq=32, Hkv=8,
             d=128, ps=16, rot=128, inter=False, dtype="bf16", src="bf16", fused=True,
             base=500000.0, scaling="bands"),
        # the verify step of a speculative batch over e4m3 pools, interleaved pairs
        dict(name="append verify e4m3", op="append", B=64, T=4, lo=4, past=2048, Hq=40, Hkv=8,
             d=128, ps=16, rot=128, inter=True, dtype="e4m3", src="bf16", fused=False,
             base=10000.0, scaling="ramp"),
        # a prompt into int8 pools
        dict(name="append 4k int8", op="append", B=2, T=2048, lo=1500, past=0, Hq=32, Hkv=8, d=128,
             ps=16, rot=64, inter=False, dtype="int8", src="bf16", fused=True, base=10000.0,
             scaling="none"),
        # one long conversation cut from 32K keys to 8K, its positions closed up
        dict(name="close b1 32k", op="close", B=1, lo=32768, hi=32768, n_keep=8192, first=4,
             Hkv=8, d=128, ps=16, rot=128, inter=False, dtype="bf16", base=500000.0,
             scaling="none"),
        # a ragged batch cut to 2,048 keys each; shorter sequences move nothing
        dict(name="close b64 8k", op="close", B=64, lo=512, hi=8192, n_keep=2048, first=4, Hkv=8,
             d=128, ps=16, rot=128, inter=False, dtype="bf16", base=500000.0, scaling="none"),
        # a batch over e4m3 pools, half of the head rotated
        dict(name="close b24 e4m3", op="close", B=24, lo=1024, hi=8192, n_keep=1500, first=4,
             Hkv=4, d=128, ps=32, rot=64, inter=True, dtype="e4m3", base=10000.0,
             scaling="linear"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "close"])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    c = dict(op=op, d=d, rot=rng.choice([d, d, d // 2, d // 4]), inter=rng.random() < 0.4,
             base=rng.choice([10000.0, 500000.0]),
             scaling=rng.choice(["none", "none", "linear", "bands", "ramp"]))
    if op == "rope":
        c.update(H=rng.choice([1, 4, 8, 12, 32, 40]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 fused=rng.choice([0, 0, 2, 16]), far=_spread(rng, 16, 1000000))
        # at most the 16K-token case's elements
        c["N"] = _spread(rng, 1, 16384 * 32 * 128 // (c["H"] * d * (2 if c["dtype"] == "f32" else 1)))
        c["N"] = min(c["N"], 60000)
        return c
    Hkv = rng.choice([1, 2, 4, 8])
    ps = rng.choice([8, 16, 16, 32, 64])
    if op == "append":
        c.update(Hkv=Hkv, Hq=Hkv * rng.choice([0, 1, 2, 4, 5, 8]), ps=ps,
                 dtype=rng.choice(["bf16", "bf16", "f32", "e4m3", "int8"]),
                 fused=rng.random() < 0.5, B=_spread(rng, 1, 96))
        c["src"] = c["dtype"] if c["dtype"] in ("bf16", "f32") else rng.choice(["bf16", "bf16", "f32"])
        rows = 8192 if c["src"] == "bf16" else 4096
        c["T"] = rng.choice([1, rng.randint(2, 8), _spread(rng, 1, max(1, rows // c["B"]))])
        c["T"] = min(c["T"], max(1, rows // c["B"]))
        c["lo"] = rng.randint(0, c["T"])
        c["past"] = _spread(rng, 1, max(8, 60000 // c["B"]))
    else:
        B = _spread(rng, 1, 96)
        hi = _spread(rng, 16, max(64, min(32768, 200000 // B)))
        c.update(B=B, hi=hi, lo=rng.choice([0, 1, hi // 8, hi // 2, hi]) if B > 1 else hi, Hkv=Hkv,
                 ps=ps, n_keep=_spread(rng, 8, max(16, hi)), first=rng.randint(0, 4),
                 dtype=rng.choice(["bf16", "bf16", "f32", "e4m3", "int8"]))
    return c


# ------------------------------------------------------------------ inputs --

def _inv_freq(c):
    """(radians a position of each pair, factor of the rotated values), in 64 bits: the
    geometric ladder base^(-2i/rot), and what long contexts make of it."""
    r = c["rot"]
    f = torch.tensor([c["base"] ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)
    turns = 8192 * f / (2 * math.pi)  # turns over the trained length
    if c["scaling"] == "linear":
        return f / 8.0, 1.0
    if c["scaling"] == "bands":  # slow pairs by 8, fast ones as they are, blended between
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / 8.0 * (1 - keep), 1.0
    if c["scaling"] == "ramp":  # a ramp over the pairs' indexes, and a factor
        def at(n):
            return r * math.log(8192 / (n * 2 * math.pi)) / (2 * math.log(c["base"]))
        low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), r - 1)
        i = torch.arange(r // 2, dtype=torch.float64)
        far = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        return f / 8.0 * far + f * (1 - far), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _rope_tables(s, c):
    f, m = _inv_freq(c)
    s["inv"] = f.to(DEV)
    # the table that a program keeps: 2^64 times each pair's turns a position, whole numbers
    s["freqs"] = torch.round(f / (2 * math.pi) * 2.0 ** 64).long().to(DEV)
    s["m"] = m


def _lens(case):
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _news(case):
    B, lo, T = case["B"], case["lo"], case["T"]
    return [T if B == 1 else lo + (T - lo) * i // (B - 1) for i in range(B)]


def _randn(shape, dtype, g):
    """N(0,1) with 1% of the values times 8, rounded once to the type."""
    x = torch.randn(shape, device=DEV, dtype=torch.bfloat16 if dtype != torch.float32 else dtype,
                    generator=g)
    hit = torch.rand(shape, device=DEV, dtype=torch.float16, generator=g) < 0.01
    return torch.where(hit, x * 8, x).to(dtype)


def _pools(s, c, P, g):
    """Pools of P pages and one spare that no table names, so that plain scatters have a place
    for rows that are not there; the framework gets the first P."""
    shape = (P + 1, c["ps"], c["Hkv"], c["d"])
    for n in ("k", "v"):
        if c["dtype"] == "int8":
            s[n] = torch.randint(-127, 128, shape, device=DEV, dtype=torch.int8, generator=g)
            s[n + "_scales"] = torch.rand((P + 1, c["Hkv"], c["ps"]), device=DEV,
                                          generator=g) * 0.045 + 0.005
        else:
            s[n] = _randn(shape, TYPES[c["dtype"]], g)


def _tables(s, lens, ps, g):
    """Shuffled pages for sequences of the given lengths."""
    blocks = [-(-n // ps) for n in lens]
    W = max(1, max(blocks))
    P = max(1, sum(blocks)) + 3
    order = torch.randperm(P, device=DEV, generator=g).int()
    table = torch.full((len(lens), W), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    s.update(table=table, W=W, P=P, lens=torch.tensor(lens, device=DEV, dtype=torch.int32))
    return P


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    c = dict(case)
    s = dict(case=c, op=c["op"])
    _rope_tables(s, c)
    d = c["d"]
    if c["op"] == "rope":
        N, H = c["N"], c["H"]
        rows = _randn((N, H + c["fused"], d), TYPES[c["dtype"]], g)
        s["x"] = rows[:, :H]
        # a few sequences' tokens one behind the other, each from a place of its own
        many = max(1, N // 1000)
        start = torch.randint(0, c["far"], (many,), device=DEV, generator=g)
        i = torch.arange(N, device=DEV)
        s["positions"] = (start[i * many // N] + i).int()
        return s
    ps, Hkv = c["ps"], c["Hkv"]
    if c["op"] == "append":
        B, T, Hq = c["B"], c["T"], c["Hq"]
        # (tokens cached, tokens new) of each sequence: the longest cached have the fewest new
        both = torch.tensor([(c["past"] * (B - b) // B, n) for b, n in enumerate(_news(c))],
                            device=DEV)[torch.randperm(B, device=DEV, generator=g)]
        past, new = both[:, 0], both[:, 1]
        P = _tables(s, (past + new).tolist(), ps, g)
        _pools(s, c, P, g)
        # right-aligned: padding first, at position -1 and slot -1
        t = torch.arange(T, device=DEV) - (T - new[:, None])
        pos = past[:, None] + t
        page = torch.gather(s["table"].long(), 1, (pos.clamp(min=0) // ps).clamp(max=s["W"] - 1))
        s["slots"] = torch.where(t >= 0, page * ps + pos % ps, -1).flatten()
        s["positions"] = torch.where(t >= 0, pos, -1).int().flatten()
        src = TYPES[c["src"]]
        if c["fused"]:
            rows = _randn((B * T, Hq + 2 * Hkv, d), src, g)
            s["q"], s["k_new"], s["v_new"] = rows.split([Hq, Hkv, Hkv], 1)
        else:
            s["q"], s["k_new"], s["v_new"] = (_randn((B * T, h, d), src, g)
                                              for h in (Hq, Hkv, Hkv))
        if Hq == 0:
            s["q"] = None
        if c["dtype"] == "int8":  # where the values that the codes stand for are read to
            s["values"] = [torch.empty((P,) + s["k"].shape[1:], device=DEV, dtype=torch.bfloat16)
                           for _ in range(2)]
        return s
    lens = torch.tensor(_lens(c))[torch.randperm(c["B"], generator=torch.Generator().manual_seed(
        int(seed)))].tolist()
    P = _tables(s, lens, ps, g)
    _pools(s, c, P, g)
    # each head keeps its first keys and others at random, as attention weights leave them
    n, B, N = c["n_keep"], c["B"], s["W"] * ps
    j = torch.arange(N, device=DEV)
    r = torch.where(j < c["first"], -1.0, torch.rand((B, Hkv, N), device=DEV, generator=g))
    r = torch.where(j < s["lens"][:, None, None], r, 2.0)
    pick = r.argsort(-1)[..., :n]
    pick = torch.where(pick < s["lens"][:, None, None], pick, N).sort(-1).values
    keep = torch.full((B, Hkv, n), -1, device=DEV, dtype=torch.int32)
    keep[..., :pick.shape[-1]] = torch.where(pick < N, pick, -1).int()
    s["keep"] = keep
    s["new_lens"] = s["lens"].clamp(max=n).int()
    if c["dtype"] == "int8":
        s["values"] = [torch.empty((P,) + s["k"].shape[1:], device=DEV, dtype=torch.bfloat16)
                       for _ in range(2)]
    return s


# --------------------------------------------------------------- the passes --

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _held(s):
    """The pools' values: of int8 pools what the codes stand for, in 16 bits (a code has 8)."""
    P = s["P"]
    if s["case"]["dtype"] != "int8":
        return s["k"][:P], s["v"][:P]
    return tuple(torch.mul(s[n][:P], s[n + "_scales"][:P].transpose(1, 2).unsqueeze(-1), out=o)
                 for n, o in zip(("k", "v"), s["values"]))


def _rotated(s, x, pos, m):
    """Rows x [..., d] (float32) rotated at pos [...], in 32 bits; the angles, which pass what
    32 bits can tell apart, in 64."""
    c = s["case"]
    r = c["rot"]
    a = pos.double().unsqueeze(-1) * s["inv"]
    cos, sin = (torch.cos(a) * m).float(), (torch.sin(a) * m).float()
    if c["inter"]:
        lo, hi = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), -1).flatten(-2)
    else:
        lo, hi = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_rope(s):
    x = s["x"]
    pos = s["positions"].unsqueeze(1)  # one angle for all heads of a token
    return _rotated(s, x.float(), pos, s["m"]).to(x.dtype)


def _quotient(x, y):
    """x / y and 0 where y is 0."""
    return torch.where(y > 0, x / torch.where(y > 0, y, 1.0), 0.0)


def _store(s, name, x, page, off, head):
    """Rows x [n..., d] (float32) into a pool's places, rounded to its type."""
    c = s["case"]
    if c["dtype"] == "int8":
        scale = x.abs().amax(-1) / torch.full((), 127.0, device=DEV)
        s[name][page, off, head] = torch.round(_quotient(x, scale[..., None])).to(torch.int8)
        s[name + "_scales"][page, head, off] = scale
    else:
        if c["dtype"] == "e4m3":
            x = x.clamp(-448.0, 448.0)
        s[name][page, off, head] = x.to(s[name].dtype)


def _plain_append(s):
    c, P, ps = s["case"], s["P"], s["case"]["ps"]
    live = s["slots"] >= 0
    slot = torch.where(live, s["slots"], P * ps)
    page, off = (slot // ps)[:, None], (slot % ps)[:, None]
    head = torch.arange(c["Hkv"], device=DEV)
    pos = s["positions"].unsqueeze(1)
    _store(s, "k", _rotated(s, s["k_new"].float(), pos, s["m"]), page, off, head)
    _store(s, "v", s["v_new"].float(), page, off, head)
    if s["q"] is None:
        return _held(s)
    q = s["q"].float()
    # padding is taken over as it is
    q = torch.where(live[:, None, None], _rotated(s, q, pos, s["m"]), q).to(s["q"].dtype)
    return (q,) + _held(s)


def _plain_close(s):
    c, ps, P, n, W = s["case"], s["case"]["ps"], s["P"], s["case"]["n_keep"], s["W"]
    B, Hkv = c["B"], c["Hkv"]
    j = torch.arange(n, device=DEV).expand(B, Hkv, n)
    # rows that stay where they are stay as they are
    moved = (j < s["new_lens"][:, None, None]) & (s["keep"] != j)
    src = torch.where(moved, s["keep"].long(), 0)
    table = s["table"].long()[:, None].expand(B, Hkv, W)

    def place(i):
        page = torch.gather(table, 2, (i // ps).clamp(max=W - 1))
        return torch.where(moved, page, P), torch.where(moved, i % ps, 0)

    head = torch.arange(Hkv, device=DEV)[:, None].expand(B, Hkv, n)
    (pd, od), (pf, of) = place(j), place(src)
    k = s["k"][pf, of, head].float()
    if c["dtype"] == "int8":
        k = k * s["k_scales"][pf, head, of].unsqueeze(-1)
        s["v_scales"][pd, head, od] = s["v_scales"][pf, head, of]
    s["v"][pd, od, head] = s["v"][pf, of, head]
    _store(s, "k", _rotated(s, k, j - src, 1.0), pd, od, head)
    return _held(s)


_plain = dict(rope=_plain_rope, append=_plain_append, close=_plain_close)


def _tl():
    import paged_kv_attention_cache_gb300 as tl
    return tl


def _own_rope(s):
    return _tl().tl_rope(s["x"], s["positions"], s["freqs"], interleaved=s["case"]["inter"],
                         rope_scale=s["m"])


def _own_append(s):
    P = s["P"]
    how = dict(interleaved=s["case"]["inter"], rope_scale=s["m"])
    if s["case"]["dtype"] == "int8":
        q = _tl().tl_kv_cache_write_rope_int8(
            s["q"], s["k_new"], s["v_new"], s["k"][:P], s["v"][:P], s["k_scales"][:P],
            s["v_scales"][:P], s["slots"], s["positions"], s["freqs"], **how)
    else:
        q = _tl().tl_kv_cache_write_rope(s["q"], s["k_new"], s["v_new"], s["k"][:P], s["v"][:P],
                                         s["slots"], s["positions"], s["freqs"], **how)
    return _held(s) if q is None else (q,) + _held(s)


def _own_close(s):
    P = s["P"]
    if s["case"]["dtype"] == "int8":
        _tl().tl_kv_cache_compact_rope_int8(
            s["k"][:P], s["v"][:P], s["k_scales"][:P], s["v_scales"][:P], s["table"], s["lens"],
            s["keep"], s["new_lens"], s["freqs"], interleaved=s["case"]["inter"])
    else:
        _tl().tl_kv_cache_compact_rope(s["k"][:P], s["v"][:P], s["table"], s["lens"], s["keep"],
                                       s["new_lens"], s["freqs"], interleaved=s["case"]["inter"])
    return _held(s)


_own = dict(rope=_own_rope, append=_own_append, close=_own_close)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    size = dict(bf16=2, f32=4, e4m3=1, int8=1)
    e = size[c["dtype"]]
    if c["op"] == "rope":
        return dict(bytes=c["N"] * (2 * c["H"] * c["d"] * e + 4) + 4 * c["rot"],
                    flops=3 * c["N"] * c["H"] * c["rot"])
    extra = 4 if c["dtype"] == "int8" else 0
    if c["op"] == "append":
        live, se = sum(_news(c)), size[c["src"]]
        row = c["d"] * (se + e) + extra
        return dict(bytes=c["B"] * c["T"] * (2 * c["Hq"] * c["d"] * se + 12)
                    + 2 * live * c["Hkv"] * row + 4 * c["rot"],
                    flops=3 * live * (c["Hq"] + c["Hkv"]) * c["rot"])
    lens = _lens(c)
    kept = sum(min(n, c["n_keep"]) for n in lens)
    moved = sum(max(0, c["n_keep"] - c["first"]) for n in lens if n > c["n_keep"])
    return dict(bytes=c["Hkv"] * (4 * moved * (c["d"] * e + extra) + 4 * kept) + 4 * c["rot"],
                flops=3 * moved * c["Hkv"] * c["rot"])


# ------------------------------------------------------------------- exact --

def _turn(c, x, pos, m):
    """Rows x [n, H, d] turned by pos [n] (or [n, H]) positions, as products of complex numbers in
    64 bits: a pair is one number, its turn exp(i pos f)."""
    r = c["rot"]
    f = _inv_freq(c)[0].to(DEV)
    pos = pos.double()
    pos = pos[:, None, None] if pos.dim() == 1 else pos[:, :, None]
    x = x.double()
    y = x.clone()
    ends = (slice(0, r, 2), slice(1, r, 2)) if c["inter"] else (slice(0, r // 2),
                                                                slice(r // 2, r))
    z = torch.complex(x[..., ends[0]].contiguous(), x[..., ends[1]].contiguous())
    z = z * torch.polar(torch.full_like(pos * f, m), pos * f)
    y[..., ends[0]], y[..., ends[1]] = z.real, z.imag
    return y


def _pool64(s, name):
    x = s[name][:s["P"]]
    x = x.float().double() if x.dtype == torch.float8_e4m3fn else x.double()
    if s["case"]["dtype"] == "int8":
        x = x * s[name + "_scales"][:s["P"]].double().permute(0, 2, 1)[..., None]
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _turn(c, s["x"], s["positions"], s["m"])
    k, v = _pool64(s, "k"), _pool64(s, "v")
    ps, Hkv, d = c["ps"], c["Hkv"], c["d"]

    def held(x):
        """Rows as their pool holds them: e4m3 within its range, int8 as whole multiples of a
        127th of the row's largest magnitude (a 32-bit number)."""
        if c["dtype"] == "e4m3":
            return x.clamp(-448.0, 448.0)
        if c["dtype"] != "int8":
            return x
        step = (x.abs().amax(-1, keepdim=True) / 127).float().double()
        return torch.round(x / step.masked_fill(step == 0, 1)) * step

    if c["op"] == "append":
        at = (s["slots"] >= 0).nonzero()[:, 0]
        rows = s["slots"][at]
        k.view(-1, Hkv, d)[rows] = held(_turn(c, s["k_new"][at], s["positions"][at], s["m"]))
        v.view(-1, Hkv, d)[rows] = held(s["v_new"][at].double())
        if s["q"] is None:
            return k, v
        q = s["q"].double()
        q[at] = _turn(c, s["q"][at], s["positions"][at], s["m"])
        return q, k, v
    old_k, old_v = k.view(-1, Hkv, d).clone(), v.view(-1, Hkv, d).clone()
    for b, n in enumerate(s["new_lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        to = s["table"][b, j // ps].long() * ps + j % ps
        for h in range(Hkv):
            i = s["keep"][b, h, :n].long()
            frm = s["table"][b, i // ps].long() * ps + i % ps
            row = held(_turn(c, old_k[frm, h:h + 1], j - i, 1.0)[:, 0])
            k.view(-1, Hkv, d)[to, h] = torch.where((i != j)[:, None], row, old_k[frm, h])
            v.view(-1, Hkv, d)[to, h] = old_v[frm, h]
    return k, v
