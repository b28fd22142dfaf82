"""Plain implementations, in 64 bits on the CPU, of the long-context operators
(page bounds, page selection, attention over selected pages, attention that
gathers key weights, eviction, compaction), from their definitions in the
header, and the tolerances their f32 outputs are held to.  Shared inputs for
the GPU tests."""
from __future__ import annotations

import math

import numpy as np
import torch

KINDS = ("bf16", "f32", "e4m3", "int8")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}


class Pools:
    """K and V pools of one kind on the CPU, with their values in f64."""

    def __init__(self, kind, P, ps, hkv, d, seed=0, only_k=False):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.P, self.ps, self.hkv, self.d = kind, P, ps, hkv, d
        self.data, self.scales = {}, {}
        for n in ("k",) if only_k else ("k", "v"):
            if kind == "int8":
                self.data[n] = torch.randint(-127, 128, (P, ps, hkv, d), generator=g,
                                             dtype=torch.int8)
                self.scales[n] = torch.rand((P, hkv, ps), generator=g) * 0.045 + 0.005
            else:
                x = torch.randn((P, ps, hkv, d), generator=g)
                x = torch.where(torch.rand(x.shape, generator=g) < 0.01, 8 * x, x)
                self.data[n] = x.to(TYPES[kind])

    def poison(self, used):
        """NaN (int8: code -128 and a NaN scale) in every slot where used [P, ps] is false."""
        for n, x in self.data.items():
            if self.kind == "int8":
                x[~used] = -128
                self.scales[n].permute(0, 2, 1)[~used] = float("nan")
            elif self.kind == "e4m3":
                x.view(torch.uint8)[~used] = 0x7F
            else:
                x[~used] = float("nan")

    def values(self, n):
        x = self.data[n].float()
        if self.kind == "int8":
            x = x * self.scales[n].permute(0, 2, 1)[..., None]
        return x

    def units(self, n):
        """Magnitudes that 16-bit weights multiply: the values; an int8 pool's codes, whose
        weights carry their scales, the largest of them brought to at least 32."""
        if self.kind != "int8":
            return self.values(n).double().abs()
        scales = self.scales[n]
        return self.data[n].double().abs() * (scales[torch.isfinite(scales)].double().max() / 32)

    def gpu(self):
        out = {n: x.cuda() for n, x in self.data.items()}
        out.update({n + "s": x.cuda() for n, x in self.scales.items()})
        return out


def tables(lens, ps, seed=0, width=None, spare=2):
    """A shuffled block table for the lengths and the number of pages it uses."""
    need = [max(0, -(-n // ps)) for n in lens]
    W = max(1, max(need)) if width is None else width
    P = sum(need) + spare
    perm = np.random.default_rng(seed).permutation(P)
    t = np.full((len(lens), W), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t), P


def used_slots(table, lens, P, ps):
    used = torch.zeros((P, ps), dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // ps], j % ps] = True
    return used


def codes(x, s):
    """round-half-even(x / s) clamped to +-127, the division in binary32."""
    x, s = np.asarray(x, np.float32), np.asarray(s, np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / s)
    return np.where(s > 0, np.clip(np.where(np.isfinite(q), q, 0), -127, 127), 0)


def bounds(values, table, lens, first, ps, b0, s0):
    """The bounds pool b0 [P, h, 2, d] int8 and scales s0 [P, h] after the call."""
    out, sc = b0.clone().numpy(), s0.clone().numpy()
    v = values.numpy()
    for b, L in enumerate(lens):
        f = max(first[b], 0) if first is not None else 0
        if L <= f:
            continue
        for i in range(f // ps, (L - 1) // ps + 1):
            page = int(table[b, i])
            live = v[page, :min(ps, L - i * ps)]
            live = np.where(np.isfinite(live), live, np.float32(0))
            both = np.stack((live.max(0), live.min(0)), 1)  # [h, 2, d]
            s = (np.abs(both).max((1, 2)) / np.float32(127)).astype(np.float32)
            out[page] = codes(both, s[:, None, None])
            sc[page] = s
    return torch.from_numpy(out), torch.from_numpy(sc)


def largest(score, n, first, last):
    """The n places of a row taken: the first and last ones, then the largest scores, the
    lowest index first among equals (NaN below everything); ascending."""
    L = len(score)
    if L <= n:
        return list(range(L))
    x = np.where(np.isnan(score), -np.inf, np.asarray(score, np.float64))
    rank = np.where(np.isnan(score), 1, 0)  # a NaN comes after a -inf
    idx = [i for i in range(L) if first <= i < L - last]
    idx.sort(key=lambda i: (-x[i], rank[i], i))
    return sorted(list(range(first)) + idx[:n - first - last] + list(range(L - last, L)))


def page_scores(q, bnd, sc, row, P):
    """Scores [h_kv, blocks] of the blocks in `row` (table entries) for q [h_q, d]."""
    hkv, d = bnd.shape[1], bnd.shape[3]
    q = q.float().numpy()
    q = np.where(np.isfinite(q), q, np.float32(0)).reshape(hkv, -1, d)
    t = (np.abs(q).max(-1) / np.float32(127)).astype(np.float32)
    a = codes(q, t[..., None]).astype(np.int64)
    ok = (row >= 0) & (row < P)
    x = bnd.numpy()[np.where(ok, row, 0)].astype(np.int64)  # [n, h, 2, d]
    s = sc.numpy()[np.where(ok, row, 0)]
    dots = np.einsum("hrd,nhd->hrn", np.maximum(a, 0), x[:, :, 0]) + \
        np.einsum("hrd,nhd->hrn", np.minimum(a, 0), x[:, :, 1])
    z = (dots.astype(np.float32) * s.T[:, None]).astype(np.float32) * t[..., None]
    z = z.astype(np.float32).max(1)
    return np.where(ok, z, -np.inf)


def page_select(q, bnd, sc, table, lens, ps, n, first, last, P):
    B, W = table.shape
    hkv = bnd.shape[1]
    out = np.full((B, hkv, n), -1, np.int32)
    ln = np.zeros(B, np.int32)
    for b, L in enumerate(lens):
        if L <= 0 or L > W * ps:
            continue
        nb = (L - 1) // ps + 1
        row = table[b, :nb].numpy()
        ln[b] = L if nb <= n else (n - 1) * ps + (L - 1) % ps + 1
        z = page_scores(q[b], bnd, sc, row, P)
        for g in range(hkv):
            got = row[largest(z[g], n, first, last)]
            out[b, g, :len(got)] = got
    return torch.from_numpy(out), torch.from_numpy(ln)


def attend(q, k, v, scale, sees):
    """(weights, output, tolerance weight) of rows q [R, d] over keys k, v [n, d] (f64);
    sees [R, n].  The third is sum_j p_j |v_j|."""
    s = (q @ k.T) * scale
    s = np.where(sees, s, -np.inf)
    top = s.max(1, keepdims=True) if s.shape[1] else np.full((len(q), 1), -np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    tot = e.sum(1, keepdims=True)
    p = e / np.where(tot > 0, tot, 1.0)
    return p, p @ v, p @ np.abs(v)


def score_error(q, k, scale):
    """A bound on the error of a score in the kernels (natural-log units): d products summed in
    f32, each addition off by at most one unit of 2^-23 of the sum of magnitudes (codes widen
    exactly, and a key's scale is one more product)."""
    return (q.shape[-1] + 4) * 2.0 ** -23 * (np.abs(q) @ np.abs(k).T).max() * scale


def out_tolerance(kind, q, k, v_mag, scale, n, v_units):
    """|out - exact| of each output.  Relative, on v_mag = sum_j p_j |v_j|: the score's error
    twice (in the weight and in the sum it is divided by), 2^-21 twice for the exponentials, the
    weight's parts (three of bf16: 2^-23; two of fp16: 2^-21; f32 none) and n + 8 roundings of the
    sums.  Absolute: fp16 parts of a weight below 2^-14 of the largest are off by up to 2^-25,
    times v_units = sum_j |v_j| (see Pools.units)."""
    parts = {"bf16": 2.0 ** -23, "f32": 0.0, "e4m3": 2.0 ** -21, "int8": 2.0 ** -21}[kind]
    rel = 2 * score_error(q, k, scale) + 2 * 2.0 ** -21 + parts + (n + 8) * 2.0 ** -23
    flat = 2.0 ** -25 * v_units if kind in ("e4m3", "int8") else 0.0
    return rel * v_mag + flat + 1e-7


def assert_within(got, want, tol, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} outputs off, worst "
                           f"{np.max(np.abs(got - want) / tol):.2f} of the tolerance")


def default_scale(d):
    return 1.0 / math.sqrt(d)
