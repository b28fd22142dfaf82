"""Plain implementations, in 64 bits on the CPU, of the rotary operators (the
rotation of rows, the append that rotates, the compaction that turns keys to
their new positions), from their definitions in the header, and the tolerances
their outputs are held to.

How far a computed rotation may be off, before its rounding to the output's
type.  A cosine or sine is within 2^-23 (tests/test_rope_tables.py), its product
with rope_scale m adds a rounding (2^-24 m), and y = lo c - hi s is one product
and one fused multiply-add, a rounding each: with a = m (|lo| + |hi|) that is at
most a (2^-23 + 2^-24) + a (1 + 2^-22) 2 x 2^-24 < 2.6 x 2^-23 a.  The rounding to
the type is half a step of the value; products below 2^-126 add less than 2^-126.
"""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32, torch.float8_e4m3fn)}


def inv_freq(rot, base=10000.0):
    return np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])


def table(f):
    """freqs of the header from radians a position (0 <= f < pi)."""
    t = np.rint(np.asarray(f, np.float64) / (2 * math.pi) * 2.0 ** 64)
    return torch.tensor([int(x) for x in t], dtype=torch.int64)


def ends(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, pos, f, interleaved, m=1.0):
    """(values, bound on a binary32 implementation's error) of rows x [..., d] in float64 at
    positions pos [...]; rows at negative positions as they are unless pos is a shift (int64)."""
    x = np.asarray(x, np.float64)
    rot = 2 * len(f)
    lo, hi = ends(rot, interleaved)
    a = np.asarray(pos, np.float64)[..., None] * f
    c, s = np.cos(a) * m, np.sin(a) * m
    y, err = x.copy(), np.zeros_like(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    e = m * (np.abs(x[..., lo]) + np.abs(x[..., hi])) * 2.6 * 2.0 ** -23 + 2.0 ** -126
    # the angle in 64 bits: a rounding of the product and one of the frequency
    e = e + m * (np.abs(x[..., lo]) + np.abs(x[..., hi])) * np.abs(a) * 2.0 ** -51
    err[..., lo] = err[..., hi] = e
    return y, err


def as_values(t):
    return (t.float() if t.dtype == torch.float8_e4m3fn else t).double().cpu().numpy()


def close(got, want, err, what):
    """Rounded values of a type within err and half a step of `want`."""
    g = as_values(got)
    half = HALF_STEP[got.dtype]
    tol = err + half * (np.abs(want) + err) * (1 + 2 * half)
    if got.dtype == torch.float8_e4m3fn:  # e4m3: subnormals every 2^-9, values up to 448
        tol = np.maximum(tol, err + 2.0 ** -10)
        want = np.clip(want, -448, 448)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(g - want) / tol):.3f} of the tolerance")


def close_int8(codes, scales, want, err, what):
    """Rows of codes [..., d] and scales [...] against values: the scale is the binary32 quotient
    of the row's largest magnitude (itself within err) by 127; a code is the nearest whole number
    to a binary32 quotient (2^-24 of up to 127 codes) of such a value."""
    c, s = codes.double().cpu().numpy(), scales.double().cpu().numpy()
    top, e = np.abs(want).max(-1), err.max(-1)
    assert (np.abs(s - top / 127) <= e / 127 + 2.0 ** -24 * (top + e) / 127 + 2.0 ** -149).all(), what
    tol = s[..., None] * (0.5 + 127 * 2.0 ** -23) + err
    bad = ~(np.abs(c * s[..., None] - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} codes off"


def randn(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    return torch.where(torch.rand(shape, generator=g) < 0.01, 8 * x, x).to(dtype)


def bits(t):
    return t.reshape(-1).contiguous().view(torch.uint8)
