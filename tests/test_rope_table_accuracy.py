"""How far the entries that tl_rope_freqs makes may be from 2^64 f_i / 2 pi, against 60 decimal
digits (no GPU).

It computes in binary64, u = 2^-53 a rounding.  A plain entry: the exponent -2i/rot is off by u of
itself, which moves base^(-2i/rot) by u ln(1/f); the power is good to an ulp, at most 2u; pi is off
by 0.4 u of itself and the division by it by u.  So f_i / 2 pi is off by at most
u f (ln(1/f) + 3.4) / 2 pi, and as f (ln(1/f) + 3.4) grows with f up to f = 1, by at most
3.4 u / 2 pi < 0.6 x 2^-53 turns: below the 2^-53 that the header states, the rounding of the entry
(2^-65 turns) included."""
from decimal import Decimal, getcontext

import pytest

import paged_kv_attention_cache_gb300 as tl

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 130, 256, 4096])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0, 1e6, 1e8])
def test_plain_entries_are_within_their_bound(rot, base):
    freqs, _ = tl.tl_rope_freqs(rot, base, device="cpu")
    for i, entry in enumerate(freqs.tolist()):
        want = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rot)).exp() / (2 * PI) * 2 ** 64
        assert abs(Decimal(entry % 2 ** 64) - want) <= 2 ** 11, i
