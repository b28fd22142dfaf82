"""How far a page's int8 score may lie from the sum it stands for, on the CPU (the GPU calls give the
definition's bits: tests/test_gpu_page_select.py).  Codes are rounded to nearest, so the score is an
estimate of the largest score a key of the page could have, above or below it, not a bound."""
import numpy as np
import pytest
import torch

from tests import long_context_ref as ref

D, PS, NB, GROUP = 128, 16, 64, 4


@pytest.mark.parametrize("kind", ["even", "wide channels", "offset channels", "tiny", "one channel"])
def test_the_score_is_within_the_codes_rounding(kind):
    g = np.random.default_rng(3)
    few = np.arange(D) < 4
    k = g.standard_normal((NB, PS, D)) * 2
    q = g.standard_normal((GROUP, D))
    if kind == "wide channels":
        k *= np.where(few, 30, 1)
    elif kind == "offset channels":
        k += np.where(few, 500, 0)
    elif kind == "tiny":
        k, q = k * 1e-20, q * 1e-10
    elif kind == "one channel":
        q *= np.arange(D) == 7
    keys = torch.from_numpy(k.astype(np.float32)).view(NB, PS, 1, D)
    table = torch.arange(NB, dtype=torch.int32).view(1, NB)
    bnd, sc = ref.bounds(keys, table, [NB * PS], None, PS, torch.zeros((NB, 1, 2, D), dtype=torch.int8),
                         torch.zeros((NB, 1)))
    qt = torch.from_numpy(q.astype(np.float32))
    M, m = (f(keys.double().numpy()[:, :, 0], 1) for f in (np.max, np.min))
    s = sc.double().numpy()[:, 0]
    code = np.abs(bnd.double().numpy()[:, 0]).max(1)  # the larger of the two, [NB, D]
    for h in range(GROUP):
        z = ref.page_scores(qt[h:h + 1], bnd, sc, table[0].numpy(), NB)[0]
        x = qt[h].double().numpy()
        t = float(np.abs(qt[h].numpy()).max() / np.float32(127))
        exact = np.maximum(x * M, x * m).sum(1)
        a = np.abs(ref.codes(qt[h].numpy(), np.float32(t)))
        # a channel: |a c - (q/t)(B/s)| <= (|a| + |c| + 1/2) / 2, both codes off by at most 1/2;
        # the divisions and two products round by 2^-24 each, the quotients of up to 127 by 2^-18
        bound = s * t * ((a + code + 0.5) / 2).sum(1) * (1 + 2.0 ** -16)
        bound += s * t * D * 127 * 127 * 3 * 2.0 ** -24
        assert np.all(np.abs(z - exact) <= bound), kind
        # every key of the page scores at most the exact sum, so at most z + bound
        assert np.all((keys.double().numpy()[:, :, 0] @ x).max(1) <= z + bound)


def test_a_channel_far_below_the_largest_counts_for_nothing():
    """Below 1/254 of the page's largest value a channel's codes are 0: the query's part along it does
    not reach the score."""
    k = torch.zeros((2, PS, 1, D))
    k[..., 0] = 254.0
    k[1, :, 0, 1] = 0.9  # the second page's keys match the query better
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    bnd, sc = ref.bounds(k, table, [2 * PS], None, PS, torch.zeros((2, 1, 2, D), dtype=torch.int8),
                         torch.zeros((2, 1)))
    assert torch.all(bnd[1, 0, :, 1] == 0) and torch.all(bnd[:, 0, :, 0] == 127)
    q = torch.zeros((1, D))
    q[0, 0], q[0, 1] = 1.0, 1.0
    z = ref.page_scores(q, bnd, sc, table[0].numpy(), 2)[0]
    assert z[0] == z[1]  # a tie, which goes to the lower block
    assert ref.largest(z, 1, 0, 0) == [0]
