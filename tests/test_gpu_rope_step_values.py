"""A decode step that rotates its queries and keys itself against its definition in 64 bits: the
keys and values it writes, and the attention of the rotated queries over the keys and values held.

The queries that meet the keys are the rotated ones rounded to the rows' type.  Where the 64-bit
rotation is not within its computed error (rope_ref.rotate) of the middle between two values of the
type, that is the same value here; elsewhere it may be the neighbour, one step away, and the scores
may be off by D = scale x (sum of step x |k|), the weights by a factor in exp(-2D) .. exp(2D), and
the output by (exp(2D) - 1) x (sum of weight x |v|).  The attention itself is held to the parity bar
of the decode."""
import numpy as np
import pytest
import torch

from paged_kv_attention_cache_gb300 import build
from tests import parity
from tests import rope_ref as ref
from tests.test_gpu_rope import Pools, i32, table, word
from tests.test_gpu_rope_step import case, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def rounded(x, err, dtype):
    """(x rounded to dtype as float64, how far the rounding of a value within err of x may be)."""
    t = torch.as_tensor(x)
    mid = t.to(dtype).double().numpy()
    lo = torch.as_tensor(x - err).to(dtype).double().numpy()
    hi = torch.as_tensor(x + err).to(dtype).double().numpy()
    return mid, np.maximum(np.abs(hi - mid), np.abs(lo - mid))


def held(pools, name):
    """A pool's values by slot [slots, h_kv, d], float64."""
    x = ref.as_values(pools.t[name]).reshape(-1, pools.hkv, pools.d)
    if pools.kind != "int8":
        return x
    s = pools.t[name + "s"].double().cpu().numpy().transpose(0, 2, 1).reshape(-1, pools.hkv)
    return x * s[..., None]


def attention(q, dq, k, v, scale):
    """Rows q [g, d] (off by up to dq) over keys and values [n, d]: (output, its bound)."""
    z = q @ k.T * scale
    w = np.exp(z - z.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    D = (dq @ np.abs(k).T * scale).max(1, keepdims=True)
    return w @ v, np.expm1(2 * D) * (w @ np.abs(v))


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("group,hkv,d,rot,inter,window,ring", [
    (4, 8, 128, 128, False, 0, 0), (4, 2, 128, 64, True, 0, 0), (1, 3, 128, 128, True, 40, 0),
    (16, 1, 128, 96, False, 0, 0), (5, 2, 128, 20, False, 33, 0), (2, 2, 64, 64, False, 0, 0),
    (4, 2, 128, 128, False, 50, 4),
])
@pytest.mark.parametrize("lens", [[700], [0, 1, 2, 16, 17, 333, 900, 48, 0],
                                  [1 + 7 * b % 300 for b in range(150)]])
def test_the_step_is_the_attention_of_the_rotated_rows(kind, group, hkv, d, rot, inter, window,
                                                       ring, lens):
    if kind in ("e4m3", "int8") and d != 128:
        pytest.skip("one-byte pools have heads of 128")
    if kind == "int8" and ring:
        pytest.skip("no such call")
    ps, m, scale = 16, 1.25, d ** -0.5
    tbl, P, slots, rows, pos = case(kind, lens, group, hkv, d, ps, seed=1, ring=ring)
    pools = Pools(kind, P, ps, hkv, d, 3)
    g = torch.Generator().manual_seed(5)
    rows = [x.copy_(torch.randn(x.shape, generator=g)) for x in rows]
    for n in "kv":
        if kind == "int8":  # values up to 2.5
            pools.t[n + "s"].copy_(0.02 * torch.rand(pools.t[n + "s"].shape, generator=g))
        else:
            pools.t[n].copy_(torch.randn(pools.t[n].shape, generator=g).to(ref.TYPES[kind]))
    pools.before = {n: x.clone() for n, x in pools.t.items()}
    q, k, v = (x.cpu() for x in rows)
    freqs, f = table(rot, 500000.0)
    err = word()
    out = step(pools, rows, slots, pos, freqs, tbl, i32(lens), scale, window, ring, inter, m, err)
    assert int(err.item()) == 0
    slots, pos = slots.cpu().numpy(), pos.cpu().numpy()
    pools.check(k, v, slots, pos, f, inter, m, kind)
    q64, e = ref.rotate(ref.as_values(q), np.maximum(pos, 0)[:, None], f, inter, m)
    q64, dq = rounded(q64, e, q.dtype)
    kv = [held(pools, n) for n in "kv"]
    got, tbl = out.double().cpu().numpy(), tbl.cpu().numpy()
    by_length = np.argsort(lens, kind="stable")
    some = range(len(lens)) if len(lens) < 10 else {0, 1, *by_length[:2], *by_length[-2:]}
    for b in some:
        n = lens[b]
        if n == 0:
            assert (got[b] == 0).all()
            continue
        at = np.arange(max(0, n - window) if window else 0, n)
        block = at // ps % ring if ring else at // ps
        there = tbl[b, block].astype(np.int64) * ps + at % ps
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            want, more = attention(q64[b, heads], dq[b, heads], kv[0][there, h], kv[1][there, h],
                                   scale)
            off = np.abs(got[b, heads] - want) - more
            assert (off <= parity.ABS_TOL).all(), (b, h, off.max())
            rel = off / np.maximum(np.abs(want), parity.REL_FLOOR)
            assert (rel <= parity.REL_TOL).all(), (b, h, rel.max())
