"""int8 pools whose V scales say nothing about the weights: the keys that carry an output may have
the smallest scales of the sequence.  The decode forms over selected pages and with weights multiply
each weight by its key's V scale and hold the product in two fp16 parts; a part is off by at most
2^-25, so what the product is brought to first decides which keys are lost.  The outputs are held to
the largest product p_j x scale_j of their own row: no key with a scale that its weight does not
earn may cost a row its digits."""
import numpy as np
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as ref

pytestmark = pytest.mark.gpu

PS, HKV, D = 16, 2, 128
LENS = [700, 40, 1500]


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def case(order, R, rows, seed):
    """Pools, table and queries with chosen scores: query row r is the unit vector of channel r, so
    its score with a key is the key's code there times 1/4, exactly.  Each row has keys of weight
    (code 100) and keys of next to none (code -10: e^-27.5 of the others)."""
    table, P = ref.tables(LENS, PS, seed=seed)
    pools = ref.Pools("int8", P, PS, HKV, D, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    pools.data["k"] = torch.zeros((P, PS, HKV, D), dtype=torch.int8)
    pools.scales["k"] = torch.full((P, HKV, PS), 0.25)
    vscale = torch.rand((P, HKV, PS), generator=g) * 0.045 + 0.005
    for b, n in enumerate(LENS):
        j = torch.arange(n)
        big = {"first": j < n // 2, "last": j >= n // 2, "mixed": j % 3 == 1, "one": j == n // 3,
               "by row": j % 2 == 1, "base moves": j < n // 2}[order]
        pg, at = table[b, j // PS].long(), j % PS
        code = torch.where(big, -10, 100)
        for r in range(rows):
            c = code + torch.randint(-6, 7, (n,), generator=g)
            if order == "by row" and r % 2 == 1:  # the other rows weigh the keys of large scales
                c = torch.where(big, 100, -10) + torch.randint(-6, 7, (n,), generator=g)
            if order == "base moves":  # scores that rise along the sequence, in steps
                c = torch.where(big, -127 + 220 * (j // 64 * 64) // n, code)
            for h in range(HKV):
                pools.data["k"][pg, at, h, r] = c.to(torch.int8)
        vscale[pg[big], :, at[big]] *= 2.0 ** R
    pools.scales["v"] = vscale
    q = torch.zeros((len(LENS), HKV, rows, D))
    for r in range(rows):
        q[:, :, r, r] = 1
    return pools, table, P, q


def check(out, weights_of, pools, table, q, T, what):
    """out [B, T, HKV, group, D]."""
    k, v = pools.values("k").double().numpy(), pools.values("v").double().numpy()
    codes = pools.data["v"].double().abs().numpy()
    vs = pools.scales["v"].double().numpy()
    group = q.shape[2] // T
    for b, n in enumerate(LENS):
        pg = table[b, :-(-n // PS)].long().numpy()
        for g in range(HKV):
            kk, vv = (x[pg][:, :, g].reshape(-1, D)[:n] for x in (k, v))
            cc, sc = codes[pg][:, :, g].reshape(-1, D)[:n], vs[pg][:, g].reshape(-1)[:n]
            for t in range(T):
                rows = slice(t * group, (t + 1) * group)
                sees = np.broadcast_to(np.arange(n) <= n - T + t, (group, n))
                qq = q[b, g, rows].double().numpy()
                p, o, mag = ref.attend(qq, kk, vv, 1.0, sees)
                # A score is exact up to its change to log2 units (two roundings) and the
                # difference from the base (one): 3 x 2^-24 of twice the largest, 32; it counts
                # twice, in the weight and in the sum.  The exponentials 2^-21 twice, two products
                # with scale and fit 2^-23, the parts 2^-21, the sums n + 8 roundings.
                rel = 2 * 3 * 2.0 ** -24 * 64 + 3 * 2.0 ** -21 + 2.0 ** -23 + (n + 8) * 2.0 ** -23
                # a product below 2^-14 of fp16 range is off by 2^-25 where the row's largest is at
                # least 2^8
                top = (p * sc).max(1)[:, None]
                tol = rel * mag + 2.0 ** -33 * top * cc.sum(0) + 1e-30
                ref.assert_within(out[b, t, g], o, tol, f"{what} b{b} g{g} t{t}")


ORDERS = ["first", "last", "mixed", "one", "by row", "base moves"]


@pytest.mark.parametrize("R", [10, 16, 20, 30])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("group,T", [(1, 1), (4, 1), (5, 1), (3, 2), (16, 1), (4, 4)])
def test_weights_with_unearned_scales(group, T, order, R):
    pools, table, P, q = case(order, R, group * T, seed=7)
    p = pools.gpu()
    # [B, HKV, T * group, D] -> [B, T, HKV * group, D]
    qq = q.view(len(LENS), HKV, T, group, D).transpose(1, 2).reshape(len(LENS), T, HKV * group, D)
    qq = qq.bfloat16().cuda().contiguous()
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    mass = torch.zeros((len(LENS), HKV, 1500), device="cuda")
    out = tl.tl_paged_attn_decode_mass_int8(qq, p["k"], p["v"], p["ks"], p["vs"], table.cuda(), lens,
                                            mass, 1.0)
    check(out.view(len(LENS), T, HKV, group, D), None, pools, table, q, T, f"{order} 2^{R}")
    if T == 1:
        pages = table[:, None].expand(-1, HKV, -1).contiguous().cuda()
        out = tl.tl_paged_attn_decode_pages_int8(qq[:, 0].contiguous(), p["k"], p["v"], p["ks"],
                                                 p["vs"], pages, lens, 1.0)
        check(out.view(len(LENS), 1, HKV, group, D), None, pools, table, q, 1, f"pages {order} 2^{R}")


@pytest.mark.parametrize("power", [-120, -100, 100, 118])
@pytest.mark.parametrize("group", [4, 16])
def test_scales_near_the_ends_of_the_range(group, power):
    """Every scale times a power of two: the outputs times it, as far as f32 holds them."""
    pools, table, P, q = case("mixed", 0, group, seed=9)
    p = pools.gpu()
    qq = q.reshape(len(LENS), HKV * group, D).bfloat16().cuda()
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    pages = table[:, None].expand(-1, HKV, -1).contiguous().cuda()

    def run(vs):
        return tl.tl_paged_attn_decode_pages_int8(qq, p["k"], p["v"], p["ks"], vs, pages, lens, 1.0)

    f = 2.0 ** power
    one, far = run(p["vs"]).double().cpu(), run(p["vs"] * f).double().cpu()
    assert torch.isfinite(far).all()
    # below 2^-118 the largest product cannot be brought to 2^8 (the factor ends at 2^126): parts of
    # 2^-25 over a product of at least 2^(126 - 120 - 8) x e^-3
    slack = 2.0 ** -25 * 2.0 ** -2 * 1e3 if power < -110 else 0.0
    assert torch.allclose(far / f, one, rtol=2.0 ** -20, atol=slack + 2.0 ** -149 / f)
