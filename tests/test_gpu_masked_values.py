"""Keys that a window masks may hold anything: NaN and infinities in their K and V rows, in the very
16-key chunk that the window starts in, leave the outputs and weights as zeros there would."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


@pytest.mark.parametrize("kind,d,ps", [("bf16", 128, 16), ("bf16", 64, 8), ("bf16", 128, 24),
                                       ("e4m3", 128, 16), ("e4m3", 128, 8), ("f32", 128, 16)])
@pytest.mark.parametrize("group,T", [(4, 1), (5, 1), (16, 1), (2, 3)])
@pytest.mark.parametrize("call", ["decode", "mass"])
def test_what_lies_before_the_window(kind, d, ps, group, T, call):
    if kind == "f32" and T > 1:
        pytest.skip("f32 pools take one token")
    lens, window, hkv = [3, 41, 100, 333, 2000], 37, 2
    table, P = ref.tables(lens, ps, seed=1)
    pools = ref.Pools(kind, P, ps, hkv, d, seed=2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((len(lens), T, hkv * group, d), generator=g)
    q = (q if kind == "f32" else q.bfloat16()).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run():
        p = pools.gpu()
        mass = torch.zeros((len(lens), hkv, 2000), device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if call == "mass":
            out = tl.tl_paged_attn_decode_mass(q, p["k"], p["v"], table.cuda(), n, mass, 0.1,
                                               window=window, error_word=err)
        elif T == 1:
            out = tl.tl_paged_attn_decode(q[:, 0].contiguous(), p["k"], p["v"], table.cuda(), n,
                                          0.1, window=window, error_word=err)
        else:
            out = tl.tl_paged_attn_decode_multi(q, p["k"], p["v"], table.cuda(), n, 0.1,
                                                window=window, error_word=err)
        assert int(err.item()) == 0
        return out, mass

    seen = torch.zeros((P, ps), dtype=torch.bool)
    for b, L in enumerate(lens):
        for j in range(max(0, L - T - window + 1), L):
            seen[table[b, j // ps], j % ps] = True
    for x in pools.data.values():
        x.view(torch.uint8 if kind == "e4m3" else x.dtype)[~seen] = 0
    want = run()
    assert torch.isfinite(want[0]).all()
    pools.poison(seen)
    got = run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if kind != "e4m3":
        for x in pools.data.values():
            x[~seen] = float("inf")
        got = run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
