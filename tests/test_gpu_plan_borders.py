"""Batches on both sides of the sizes at which the decode forms with weights and over selected pages
go from planning in their own blocks to a plan launch: the same answers."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build
from tests import long_context_ref as ref
from tests.test_gpu_evict import check_mass, run_mass

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


@pytest.mark.parametrize("kind,T,B,hkv", [
    ("bf16", 1, 24, 8), ("bf16", 1, 25, 8), ("bf16", 1, 12, 16), ("bf16", 1, 13, 16),
    ("bf16", 1, 32, 6), ("bf16", 1, 33, 2), ("bf16", 6, 32, 8), ("bf16", 6, 17, 16),
    ("e4m3", 1, 64, 8), ("e4m3", 1, 65, 8), ("int8", 6, 64, 3), ("int8", 6, 65, 3)])
def test_both_sides_of_the_rule(kind, T, B, hkv):
    lens = [(97 * b) % 700 for b in range(B)]
    lens[B // 2] = 2500
    table, P = ref.tables(lens, 16, seed=1)
    pools = ref.Pools(kind, P, 16, hkv, 128, seed=2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((B, T, 2 * hkv, 128), generator=g).bfloat16()
    mass0 = torch.rand((B, hkv, 2500), generator=g)
    mass = mass0.cuda()
    scale = ref.default_scale(128)
    p = pools.gpu()
    out = run_mass(pools, q, table, lens, mass, scale, p=p)
    check_mass(out, mass, mass0, pools, q, table, lens, scale, 0, f"{kind} b{B}")
    if T == 1:  # the whole sequence as its selected pages
        pages = table[:, None].expand(-1, hkv, -1).contiguous().cuda()
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        whole = (tl.tl_paged_attn_decode_pages_int8 if kind == "int8" else
                 tl.tl_paged_attn_decode_pages)
        scales = (p["ks"], p["vs"]) if kind == "int8" else ()
        same = whole(q[:, 0].cuda(), p["k"], p["v"], *scales, pages, n, scale)
        check_mass(same[:, None], mass, mass0, pools, q, table, lens, scale, 0, f"pages {kind}")
