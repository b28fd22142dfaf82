"""Lengths at the end of the 32-bit positions.  A decode stage covers 32 keys from a chunk's start,
so within 32 of 2^31 its last position would wrap: such lengths are reported and read nothing."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("L", [2**31 - 1, 2**31 - 16, 2**31 - 63])
def test_a_length_whose_last_stage_would_wrap(kind, L):
    build.build()
    ps, n = 256, 2**31 // 256
    g = torch.Generator().manual_seed(1)
    q = torch.randn((2, 4, 128), generator=g).bfloat16().cuda()
    lens = torch.tensor([L, 300], dtype=torch.int32, device="cuda")
    pages = torch.zeros((2, 1, n), dtype=torch.int32, device="cuda")  # one page, again and again
    if kind == "int8":
        k, v = (torch.randint(-127, 128, (2, ps, 1, 128), generator=g, dtype=torch.int8).cuda()
                for _ in range(2))
        sc = tuple(torch.rand((2, 1, ps), generator=g).cuda() * 0.02 for _ in range(2))
        calls = (tl.tl_paged_attn_decode_pages_int8, tl.tl_paged_attn_decode_int8)
    else:
        k, v = (torch.randn((2, ps, 1, 128), generator=g).bfloat16().cuda() for _ in range(2))
        sc = ()
        calls = (tl.tl_paged_attn_decode_pages, tl.tl_paged_attn_decode)
    for call, table in zip(calls, (pages, pages.view(2, n))):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((2, 4, 128), 7.0, device="cuda")
        call(q, k, v, *sc, table, lens, 0.1, out=out, error_word=err)
        assert int(err.item()) == tl.TL_DEVERR_CONTEXT_RANGE
        assert torch.all(out[0] == 0)
        err.zero_()
        alone = call(q[1:], k, v, *sc, table[1:, ..., :2].contiguous(), lens[1:], 0.1,
                     error_word=err)
        assert int(err.item()) == 0 and torch.allclose(out[1], alone[0], rtol=0, atol=1e-5)
