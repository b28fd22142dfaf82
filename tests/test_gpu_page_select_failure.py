"""The page scores' kernel with a wait that runs out, made without a fault: a
separate build in which the first stage of one CTA expects 16 bytes that no
copy delivers (every copy it does issue lands) and the wait bound is about 16
ms.  The call returns, the error word tells, and the context stays usable.
The product library has neither setting."""
import ctypes
import time

import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import _lib, build
from tests import long_context_ref as ref

pytestmark = pytest.mark.gpu


def test_a_wait_for_page_codes_that_runs_out_sets_the_timeout_bit():
    path = build.build_variant("stall_page_scores", ["api.cu", "page_select.cu"],
                               ["TL_TEST_STALL_FIRST_STAGE=1", "TL_WAIT_CYCLES=(1ll<<25)"])
    lib = ctypes.CDLL(path)
    for name in ("tl_kv_page_select", "tl_get_device_error"):
        getattr(lib, name).argtypes, getattr(lib, name).restype = _lib.SIGNATURES[name]
    lens = [3000, 500]
    table, P = ref.tables(lens, 16, seed=1)
    g = torch.Generator().manual_seed(2)
    hi = torch.randint(0, 128, (P, 2, 128), generator=g)
    bnd = torch.stack((hi, -hi), 2).to(torch.int8)
    sc = torch.rand((P, 2), generator=g)
    q = torch.randn((2, 8, 128), generator=g).bfloat16()
    d = [x.cuda() for x in (q, bnd, sc, table)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pages = torch.zeros((2, 2, 10), dtype=torch.int32, device="cuda")
    got = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = tl.alloc_workspace(tl.tl_kv_page_select_workspace_size(2, 8, 2, 128, table.shape[1]), "cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    t0 = time.time()
    st = lib.tl_kv_page_select(d[0].data_ptr(), tl.TL_BF16, d[1].data_ptr(), d[2].data_ptr(),
                               d[3].data_ptr(), table.shape[1], ln.data_ptr(), 10, 0, 1,
                               pages.data_ptr(), got.data_ptr(), 2, 8, 2, 128, P, 16,
                               ws.data_ptr(), ws.numel(), err.data_ptr(), stream)
    assert st == tl.TL_OK
    bits = ctypes.c_uint32(0)
    st = lib.tl_get_device_error(err.data_ptr(), ctypes.byref(bits), 0, stream)
    assert time.time() - t0 < 30.0  # the bounded waits ended the kernel
    assert st == tl.TL_ERR_DEVICE_TIMEOUT and bits.value & tl.TL_DEVERR_TIMEOUT
    # the context is still usable: the product library selects as it should
    pages, got = tl.tl_kv_page_select(d[0], d[1], d[2], d[3], ln, 16, 10)
    want_t, want_l = ref.page_select(q, bnd, sc, table, lens, 16, 10, 0, 1, P)
    assert torch.equal(pages.cpu(), want_t) and torch.equal(got.cpu(), want_l)
