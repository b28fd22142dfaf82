"""The rotary calls' own buffers belong to the stream they run on, as test_call_buffers.py checks
for the other calls."""
import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from tests import test_call_buffers as base


def freqs(c):
    return torch.arange(1, 65, device=c.q.device) << 50


def now(c):
    return c.lens - 1


CALLS = {
    "rope": (1, lambda c, s: tl.tl_rope(c.q, now(c), freqs(c), stream=s)),
    "write_rope": (1, lambda c, s: tl.tl_kv_cache_write_rope(
        c.q, c.kn, c.vn, c.k, c.v, c.slots, now(c), freqs(c), stream=s)),
    "write_rope_int8": (1, lambda c, s: tl.tl_kv_cache_write_rope_int8(
        c.q, c.kn, c.vn, c.kc, c.vc, c.ks, c.vs, c.slots, now(c), freqs(c), stream=s)),
    "decode_write_rope": (2, lambda c, s: tl.tl_paged_attn_decode_write_rope(
        c.q, c.kn, c.vn, c.slots, now(c), freqs(c), c.k, c.v, c.table, c.lens, 0.1, stream=s)),
    "decode_write_rope_int8": (2, lambda c, s: tl.tl_paged_attn_decode_write_rope_int8(
        c.q, c.kn, c.vn, c.slots, now(c), freqs(c), c.kc, c.vc, c.ks, c.vs, c.table, c.lens, 0.1,
        stream=s)),
    "decode_write_rope_ring": (2, lambda c, s: tl.tl_paged_attn_decode_write_rope_ring(
        c.q, c.kn, c.vn, c.slots, now(c), freqs(c), c.k, c.v, c.table, c.lens, 0.1, window=20,
        ring_pages=base.W, stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_buffers_are_allocated_on_the_calls_stream(name, monkeypatch):
    monkeypatch.setitem(base.CALLS, name, CALLS[name])
    monkeypatch.setattr(tl.api, "_need_rows", lambda t, *a, **k: t.stride(0))
    base.test_own_buffers_are_allocated_on_the_calls_stream(name, monkeypatch)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_stream_that_is_not_current(name, handle, monkeypatch):
    monkeypatch.setitem(base.CALLS, name, CALLS[name])
    # (the arguments made on the current stream are kept until the wait is over)
    kept = []
    for maker in ("now", "freqs"):
        f = globals()[maker]
        monkeypatch.setitem(globals(), maker, lambda c, f=f: kept.append(f(c)) or kept[-1])
    base.test_a_call_on_a_stream_that_is_not_current(name, handle, monkeypatch)
