"""The buffers that a call allocates for itself (outputs and workspaces that were not given)
belong to the stream it runs on: with a stream passed while another one is current, no later
allocation may get a block that the call's kernels still use."""
import contextlib
import types

import pytest
import torch

import paged_kv_attention_cache_gb300 as tl
from paged_kv_attention_cache_gb300 import api, build

B, HQ, HKV, D, P, PS, W, T = 2, 8, 2, 128, 6, 16, 3, 2
BF, I8, I32, F32 = torch.bfloat16, torch.int8, torch.int32, torch.float32


def inputs(device):
    g = torch.Generator().manual_seed(1)
    c = dict(q=torch.randn((B, HQ, D), generator=g).to(BF),
             qt=torch.randn((B, T, HQ, D), generator=g).to(BF),
             k=torch.randn((P, PS, HKV, D), generator=g).to(BF),
             v=torch.randn((P, PS, HKV, D), generator=g).to(BF),
             kc=torch.randint(-127, 128, (P, PS, HKV, D), generator=g, dtype=I8),
             vc=torch.randint(-127, 128, (P, PS, HKV, D), generator=g, dtype=I8),
             ks=torch.rand((P, HKV, PS), generator=g) * 0.04,
             vs=torch.rand((P, HKV, PS), generator=g) * 0.04,
             kn=torch.randn((B, HKV, D), generator=g).to(BF),
             vn=torch.randn((B, HKV, D), generator=g).to(BF),
             slots=torch.tensor([39, 5 * PS + 14], dtype=torch.int64),
             table=torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=I32),
             lens=torch.tensor([40, 47], dtype=I32),
             positions=torch.tensor([[38, 39], [45, 46]], dtype=I32),
             bounds=torch.randint(0, 128, (P, HKV, 2, D), generator=g, dtype=I8),
             bscales=torch.rand((P, HKV), generator=g),
             pages=torch.tensor([[[0, 2], [1, 2]], [[3, 5], [4, 5]]], dtype=I32),
             plens=torch.tensor([24, 31], dtype=I32),
             mass=torch.rand((B, HKV, 48), generator=g))
    c["bounds"][:, :, 1] *= -1
    return types.SimpleNamespace(**{n: x.to(device) for n, x in c.items()})


# every call that allocates, with neither an output nor a workspace given, and how many buffers
CALLS = {
    "decode": (2, lambda c, s: tl.tl_paged_attn_decode(c.q, c.k, c.v, c.table, c.lens, 0.1,
                                                       stream=s)),
    "decode_int8": (2, lambda c, s: tl.tl_paged_attn_decode_int8(
        c.q, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, 0.1, stream=s)),
    "decode_write": (2, lambda c, s: tl.tl_paged_attn_decode_write(
        c.q, c.kn, c.vn, c.slots, c.k, c.v, c.table, c.lens, 0.1, stream=s)),
    "decode_write_int8": (2, lambda c, s: tl.tl_paged_attn_decode_write_int8(
        c.q, c.kn, c.vn, c.slots, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, 0.1, stream=s)),
    "decode_multi": (2, lambda c, s: tl.tl_paged_attn_decode_multi(
        c.qt, c.k, c.v, c.table, c.lens, 0.1, stream=s)),
    "decode_multi_int8": (2, lambda c, s: tl.tl_paged_attn_decode_multi_int8(
        c.qt, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, 0.1, stream=s)),
    "decode_ring": (2, lambda c, s: tl.tl_paged_attn_decode_ring(
        c.q, c.k, c.v, c.table, c.lens, 0.1, window=20, ring_pages=W, stream=s)),
    "decode_ring_int8": (2, lambda c, s: tl.tl_paged_attn_decode_ring_int8(
        c.q, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, 0.1, window=20, ring_pages=W, stream=s)),
    "decode_write_ring": (2, lambda c, s: tl.tl_paged_attn_decode_write_ring(
        c.q, c.kn, c.vn, c.slots, c.k, c.v, c.table, c.lens, 0.1, window=20, ring_pages=W,
        stream=s)),
    "prefill": (2, lambda c, s: tl.tl_paged_attn_prefill(c.qt, c.k, c.v, c.table, c.positions, 0.1,
                                                         stream=s)),
    "prefill_int8": (2, lambda c, s: tl.tl_paged_attn_prefill_int8(
        c.qt, c.kc, c.vc, c.ks, c.vs, c.table, c.positions, 0.1, stream=s)),
    "prefill_ring": (2, lambda c, s: tl.tl_paged_attn_prefill_ring(
        c.qt, c.k, c.v, c.table, c.positions, 0.1, window=20, ring_pages=W, stream=s)),
    "prefill_ring_int8": (2, lambda c, s: tl.tl_paged_attn_prefill_ring_int8(
        c.qt, c.kc, c.vc, c.ks, c.vs, c.table, c.positions, 0.1, window=20, ring_pages=W,
        stream=s)),
    "page_select": (3, lambda c, s: tl.tl_kv_page_select(
        c.q, c.bounds, c.bscales, c.table, c.lens, PS, 2, stream=s)),
    "decode_pages": (2, lambda c, s: tl.tl_paged_attn_decode_pages(
        c.q, c.k, c.v, c.pages, c.plens, 0.1, stream=s)),
    "decode_pages_int8": (2, lambda c, s: tl.tl_paged_attn_decode_pages_int8(
        c.q, c.kc, c.vc, c.ks, c.vs, c.pages, c.plens, 0.1, stream=s)),
    "decode_mass": (2, lambda c, s: tl.tl_paged_attn_decode_mass(
        c.qt, c.k, c.v, c.table, c.lens, c.mass, 0.1, stream=s)),
    "decode_mass_int8": (2, lambda c, s: tl.tl_paged_attn_decode_mass_int8(
        c.qt, c.kc, c.vc, c.ks, c.vs, c.table, c.lens, c.mass, 0.1, stream=s)),
    "evict_select": (2, lambda c, s: tl.tl_kv_evict_select(c.mass, c.lens, 8, stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_buffers_are_allocated_on_the_calls_stream(name, monkeypatch):
    """The binding alone, on the CPU: checks and launch replaced, allocations watched."""
    build.build()
    side, current, on, made, kept = object(), object(), [None], [], []

    @contextlib.contextmanager
    def stream(s):
        before, on[0] = on[0], s
        yield
        on[0] = before

    empty = torch.empty
    monkeypatch.setattr(api, "_need", lambda *a, **k: None)
    monkeypatch.setattr(api, "_run", lambda *a: None)
    monkeypatch.setattr(api, "_alloc_stream", lambda s, d: s, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (made.append(on[0]), empty(*a, **k))[1])
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: kept.append((t.data_ptr(), s)))
    buffers, call = CALLS[name]
    c = inputs("cpu")
    del made[:]
    got = call(c, side)
    assert made == [side] * buffers
    # what is returned is used on the current stream too
    got = got if isinstance(got, tuple) else (got,)
    assert sorted(kept) == sorted((t.data_ptr(), current) for t in got)
    del made[:], kept[:]
    call(c, None)
    assert made == [None] * buffers and not kept


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_stream_that_is_not_current(name, handle, monkeypatch):
    """Its kernels wait behind other work of the side stream; meanwhile the current stream
    allocates blocks of the workspace's and the output's sizes and gets others."""
    build.build()
    _, call = CALLS[name]
    c = inputs("cuda")
    first = call(c, None)  # the module's kernels are loaded
    first = [t.clone() for t in (first if isinstance(first, tuple) else (first,))]
    torch.cuda.synchronize()
    sizes = []
    alloc = api.alloc_workspace
    monkeypatch.setattr(api, "alloc_workspace", lambda n, d: sizes.append(alloc(n, d)) or sizes[-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 200 ms
    c2 = inputs("cuda") if "write" in name or "mass" in name else c
    side.wait_stream(torch.cuda.current_stream())
    got = call(c2, side.cuda_stream if handle else side)
    used = [(w.data_ptr(), w.numel()) for w in sizes]
    del sizes[:]  # the call's own reference is gone too: its block may be reused
    later = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in used for _ in range(3)]
    got = got if isinstance(got, tuple) else (got,)
    later += [torch.empty_like(t) for t in got for _ in range(3)]
    assert not side.query()  # still behind the wait
    own = [p for p, _ in used] + [t.data_ptr() for t in got]
    assert not set(own) & {t.data_ptr() for t in later}
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, first):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_passed_stream_inside_a_capture():
    """A step captured with a forked stream passed to its calls, replayed over new inputs."""
    build.build()
    c = inputs("cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step(stream):
        pages, lens = tl.tl_kv_page_select(c.q, c.bounds, c.bscales, c.table, c.lens, PS, 2,
                                           stream=stream)
        return tl.tl_paged_attn_decode_pages(c.q, c.k, c.v, pages, lens, 0.1, stream=stream)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step(None)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            side.wait_stream(main)
            step(side)  # its buffers are dropped inside the capture
            out = step(side)
            main.wait_stream(side)
    torch.cuda.synchronize()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        c.q.copy_(torch.randn((B, HQ, D), generator=g).to(BF))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(None))
