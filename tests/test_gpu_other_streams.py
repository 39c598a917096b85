"""Buffers that a call makes itself, on a stream that is not the current one: torch hands freed memory out again in the
order of the stream it was taken on, so they have to be that stream's."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R
from test_gpu_decode_q4 import Case, _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Recorder:
    """The library with every call that takes device pointers noted down instead of made."""
    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name.endswith("workspace_size") or name == "pa_status_string":
            return fn

        def call(*args):
            self.calls.append((name, args))
            return pa.OK
        return call


def stream_kinds(s):
    return {"stream": s, "handle": s.cuda_stream}


def small():
    """Arguments of one call of each kind (two sequences, 4 / 2 heads of 128, blocks of 16)."""
    i32 = dict(dtype=torch.int32, device=DEV)
    S, H, Hkv, D, B, nb = 2, 4, 2, 128, 16, 4
    z = dict(bt=torch.arange(nb, **i32).view(S, 2), ctx=torch.full((S,), 20, **i32), start=torch.full((S,), 19, **i32),
             cu=torch.arange(S + 1, **i32), slot=torch.tensor([20, 50], device=DEV), pos=torch.full((S,), 19, **i32))
    z["q"] = torch.randn(S, H, D, device=DEV).bfloat16()
    z["kv"] = torch.randn(S, Hkv, D, device=DEV).bfloat16()
    z["k"], z["v"] = (torch.randn(nb, B, Hkv, D, device=DEV).bfloat16() for _ in "kv")
    z["k4"], z["v4"] = (R.new_pool(nb, B, Hkv, D, DEV, fill=0x11) for _ in "kv")
    z["tab"] = R.table(64, D).to(DEV)
    return z


NEW = {
    "decode_q4": lambda z, **kw: [pa.decode_q4(z["q"], z["k4"], z["v4"], z["bt"], z["ctx"], 0.1, **kw)],
    "rope_and_cache": lambda z, **kw: [pa.rope_and_cache(z["q"], z["kv"], z["kv"], z["tab"], z["pos"], z["k"], z["v"],
                                                         z["slot"], **kw)],
    "rope_and_cache_q4": lambda z, **kw: [pa.rope_and_cache_q4(z["q"], z["kv"], z["kv"], z["tab"], z["pos"], z["k4"],
                                                               z["v4"], z["slot"], **kw)],
}
OLD = {
    "compute_slot_mapping": lambda z, **kw: [pa.compute_slot_mapping(z["bt"], z["start"], z["cu"], 4, 2, **kw)],
    "decode": lambda z, **kw: [pa.decode(z["q"], z["k"], z["v"], z["bt"], z["ctx"], 0.1, **kw)],
    "decode_step": lambda z, **kw: list(pa.decode_step(z["q"], z["kv"], z["kv"], z["k"], z["v"], z["bt"], z["ctx"],
                                                       z["start"], z["cu"], 0.1, **kw)),
    "varlen_prefill": lambda z, **kw: [pa.varlen_prefill(z["q"], z["cu"], z["k"], z["v"], z["bt"], z["ctx"], 0.1, 1, **kw)],
    "varlen_step": lambda z, **kw: list(pa.varlen_step(z["q"], z["kv"], z["kv"], z["k"], z["v"], z["cu"], z["bt"], z["ctx"],
                                                       z["start"], 0.1, 1, **kw)),
}
CALLS = {**NEW, **OLD}


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", list(CALLS))
def test_memory_given_back_is_not_handed_out_on_the_current_stream(name, kind, monkeypatch):
    """Nothing is launched here: the pointers of the call are noted, and none of those it made itself may come back
    from the current stream's part of the allocator while the other stream could still be at work on them."""
    z = small()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    rec = Recorder(pa.load())
    monkeypatch.setattr(pa, "_lib", rec)
    made = CALLS[name](z, stream=stream_kinds(s)[kind])
    (called, args), = rec.calls
    assert args[-1] == s.cuda_stream
    given = [t.data_ptr() for t in z.values()]
    mine = {p for p in args if isinstance(p, int) and p > 1 << 32 and p not in given and p != s.cuda_stream}
    sizes = {t.numel() * t.element_size() for t in made}
    assert mine >= {t.data_ptr() for t in made}
    del made
    if "decode" in name or "varlen" in name:
        sizes |= {pa.decode_workspace_size(2, 4, 2, 128, 16, 2), pa.decode_q4_workspace_size(2, 4, 2, 128, 16, 2),
                  pa.varlen_prefill_workspace_size(2, 2, 4, 2, 128, 16, 2)}
        assert len(mine) >= 2
    again = [torch.empty(max(n, 16), dtype=torch.uint8, device=DEV) for n in sorted(sizes) for _ in range(4)]
    assert not mine & {t.data_ptr() for t in again}


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", list(CALLS))
def test_calls_on_another_stream_give_the_same(name, kind):
    z = small()
    want = CALLS[name](z)
    z2 = {k: t.clone() for k, t in z.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = CALLS[name](z2, stream=stream_kinds(s)[kind])
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handle(handle):
    """0 and 1 name the device's default stream; here another one is current."""
    c = Case([700, 20, 5], 8, 2, 128, 16, torch.bfloat16, seed=91)
    ref = c.run()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_two_streams_with_the_calls_own_buffers():
    cs = [Case([3000, 17, 900], 8, 2, 128, 16, torch.bfloat16, seed=92 + i) for i in range(2)]
    refs = [c.run() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale, stream=s) for c, s in zip(cs, streams)]
        other = torch.full((8 << 20,), 3, dtype=torch.uint8, device=DEV)   # the current stream's memory, meanwhile
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)
        del outs, other
    torch.cuda.synchronize()


def test_a_captured_call_on_a_forked_stream():
    """Inside a capture, a call on a stream forked from the captured one, with its own buffers."""
    c = Case([700, 20, 5], 8, 2, 128, 16, torch.bfloat16, seed=95)
    ref = c.run()
    s, fork = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fork.wait_stream(torch.cuda.current_stream())
        out = pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale, stream=fork)
        torch.cuda.current_stream().wait_stream(fork)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
