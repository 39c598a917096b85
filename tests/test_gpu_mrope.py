"""The rotary cache writes with several position axes: against the formula in 64 bits, and bit for bit against the call
with one position a token over a table made for the purpose (row t holds what token t's axes look up)."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R
from test_gpu_rope_q4 import DEV, SHAPES, _lib, bits, check_rows, inputs  # noqa: F401  (_lib builds the library)

pytestmark = pytest.mark.gpu


def axes_of(R_, A, layout, seed):
    """The axis of every pair: sections, taking turns, or any."""
    i = np.arange(R_)
    if layout == "sections":
        return np.minimum(i * (A + 1) // max(R_, 1), A - 1).astype(np.int32)
    if layout == "turns":
        return (i % A).astype(np.int32)
    return np.random.default_rng(seed).integers(0, A, R_).astype(np.int32)


class Case:
    def __init__(self, n, H, Hkv, D, rot, B, dtype, A, layout="sections", rows="fused", seed=0, max_pos=5000, stride=0):
        rng = np.random.default_rng(seed)
        self.n, self.H, self.Hkv, self.D, self.rot, self.B, self.dtype = n, H, Hkv, D, rot, B, dtype
        self.q, self.k, self.v = inputs(n, H, Hkv, D, dtype, rows, seed + 1)
        self.nb = -(-(n + 7) // B) + 2
        self.slots = torch.from_numpy(rng.permutation(self.nb * B)[:n].astype(np.int64)).to(DEV)
        pos = rng.integers(0, max_pos, size=(A, n + stride)).astype(np.int32)
        pos[0, 0], pos[A - 1, n - 1] = max_pos - 1, 0
        self.pos = torch.from_numpy(pos).to(DEV)[:, :n]      # a view of a wider buffer when stride > 0
        self.axis = torch.from_numpy(axes_of(rot // 2, A, layout, seed)).to(DEV)
        self.tab = R.table(max_pos, rot).to(DEV)

    def pools(self, q4, fill=5.0):
        if q4:
            return tuple(R.new_pool(self.nb, self.B, self.Hkv, self.D, DEV, seed=s) for s in (1, 2))
        return tuple(torch.full((self.nb, self.B, self.Hkv, self.D), fill, dtype=self.dtype, device=DEV) for _ in "kv")

    def own_table(self):
        """[n, rot]: the cosines and sines that each token's axes look up."""
        i = np.arange(self.rot // 2)
        p = self.pos.cpu().numpy()[self.axis.cpu().numpy()].T
        t = self.tab.cpu().numpy()
        return torch.from_numpy(np.ascontiguousarray(np.concatenate([t[p, i], t[p, self.rot // 2 + i]], 1))).to(DEV)

    def run(self, q4, inter, **kw):
        """(bytes of q_out and of both pools, status) of the call under test."""
        kc, vc = self.pools(q4)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full((self.n, self.H, self.D), 9.0, dtype=self.dtype, device=DEV)
        a = dict(q=self.q, key=self.k, value=self.v, cos_sin=self.tab, positions=self.pos, pair_axis=self.axis,
                 slot_mapping=self.slots, interleaved=inter, q_out=out, dev_status=st)
        (pa.mrope_and_cache_q4 if q4 else pa.mrope_and_cache)(k_cache=kc, v_cache=vc, **{**a, **kw})
        return [t.view(torch.uint8) for t in (out, kc, vc)], pa.get_device_status(st)

    def run_one_axis(self, q4, inter, skip=()):
        kc, vc = self.pools(q4)
        out = torch.full((self.n, self.H, self.D), 9.0, dtype=self.dtype, device=DEV)
        slots = self.slots.clone()
        slots[list(skip)] = -1
        (pa.rope_and_cache_q4 if q4 else pa.rope_and_cache)(
            self.q, self.k, self.v, self.own_table(), torch.arange(self.n, dtype=torch.int32, device=DEV), kc, vc, slots,
            interleaved=inter, q_out=out)
        return [t.view(torch.uint8) for t in (out, kc, vc)]


def same(got, want):
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("A,layout", [(3, "sections"), (3, "turns"), (2, "any"), (4, "any"), (1, "any")])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[4] and s[1]], ids=str)
def test_mrope_and_cache(shape, A, layout, dtype):
    n, H, Hkv, D, rot, inter, B, rows = shape
    c = Case(n, H, Hkv, D, rot, B, dtype, A, layout, rows, seed=n + A, stride=3)
    got, status = c.run(False, inter)
    assert status == 0
    tok = np.arange(n)
    check_rows(got[0].view(dtype), *R.rotate(c.q, c.own_table(), tok, rot, inter), dtype, "q_out")
    kc = got[1].view(dtype).cpu().reshape(-1, Hkv, D)
    check_rows(kc[c.slots.cpu()], *R.rotate(c.k, c.own_table(), tok, rot, inter), dtype, "k_cache")
    same(got, c.run_one_axis(False, inter))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("A,layout", [(3, "sections"), (4, "any")])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] in (64, 128) and s[6] in (8, 16, 32) and s[4] and s[1]], ids=str)
def test_mrope_and_cache_q4(shape, A, layout, dtype):
    n, H, Hkv, D, rot, inter, B, rows = shape
    c = Case(n, H, Hkv, D, rot, B, dtype, A, layout, rows, seed=n + A)
    c.k[0, 0, :5] = float("nan")
    c.v[0, 0, 40] = float("inf")
    got, status = c.run(True, inter)
    assert status == 0
    same(got, c.run_one_axis(True, inter))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv,D,rot,inter", [(32, 8, 128, 128, False), (7, 3, 64, 64, False), (8, 2, 128, 64, True),
                                               (3, 1, 64, 32, False), (4, 4, 128, 36, False), (150, 75, 128, 64, False)])
def test_long_batches_with_padding_and_bad_tokens(q4, H, Hkv, D, rot, inter, dtype):
    """Two tokens a CTA; a token is skipped for padding (whose positions may be anything), a slot past the pool, and a
    position out of range on any axis."""
    n = 1301 if H < 100 else 9
    c = Case(n, H, Hkv, D, rot, 16, dtype, 3, "turns", seed=4)
    pad, far = [0, 3, n - 1], [5]
    off = [(0, 6, -1), (1, 7, 5000), (2, n - 2, 2 ** 31 - 1)]
    want = c.run_one_axis(q4, inter, pad + far + [t for _, t, _ in off])
    c.slots[pad] = -1
    c.pos[:, pad] = -2 ** 31
    same(c.run(q4, inter)[0], c_with(c, pad, q4, inter))
    assert c.run(q4, inter)[1] == 0                          # padding is no error
    c.slots[far] = c.nb * 16
    for a, t, p in off:
        c.pos[a, t] = p
    got, status = c.run(q4, inter)
    assert status == pa.ERR_OUT_OF_RANGE
    same(got, want)


def c_with(c, skip, q4, inter):
    """The one-axis call with some tokens skipped, their positions put in range for the table."""
    keep = c.pos.clone()
    c.pos[:, skip] = 0
    want = c.run_one_axis(q4, inter, skip)
    c.pos.copy_(keep)
    return want


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("n,rot", [(40, 128), (1301, 128), (40, 36), (1301, 64)])
@pytest.mark.parametrize("bad", [-1, 3, 2 ** 31 - 1])
def test_an_axis_out_of_range_skips_every_token(q4, n, rot, bad):
    c = Case(n, 8, 2, 128, rot, 16, torch.bfloat16, 3, seed=6)
    c.axis[rot // 2 - 1] = bad
    got, status = c.run(q4, False)
    assert status == pa.ERR_OUT_OF_RANGE
    kc, vc = c.pools(q4)
    same(got, [t.view(torch.uint8) for t in (torch.full_like(c.q.contiguous(), 9.0), kc, vc)])


@pytest.mark.parametrize("q4", [False, True])
def test_equal_axes_are_one_axis(q4):
    """Text: every axis holds the same position, as rows of their own or as one row expanded."""
    c = Case(37, 8, 2, 128, 128, 16, torch.bfloat16, 3, "turns", seed=7)
    row = c.pos[:1].contiguous()
    kc, vc = c.pools(q4)
    out = torch.full((c.n, c.H, c.D), 9.0, dtype=c.dtype, device=DEV)
    (pa.rope_and_cache_q4 if q4 else pa.rope_and_cache)(c.q, c.k, c.v, c.tab, row[0], kc, vc, c.slots, q_out=out)
    want = [t.view(torch.uint8) for t in (out, kc, vc)]
    for pos in (row.repeat(3, 1), row.expand(3, c.n)):
        got, status = c.run(q4, False, positions=pos)
        assert status == 0
        same(got, want)


@pytest.mark.parametrize("q4", [False, True])
def test_no_queries_one_token_no_tokens_in_place(q4):
    fn = pa.mrope_and_cache_q4 if q4 else pa.mrope_and_cache
    c = Case(5, 4, 2, 64, 64, 16, torch.float32, 2, rows="plain", seed=8)
    want = c.run_one_axis(q4, False)
    kc, vc = c.pools(q4)
    assert fn(None, c.k, c.v, c.tab, c.pos, c.axis, kc, vc, c.slots) is None
    same([t.view(torch.uint8) for t in (kc, vc)], want[1:])
    kc, vc = c.pools(q4)
    for i in range(5):   # token by token: strides of a single token may be anything
        fn(None, c.k[i:i + 1], c.v[i:i + 1], c.tab, c.pos[:, i:i + 1], c.axis, kc, vc, c.slots[i:i + 1])
    same([t.view(torch.uint8) for t in (kc, vc)], want[1:])
    e = torch.zeros(0, 2, 64, device=DEV)
    fn(None, e, e, c.tab, c.pos[:, :0], c.axis, kc, vc, c.slots[:0])
    same([t.view(torch.uint8) for t in (kc, vc)], want[1:])
    kc, vc = c.pools(q4)
    got = fn(c.q, c.k, c.v, c.tab, c.pos, c.axis, kc, vc, c.slots, q_out=c.q)
    same([t.view(torch.uint8) for t in (got, kc, vc)], want)


def test_far_tables_past_32_bits_of_bytes():
    """A table of more than 4 GiB: its last rows are looked up."""
    rot, max_pos = 512, (5 << 30) // (512 * 4)
    c = Case(3, 2, 1, 512, rot, 16, torch.float32, 2, rows="plain", seed=9, max_pos=64)
    tab = torch.zeros(max_pos, rot, device=DEV)
    tab[-64:] = c.tab
    want = c.run_one_axis(False, False)
    got, status = c.run(False, False, cos_sin=tab, positions=c.pos + (max_pos - 64))
    assert status == 0
    same(got, want)


@pytest.mark.parametrize("q4", [False, True])
def test_a_captured_call_follows_its_buffers_on_another_stream(q4):
    c = Case(19, 8, 2, 128, 128, 16, torch.bfloat16, 3, "turns", seed=10)
    kc, vc = c.pools(q4)
    out = torch.full((c.n, c.H, c.D), 9.0, dtype=c.dtype, device=DEV)
    pos = c.pos.contiguous()
    fn = pa.mrope_and_cache_q4 if q4 else pa.mrope_and_cache
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        fn(c.q, c.k, c.v, c.tab, pos, c.axis, kc, vc, c.slots, q_out=out)
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        c.pos = torch.randint(0, 5000, pos.shape, generator=g, dtype=torch.int32).to(DEV)
        c.axis.copy_(torch.randint(0, 3, (64,), generator=g, dtype=torch.int32))
        pos.copy_(c.pos)
        for t, f in zip((kc, vc), c.pools(q4)):
            t.copy_(f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same([t.view(torch.uint8) for t in (out, kc, vc)], c.run_one_axis(q4, False))
