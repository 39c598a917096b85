"""GPU parity of decode attention over 4-bit pools against 64-bit attention on the values that the pools stand for."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa
from pagedattention_kv_cache_reshape_gb300 import workloads as W

import q4_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_kv_cache_reshape_gb300 import build
    build.build()
    pa.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Case:
    """A batch over a shuffled 4-bit pool.  Every byte that no sequence owns is 0xff (a NaN scale, codes 15)."""

    def __init__(self, ctx, H, Hkv, D, B, dtype, seed, spread=1.0, max_blocks=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.H, self.Hkv, self.D, self.B, self.dtype = np.asarray(ctx), H, Hkv, D, B, dtype
        S = len(ctx)
        need = [-(-int(c) // B) for c in ctx]
        self.nb = sum(need) + 3
        perm = rng.permutation(self.nb).astype(np.int32)
        self.mb = max_blocks or max(need)
        bt = np.full((S, self.mb), -1, np.int32)
        at = 0
        wide = [torch.randn(self.nb, B, Hkv, D, generator=g).to(torch.bfloat16).to(DEV) * spread for _ in "kv"]
        used = np.zeros((self.nb, B), bool)
        for s in range(S):
            ids = perm[at:at + need[s]]
            at += need[s]
            bt[s, :need[s]] = ids
            used[ids] = True
            if ctx[s] % B:
                used[ids[-1], ctx[s] % B:] = False
        self.k4, self.v4 = (R.new_pool(self.nb, B, Hkv, D, DEV, fill=0xff) for _ in "kv")
        ident = torch.arange(self.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
        pa.quantize_blocks_q4(wide[0], wide[1], self.k4, self.v4, ident)
        for pool in (self.k4, self.v4):
            un = torch.from_numpy(~used).to(DEV)
            codes = pool[:, :, :B * D // 2].unflatten(2, (B, D // 2))
            scales = pool[:, :, B * D // 2:].unflatten(2, (B, D // 16))
            codes[un[:, None, :].expand(-1, Hkv, -1)] = 0xff
            scales[un[:, None, :].expand(-1, Hkv, -1)] = 0xff
        self.bt, self.cl = torch.from_numpy(bt).to(DEV), torch.from_numpy(self.ctx.astype(np.int32)).to(DEV)
        self.q = torch.randn(S, H, D, generator=g).to(dtype).to(DEV)
        self.scale = W.fp32_scale(D)

    def run(self, **kw):
        kw = {"dev_status": torch.zeros(1, dtype=torch.int32, device=DEV), **kw}
        out = pa.decode_q4(self.q, self.k4, self.v4, kw.pop("bt", self.bt), kw.pop("cl", self.cl), self.scale, **kw)
        if kw["dev_status"] is not None:
            assert pa.get_device_status(kw["dev_status"]) == 0
        return out

    def check(self, out, seqs=None, what=""):
        k, v = R.values(self.k4, "k", self.B, self.D), R.values(self.v4, "v", self.B, self.D)
        bt, q, o = self.bt.cpu().numpy(), R.f64(self.q), R.f64(out)
        for s in range(len(self.ctx)) if seqs is None else seqs:
            n = int(self.ctx[s])
            ids = bt[s, :-(-n // self.B)]
            kr, vr = k[ids].reshape(-1, self.Hkv, self.D)[:n], v[ids].reshape(-1, self.Hkv, self.D)[:n]
            ref, mean, mag = R.attention(q[s], kr, vr, self.scale)
            # Logits.  fp32 sums of exact products; with bf16 queries the codes enter as n (up to 15, against 7 for
            # n - 8) and the surplus is taken off in the same sum, so its fp32 steps are those of a sum some
            # 2 * 15 / 7 < 5 times the values' own; 16 roundings or truncations (2^-23) at most lie on a sum's way.
            # The base-2 exponential and its fp32 argument add 2^-22 each of their magnitude.
            bf16 = self.dtype == torch.bfloat16
            dx = mag * ((5 if bf16 else 1) * 16 * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -21
            # Weights: one rounding to fp16 (2^-11 at most, the scale of V folded in before it); fp32 calls split
            # them into three bf16 parts and drop 2^-24.  Both sums round in fp32, at most one step a token block.
            dp = 2.0 ** -11 if bf16 else 2.0 ** -24
            steps = (n / 16 + 16) * 2.0 ** -23
            half = 2.0 ** -8 if bf16 else 2.0 ** -24
            extra = 0.0
            if bf16:
                # q in fp16, its largest element at 2^14 or more and half of the elements divided by 16: what lies
                # under the smallest step, 2^-24, is off by at most 16 * 2^-25 / 2^14 of the largest.
                G = self.H // self.Hkv
                ksum = np.repeat(np.abs(kr).sum(-1).max(0), G)
                dx = dx + 2.0 ** -35 * np.abs(q[s]).max(-1) * abs(self.scale) * ksum
                # Codes enter the second product as n too: a block of tokens is added as sum(n w s) and then
                # -sum(8 w s), each a product whose 16 addends and sum are cut at 2^-24 of the largest, 15 w s at
                # most: 2 * 17 * 15 * 2^-24 of sum(w s) over the sequence.
                zero = np.abs(np.repeat(R.scales(self.v4, self.B, self.D)[ids].reshape(-1, self.Hkv, self.D)[:n], G, 1))
                x = self.scale * np.einsum("hd,nhd->hn", q[s], np.repeat(kr, G, 1))
                w = np.exp(x - x.max(-1, keepdims=True))
                extra = 2 * 17 * 15 * 2.0 ** -24 * np.einsum("hn,nhd->hd", w / w.sum(-1, keepdims=True), zero)
                # A weight times a scale, the largest scale at 2^6 or more, has the fp16 step 2^-24 at least: half of
                # it, times |n - 8| <= 8, a token; the weights' sum is 1 or more in units of the largest.
                extra = extra + n * 8 * 2.0 ** -25 / 2.0 ** 6 * zero.max((0, 2)).reshape(-1, 1)
            rel = 2 * dx[:, None] + dp + 2 * steps
            tol = half * np.abs(ref) * (1 + rel) + rel * mean * (1 + half) + extra + 1e-30
            err = np.abs(o[s] - ref)
            assert np.all(np.isfinite(o[s])), f"{what} seq {s}: non-finite"
            assert np.all(err <= tol), f"{what} seq {s} (ctx {n}): {float((err / tol).max()):.2f} of the bound"
            if self.dtype == torch.bfloat16 and n > 1:   # the largest possible roundings do not all meet
                assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref), f"{what} seq {s}: relative RMS"


GROUPS = [(1, 1), (4, 4), (8, 2), (14, 2), (8, 1), (9, 1), (16, 1), (34, 2), (32, 1), (5, 5)]
EDGES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129, 300]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("H,Hkv", GROUPS)
def test_decode_matches_64_bits(H, Hkv, B, D, dtype):
    c = Case(EDGES, H, Hkv, D, B, dtype, seed=H * 100 + B)
    c.check(c.run(), what=f"{H}/{Hkv} B{B} D{D}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctx", [[1], [16], [17], [255], [5000], [1, 9000, 1, 40], [20000]], ids=str)
def test_decode_of_few_sequences(ctx, dtype):
    c = Case(ctx, 8, 2, 128, 16, dtype, seed=len(ctx) + ctx[0])
    c.check(c.run(), what=str(ctx))


@pytest.mark.parametrize("H,Hkv,D,B", [(32, 8, 128, 16), (4, 4, 64, 8), (24, 1, 128, 32)])
def test_decode_of_many_sequences(H, Hkv, D, B):
    rng = np.random.default_rng(5)
    ctx = np.concatenate([rng.integers(1, 40, 700), W.power_law_lengths(rng, 200, 1.2, 1, 1200)])
    c = Case(rng.permutation(ctx), H, Hkv, D, B, torch.bfloat16, seed=6)
    c.check(c.run(), seqs=list(range(0, 900, 7)) + [899], what="many")


@pytest.mark.parametrize("S", [4096, 4097, 9000])
def test_decode_of_thousands_of_sequences(S):
    """Above 4096 sequences the prefix over the lengths is made by a kernel of its own."""
    rng = np.random.default_rng(S)
    ctx = rng.integers(1, 30, S)
    ctx[S // 2] = 3000
    c = Case(ctx, 4, 1, 64, 8, torch.bfloat16, seed=S)
    out = c.run()
    c.check(out, seqs=[0, 1, S // 2 - 1, S // 2, S // 2 + 1, S - 2, S - 1] + list(range(3, S, 97)), what="thousands")
    # a sequence without a valid length among them
    cl = c.cl.clone()
    cl[S - 1], cl[5] = 0, -3
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = torch.full_like(out, 9.0)
    pa.decode_q4(c.q, c.k4, c.v4, c.bt, cl, c.scale, out=got, dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    assert torch.all(got[[5, S - 1]] == 9.0)
    c.check(got, seqs=[0, 4, 6, S // 2, S - 2], what="beside bad lengths")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv,D", [(4, 1, 128), (16, 1, 64), (40, 8, 128), (18, 1, 128)])
@pytest.mark.parametrize("pages", [60, 400])
def test_one_cta_a_head_and_the_split_agree_with_64_bits(pages, H, Hkv, D, dtype):
    """Few heads over short tables take a CTA a head; over long ones the work is split, whatever the lengths."""
    c = Case([960, 1, 777, 17], H, Hkv, D, 16, dtype, seed=pages + H, max_blocks=pages)
    c.check(c.run(), what=f"{pages} pages")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,H,Hkv,D,B,top", [(80, 8, 8, 128, 16, 512), (400, 4, 1, 64, 8, 100), (60, 64, 8, 128, 32, 300),
                                             (200, 24, 2, 64, 16, 64), (4500, 2, 1, 64, 8, 40)])
def test_many_heads_over_short_tables(S, H, Hkv, D, B, top, dtype):
    """Shares that end between heads, with sequences of no valid length among them."""
    rng = np.random.default_rng(S)
    ctx = rng.integers(1, top + 1, S)
    ctx[:3] = top, 1, top
    c = Case(ctx, H, Hkv, D, B, dtype, seed=S)
    ref = c.run()
    some = [0, 1, 2, S - 1] + list(range(3, S, max(1, S // 60)))
    c.check(ref, seqs=some, what="whole heads")
    for gone in ([0, 1], [S - 1], list(range(5, S - 5)), list(range(0, S, 2))):
        cl = c.cl.clone()
        cl[gone] = 0
        out = torch.full_like(ref, 9.0)
        pa.decode_q4(c.q, c.k4, c.v4, c.bt, cl, c.scale, out=out)
        live = [s for s in range(S) if s not in set(gone)]
        assert torch.all(out[gone] == 9.0)
        c.check(out, seqs=[s for s in some if s not in set(gone)], what="some without a length")
        assert torch.isfinite(out[live].float()).all()


def test_heads_cut_between_many_ctas():
    """One long sequence of one kv-head: every CTA holds a piece of the same head."""
    for dtype, H in ((torch.bfloat16, 3), (torch.bfloat16, 12), (torch.float32, 9)):
        c = Case([16 * 152 * 12 + 5], H, 1, 128, 16, dtype, seed=H)
        c.check(c.run(), what=f"{H} heads")


@pytest.mark.parametrize("H,Hkv,D,B", [(8, 2, 128, 16), (8, 1, 64, 32), (12, 1, 128, 8)])
def test_every_length_up_to_two_blocks_of_a_step(H, Hkv, D, B):
    c = Case(list(range(1, 70)), H, Hkv, D, B, torch.bfloat16, seed=40)
    c.check(c.run(), what="each length")


def test_scales_of_v_far_apart():
    """Scales of V over forty powers of two, rising and falling along the sequence: the lift moves both ways' weights."""
    for order in (1, -1):
        c = Case([700], 8, 2, 128, 16, torch.bfloat16, seed=41)
        e = torch.linspace(-20.0 * order, 20.0 * order, 700, device=DEV)
        v = torch.randn(c.nb, 16, 2, 128, device=DEV)
        flat = torch.ones(44 * 16, device=DEV)
        flat[:700] = torch.exp2(e)
        v[c.bt[0, :44].long()] *= flat.view(44, 16, 1, 1)
        k = torch.randn(c.nb, 16, 2, 128, device=DEV)
        ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
        pa.quantize_blocks_q4(k, v, c.k4, c.v4, ident)
        c.check(c.run(), what=f"order {order}")


def test_zero_queries_and_zero_scale_give_the_mean():
    for dtype in (torch.bfloat16, torch.float32):
        c = Case([5, 333, 16], 6, 2, 64, 16, dtype, seed=43)
        c.q[1] = 0
        c.check(c.run(), what="zero rows")
        c.scale = 0.0
        c.check(c.run(), what="zero scale")
        c.scale = -0.3
        c.check(c.run(), what="negative scale")


def test_queries_of_extreme_size():
    for factor in (2.0 ** -60, 2.0 ** 40):
        c = Case([40, 500], 8, 2, 128, 16, torch.bfloat16, seed=44)
        c.q *= factor
        c.scale = 0.1 / factor
        c.check(c.run(), what=f"q times {factor}")


def test_long_single_sequence_and_large_logits():
    c = Case([70001], 4, 1, 128, 16, torch.bfloat16, seed=9)
    c.check(c.run(), what="long")
    # logits of several hundred: one token takes nearly all the weight
    c = Case([3, 50, 700, 4097], 8, 2, 64, 16, torch.bfloat16, seed=10, spread=8.0)
    c.check(c.run(), what="peaked")
    c = Case([3, 50, 700, 4097], 8, 2, 64, 16, torch.float32, seed=11, spread=8.0)
    c.check(c.run(), what="peaked f32")


def test_rising_logits_move_the_running_maximum():
    """Keys along q, growing with the position: every block raises the maximum."""
    for sign in (1.0, -1.0):
        c = Case([1600], 4, 1, 128, 16, torch.bfloat16, seed=12)
        qd = c.q[0, 0].float()
        n = 1600
        k = torch.zeros(c.nb, 16, 1, 128, device=DEV)
        order = c.bt[0, :100].long()
        k[order] = (qd * 0.2 * torch.linspace(0, sign, n, device=DEV)[:, None]).view(100, 16, 1, 128)
        v = torch.randn(c.nb, 16, 1, 128, device=DEV)
        ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
        pa.quantize_blocks_q4(k, v, c.k4, c.v4, ident)
        c.check(c.run(), what=f"slope {sign}")


def test_misaligned_queries_and_outputs():
    for dtype in (torch.bfloat16, torch.float32):
        c = Case([40, 200, 3], 6, 2, 128, 16, dtype, seed=14)
        ref = c.run()
        buf = torch.zeros(2 * c.q.numel() + 2, dtype=dtype, device=DEV)
        q = buf[1:1 + c.q.numel()].view_as(c.q).copy_(c.q)
        out = buf[1 + c.q.numel():1 + 2 * c.q.numel()].view_as(c.q)
        pa.decode_q4(q, c.k4, c.v4, c.bt, c.cl, c.scale, out=out)
        assert torch.equal(out, ref) and buf[0] == 0 and buf[-1] == 0


def test_results_do_not_depend_on_the_blocks_nor_on_the_run():
    c = Case(list(range(1, 600, 37)), 8, 2, 128, 16, torch.bfloat16, seed=15)
    a = c.run()
    for _ in range(5):
        assert torch.equal(a, c.run())
    perm = torch.randperm(c.nb, device=DEV)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(c.nb, device=DEV)
    bt = torch.where(c.bt >= 0, inv[c.bt.clamp(min=0).long()].int(), c.bt)
    c.k4, c.v4 = c.k4[perm].contiguous(), c.v4[perm].contiguous()
    assert torch.equal(a, c.run(bt=bt))


def test_shared_blocks_are_read_by_every_sequence():
    c = Case([64, 64, 80], 8, 2, 128, 16, torch.bfloat16, seed=16)
    c.bt[1] = c.bt[0]
    c.bt[2, :4] = c.bt[0, :4]
    c.check(c.run(), what="shared")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_lengths_and_blocks_are_reported_and_harm_no_other_row(dtype):
    ctx = [33, 100, 16, 250, 90, 1]
    c = Case(ctx, 8, 2, 128, 16, dtype, seed=17, max_blocks=16)
    ref = c.run()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for bad in (0, -5, 16 * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        cl = c.cl.clone()
        cl[2] = bad
        out = torch.full_like(ref, 9.0)
        pa.reset_device_status(st)
        pa.decode_q4(c.q, c.k4, c.v4, c.bt, cl, c.scale, out=out, dev_status=st)
        assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
        live = torch.tensor([0, 1, 3, 4, 5], device=DEV)
        assert torch.all(out[2] == 9.0)
        c.check(torch.cat([out[:2], ref[2:3], out[3:]]), seqs=[0, 1, 3, 4, 5], what=f"beside a length of {bad}")
    for bad in (-1, -2 ** 31, c.nb, 2 ** 31 - 1):
        bt = c.bt.clone()
        bt[3, 7] = bad
        pa.reset_device_status(st)
        out = torch.full_like(ref, 9.0)
        pa.decode_q4(c.q, c.k4, c.v4, bt, c.cl, c.scale, out=out, dev_status=st)
        assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
        assert torch.equal(out[live[live != 3]], ref[live[live != 3]])
    # all lengths bad, and no status word: nothing is written, nothing fails
    out = torch.full_like(ref, 9.0)
    pa.decode_q4(c.q, c.k4, c.v4, c.bt, torch.zeros_like(c.cl), c.scale, out=out)
    assert torch.all(out == 9.0)


def test_nan_in_visible_rows_stays_in_its_head():
    c = Case([50], 4, 2, 128, 16, torch.bfloat16, seed=18)
    ref = c.run()
    B, D = 16, 128
    blk = int(c.bt[0, 1])
    c.k4[blk, 1, B * D // 2 + 5 * (D // 16):B * D // 2 + 5 * (D // 16) + 2] = 0xff
    out = c.run()
    assert torch.equal(out[0, :2], ref[0, :2]) and torch.all(torch.isnan(out[0, 2:].float()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity_in_a_query_stay_in_its_head(dtype):
    c = Case([300, 33], 6, 2, 128, 16, dtype, seed=45)
    ref = c.run()
    c.q[0, 1, 7] = float("nan")
    c.q[1, 4, 100] = float("inf")
    out = c.run()
    bad = torch.zeros(2, 6, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 4] = True
    assert torch.equal(out[~bad], ref[~bad]) and not torch.isfinite(out[bad].float()).any()


def test_nan_scale_of_v_stays_in_its_dims():
    c = Case([90], 4, 2, 128, 16, torch.bfloat16, seed=46)
    ref = c.run()
    B, D = 16, 128
    at = B * D // 2 + 3 * (D // 16) + 2 * 2            # token 3, group 2
    c.v4[int(c.bt[0, 2]), 0, at:at + 2] = 0xff
    out = c.run()
    assert torch.equal(out[0, 2:], ref[0, 2:]) and torch.isnan(out[0, :2, 64:96].float()).all()
    other = torch.cat([out[0, :2, :64], out[0, :2, 96:]], 1).float()
    want = torch.cat([ref[0, :2, :64], ref[0, :2, 96:]], 1).float()
    assert torch.allclose(other, want, rtol=2.0 ** -7, atol=1e-3)   # the lift may differ: roundings of weights and result


def test_workspace_contents_do_not_matter_and_calls_may_share_it_in_order():
    a = Case([700, 20, 5, 3000], 8, 2, 128, 16, torch.bfloat16, seed=19)
    b = Case([9, 4000], 32, 8, 128, 16, torch.bfloat16, seed=20)
    ra, rb = a.run(), b.run()
    need = max(pa.decode_q4_workspace_size(4, 8, 2, 128, 16, a.mb), pa.decode_q4_workspace_size(2, 32, 8, 128, 16, b.mb))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(a.run(workspace=ws), ra) and torch.equal(b.run(workspace=ws), rb)


def test_captured_and_replayed_on_another_stream():
    c = Case([700, 20, 5, 3000], 8, 2, 128, 16, torch.bfloat16, seed=21)
    ref = c.run()
    ws = torch.empty(pa.decode_q4_workspace_size(4, 8, 2, 128, 16, c.mb), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # new lengths in the captured buffers
    c.cl.copy_(torch.tensor([60, 7, 4, 2999], dtype=torch.int32, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale))


def test_two_streams_with_workspaces_of_their_own():
    cs = [Case([3000, 17, 900], 8, 2, 128, 16, torch.bfloat16, seed=22 + i) for i in range(2)]
    refs = [c.run() for c in cs]
    outs = [torch.zeros_like(r) for r in refs]
    wss = [torch.empty(pa.decode_q4_workspace_size(3, 8, 2, 128, 16, c.mb), dtype=torch.uint8, device=DEV) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, o, w, s in zip(cs, outs, wss, streams):
            pa.decode_q4(c.q, c.k4, c.v4, c.bt, c.cl, c.scale, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


def test_blocks_past_32_bits_of_bytes():
    """Pools of more than 4 GiB: the same blocks at both ends give the same bits."""
    for B, H, Hkv, D, dtype in ((16, 32, 8, 128, torch.bfloat16), (8, 6, 6, 64, torch.float32)):
        c = Case([100, 7, 333], H, Hkv, D, B, dtype, seed=47)
        ref = c.run()
        per = c.k4[0].numel()
        nb = (4 << 30) // per + 2 * c.nb
        far = nb - c.nb
        for name in ("k4", "v4"):
            pool = torch.zeros(nb, *getattr(c, name).shape[1:], dtype=torch.uint8, device=DEV)
            pool[far:] = getattr(c, name)
            setattr(c, name, pool)
        out = c.run(bt=torch.where(c.bt >= 0, c.bt + far, c.bt).int())
        assert far * per > 1 << 32 and torch.equal(out, ref)


def test_no_sequences():
    c = Case([5], 4, 2, 64, 16, torch.bfloat16, seed=24)
    out = pa.decode_q4(c.q[:0], c.k4, c.v4, c.bt[:0], c.cl[:0], c.scale)
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("B", [8, 16, 32])
def test_a_request_served_from_the_4_bit_cache(B):
    """Prompt prefilled in a bf16 pool, its blocks turned to 4 bits, then tokens decoded one by one: rotation with
    append, and attention, through the block manager's tables."""
    H, Hkv, D, steps = 8, 2, 128, 2 * B + 3
    prompts = [B + 3, 5, 3 * B]
    S = len(prompts)
    mb = (max(prompts) + steps) // B + 2
    bm = pa.BlockManager(S * mb + 4, B, mb)
    tab = R.table(512, D).to(DEV)
    scale = W.fp32_scale(D)
    g = torch.Generator().manual_seed(30)
    k16 = torch.zeros(bm.num_blocks, B, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v16 = torch.zeros_like(k16)
    k4, v4 = (R.new_pool(bm.num_blocks, B, Hkv, D, DEV, fill=0xff) for _ in "kv")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hist_k, hist_v = [[] for _ in prompts], [[] for _ in prompts]

    def fresh(n):
        x = torch.randn(n, (H + 2 * Hkv) * D, generator=g).bfloat16().to(DEV)
        return tuple(t.unflatten(1, (-1, D)) for t in x.split([H * D, Hkv * D, Hkv * D], 1))

    def step(lens, before, into4):
        n = int(sum(lens))
        for s, m in enumerate(lens):
            assert bm.allocate_slots(s, m) == pa.OK
        bt = bm.tables(range(S), mb)[0].to(DEV)
        start = torch.tensor(before, dtype=torch.int32, device=DEV)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        slots = pa.compute_slot_mapping(bt, start, cu, bm.num_blocks, n, block_size=B, dev_status=st)
        pos = torch.cat([torch.arange(b, b + m) for b, m in zip(before, lens)]).int().to(DEV)
        q, k, v = fresh(n)
        if into4:
            qo = pa.rope_and_cache_q4(q, k, v, tab, pos, k4, v4, slots, dev_status=st)
        else:
            qo = pa.rope_and_cache(q, k, v, tab, pos, k16, v16, slots, dev_status=st)
        kr = torch.from_numpy(R.rotate(k, tab, pos.cpu().numpy(), D, False)[0]).float().bfloat16()
        at = 0
        for s, m in enumerate(lens):
            hist_k[s].append(kr[at:at + m])
            hist_v[s].append(v[at:at + m].cpu())
            at += m
        ctx = torch.tensor([b + m for b, m in zip(before, lens)], dtype=torch.int32, device=DEV)
        return bt, ctx, cu, q, qo

    bt, ctx, cu, q, qo = step(prompts, [0] * S, False)
    pre = pa.varlen_prefill(qo, cu, k16, v16, bt, ctx, scale, max(prompts), dev_status=st)
    assert torch.isfinite(pre).all()
    own = bt[bt >= 0]
    pa.quantize_blocks_q4(k16, v16, k4, v4, torch.stack([own, own], 1).contiguous(), dev_status=st)
    before = list(prompts)
    for t in range(steps):
        bt, ctx, cu, q, qo = step([1] * S, before, True)
        before = [b + 1 for b in before]
        out = pa.decode_q4(qo, k4, v4, bt, ctx, scale, dev_status=st)
        if t % 5 and t != steps - 1:
            continue
        qr = R.rotate(q, tab, [b - 1 for b in before], D, False)[0]
        for s in range(S):
            def vals(hist):
                nib, sb = R.quantize(torch.cat(hist).float().numpy())
                return ((nib.astype(np.float64) - 8).reshape(*nib.shape[:2], -1, 32)
                        * (sb.astype(np.uint32) << 16).view(np.float32)[..., None]).reshape(nib.shape)
            ref = R.attention(qr[s], vals(hist_k[s]), vals(hist_v[s]), scale)[0]
            err = np.abs(R.f64(out[s]) - ref)
            # roundings of q (2^-8 of logits of a few units), of the weights and of the result
            assert err.max() <= 4e-2 and np.linalg.norm(err) <= 1.5e-2 * np.linalg.norm(ref), (t, s)
    assert pa.get_device_status(st) == 0
    bm.close()
