"""GPU parity of the position rotation with its cache write, of the 4-bit rows and of the block conversions, against
the 64-bit reference in q4_reference.py.  Cache bytes are compared bit for bit where the format defines them."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_kv_cache_reshape_gb300 import build
    build.build()
    pa.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


def inputs(n, H, Hkv, D, dtype, layout, seed):
    """q, key, value [n, heads, D]: views of one fused projection, separate, or at an odd element offset."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, (H + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
    if layout == "fused":
        return tuple(t.unflatten(1, (-1, D)) for t in x.split([H * D, Hkv * D, Hkv * D], 1))
    out = []
    for t in x.split([H * D, Hkv * D, Hkv * D], 1):
        flat = torch.empty(t.numel() + 1, dtype=dtype, device=DEV)[1 if layout == "odd" else 0:]
        flat = flat[:t.numel()].copy_(t.reshape(-1))
        out.append(flat.view(n, -1, D))
    return tuple(out)


def check_rows(got, ref, mag, dtype, what):
    """One rounding to the type (through fp32), and two roundings of fp32 products and one of their sum."""
    err = np.abs(R.f64(got) - ref)
    tol = HALF[dtype] * (1 + 2 ** -8) * np.abs(ref) + 3 * 2.0 ** -24 * mag
    assert np.all(err <= tol), f"{what}: {float((err - tol).max()):.3e} over the bound"


SHAPES = [  # n, H, Hkv, D, rot, interleaved, B, layout
    (1, 1, 1, 64, 64, False, 16, "fused"), (37, 32, 8, 128, 128, False, 16, "fused"),
    (37, 8, 2, 128, 128, True, 8, "plain"), (5, 14, 2, 128, 64, False, 32, "fused"),
    (300, 4, 4, 64, 32, True, 16, "fused"), (9, 6, 3, 64, 24, False, 16, "odd"),
    (3, 2, 2, 96, 96, False, 5, "plain"), (3, 3, 1, 40, 14, True, 1, "plain"), (4, 2, 1, 63, 62, False, 7, "odd"),
    (6, 5, 5, 128, 2, True, 16, "fused"), (6, 5, 5, 128, 2, False, 16, "odd"), (11, 40, 2, 256, 128, False, 16, "fused"),
    (17, 12, 4, 64, 0, False, 16, "fused"), (8, 0, 8, 128, 128, False, 16, "plain"), (130, 71, 1, 64, 64, False, 16, "fused"),
    (7, 4, 2, 128, 48, False, 16, "fused"), (7, 4, 2, 128, 80, False, 16, "plain"), (7, 4, 2, 128, 16, True, 16, "fused"),
]


def make_case(n, H, Hkv, D, rot, B, seed, extra=7, max_pos=5000):
    rng = np.random.default_rng(seed)
    nb = -(-(n + extra) // B) + 2
    slots = rng.permutation(nb * B)[:n].astype(np.int64)
    pos = rng.integers(0, max_pos, size=n).astype(np.int32)
    pos[:2] = (max_pos - 1, 0)[:n]
    return nb, torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV), R.table(max_pos, rot).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope_and_cache_matches_the_formula(shape, dtype):
    n, H, Hkv, D, rot, inter, B, layout = shape
    q, k, v = inputs(n, H, Hkv, D, dtype, layout, 11)
    nb, slots, pos, tab = make_case(n, H, Hkv, D, rot, B, 12)
    kc = torch.full((nb, B, Hkv, D), 7.0, dtype=dtype, device=DEV)
    vc = torch.full_like(kc, -3.0)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.rope_and_cache(q if H else None, k, v, tab if rot else None, pos if rot else None, kc, vc, slots,
                            interleaved=inter, dev_status=st)
    assert pa.get_device_status(st) == 0
    p = pos.cpu().numpy()
    if H:
        check_rows(out, *R.rotate(q, tab, p, rot, inter), dtype, "q_out")
    else:
        assert out is None
    s = slots.cpu()
    got_k = kc.cpu().reshape(nb * B, Hkv, D)
    check_rows(got_k[s], *R.rotate(k, tab, p, rot, inter), dtype, "k_cache")
    want_v = torch.full((nb * B, Hkv, D), -3.0, dtype=dtype)
    want_v[s] = v.cpu()
    assert torch.equal(bits(vc.cpu().reshape(nb * B, Hkv, D)), bits(want_v))
    rest = torch.ones(nb * B, dtype=torch.bool)
    rest[s] = False
    assert torch.all(got_k[rest] == 7.0)   # no other slot is touched


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,D,rot", [(torch.bfloat16, 128, 128), (torch.float32, 64, 32), (torch.bfloat16, 80, 36)])
def test_rope_in_place_equals_apart(dtype, D, rot, inter):
    q, k, v = inputs(33, 6, 2, D, dtype, "plain", 3)
    nb, slots, pos, tab = make_case(33, 6, 2, D, rot, 16, 4)
    kc = torch.zeros(nb, 16, 2, D, dtype=dtype, device=DEV)
    vc = torch.zeros_like(kc)
    want = pa.rope_and_cache(q, k, v, tab, pos, kc, vc, slots, interleaved=inter)
    got = pa.rope_and_cache(q, k, v, tab, pos, kc, vc, slots, interleaved=inter, q_out=q)
    assert got is q and torch.equal(bits(q), bits(want))


@pytest.mark.parametrize("q4", [False, True])
def test_rope_skips_padding_and_reports_bad_slots_and_positions(q4):
    n, H, Hkv, D, B = 40, 8, 2, 128, 16
    q, k, v = inputs(n, H, Hkv, D, torch.bfloat16, "fused", 5)
    nb, slots, pos, tab = make_case(n, H, Hkv, D, D, B, 6, max_pos=100)
    fn = pa.rope_and_cache_q4 if q4 else pa.rope_and_cache

    def pools():
        if q4:
            return R.new_pool(nb, B, Hkv, D, DEV, seed=1), R.new_pool(nb, B, Hkv, D, DEV, seed=2)
        return (torch.full((nb, B, Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV),
                torch.full((nb, B, Hkv, D), 6.0, dtype=torch.bfloat16, device=DEV))
    full = pools()
    ref = fn(q, k, v, tab, pos, *full, slots)
    bad = {"pad": [0, 7, n - 1], "slot": [3], "pos": [9, 20]}
    s2, p2 = slots.clone(), pos.clone()
    s2[bad["pad"]] = -1
    p2[bad["pad"]] = 2 ** 31 - 1          # never read
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pools()
    out = torch.full((n, H, D), 9.0, dtype=torch.bfloat16, device=DEV)
    fn(q, k, v, tab, p2, *got, s2, q_out=out, dev_status=st)
    assert pa.get_device_status(st) == 0   # padding is no error
    live = torch.ones(n, dtype=torch.bool, device=DEV)
    live[bad["pad"]] = False
    assert torch.equal(out[live], ref[live]) and torch.all(out[~live] == 9.0)
    s2[bad["slot"]] = nb * B
    p2[bad["pos"]] = torch.tensor([-1, 100], dtype=torch.int32, device=DEV)
    got = pools()
    out.fill_(9.0)
    fn(q, k, v, tab, p2, *got, s2, q_out=out, dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    live[bad["slot"] + bad["pos"]] = False
    assert torch.equal(out[live], ref[live]) and torch.all(out[~live] == 9.0)
    # the pools hold the live rows and, everywhere else, what they held
    keep = pools()
    fn(q[live], k[live], v[live], tab, pos[live], *keep, slots[live])
    for a, b in zip(got, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] in (64, 128) and s[6] in (8, 16, 32)], ids=str)
def test_rope_into_4_bit_pools_equals_rope_then_quantize(shape, dtype):
    n, H, Hkv, D, rot, inter, B, layout = shape
    q, k, v = inputs(n, H, Hkv, D, dtype, layout, 21)
    k[0, 0, :5] = float("nan")
    v[0, 0, 40] = float("inf")
    v[n - 1] = 0
    nb, slots, pos, tab = make_case(n, H, Hkv, D, rot, B, 22)
    args = (q if H else None, k, v, tab if rot else None, pos if rot else None)
    k4, v4 = R.new_pool(nb, B, Hkv, D, DEV, fill=0), R.new_pool(nb, B, Hkv, D, DEV, fill=0)
    out4 = pa.rope_and_cache_q4(*args, k4, v4, slots, interleaved=inter)
    kc = torch.zeros(nb, B, Hkv, D, dtype=dtype, device=DEV)
    vc = torch.zeros_like(kc)
    out = pa.rope_and_cache(*args, kc, vc, slots, interleaved=inter)
    if H:
        assert torch.equal(bits(out4), bits(out))
    k8, v8 = torch.empty_like(k4), torch.empty_like(v4)
    pairs = torch.arange(nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
    pa.quantize_blocks_q4(kc, vc, k8, v8, pairs)
    # both pools agree on every written row, and the rest of the appended pool is as it was
    want_k, want_v = np.zeros(tuple(k4.shape), np.uint8), np.zeros(tuple(v4.shape), np.uint8)
    fk, fv = kc.float().cpu().numpy().reshape(-1, Hkv, D), vc.float().cpu().numpy().reshape(-1, Hkv, D)
    for s in slots.tolist():
        for h in range(Hkv):
            R.store(want_k, "k", s // B, h, s % B, *R.quantize(fk[s, h]), B, D)
            R.store(want_v, "v", s // B, h, s % B, *R.quantize(fv[s, h]), B, D)
    assert np.array_equal(k4.cpu().numpy(), want_k) and np.array_equal(v4.cpu().numpy(), want_v)
    a, b = R.values(k4, "k", B, D).reshape(-1, Hkv, D), R.values(k8, "k", B, D).reshape(-1, Hkv, D)
    s = slots.cpu().numpy()
    assert np.array_equal(a[s], b[s], equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q4,H,Hkv,D,rot,inter", [
    (False, 32, 8, 128, 128, False), (False, 5, 3, 96, 64, True), (True, 32, 8, 128, 128, False),
    (True, 7, 3, 64, 64, False), (True, 4, 4, 128, 128, True), (True, 6, 2, 64, 0, False), (True, 8, 2, 128, 64, False),
    (True, 3, 1, 64, 32, True), (True, 0, 5, 128, 128, False)])
def test_long_batches_equal_short_ones(q4, H, Hkv, D, rot, inter, dtype):
    """1301 tokens at once (two a CTA) against the same tokens in calls of 100 (one a CTA), with padding, a bad slot
    and a bad position among them: every byte."""
    n, B = 1301, 16
    q, k, v = inputs(n, H, Hkv, D, dtype, "fused", 51)
    nb, slots, pos, tab = make_case(n, H, Hkv, D, rot, B, 52, max_pos=3000)
    slots[[0, 17, 640, 641, n - 1]] = -1
    slots[33] = nb * B
    if rot:
        pos[[50, 900]] = torch.tensor([-7, 3000], dtype=torch.int32, device=DEV)
    fn = pa.rope_and_cache_q4 if q4 else pa.rope_and_cache

    def run(step):
        if q4:
            kc, vc = R.new_pool(nb, B, Hkv, D, DEV, seed=1), R.new_pool(nb, B, Hkv, D, DEV, seed=2)
        else:
            kc, vc = (torch.full((nb, B, Hkv, D), 5.0, dtype=dtype, device=DEV) for _ in "kv")
        out = torch.full((n, H, D), 9.0, dtype=dtype, device=DEV) if H else None
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        for i in range(0, n, step):
            j = slice(i, i + step)
            fn(q[j] if H else None, k[j], v[j], tab if rot else None, pos[j] if rot else None, kc, vc, slots[j],
               interleaved=inter, q_out=out[j] if H else None, dev_status=st)
        assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
        return [t.contiguous().view(torch.uint8) for t in (kc, vc, out) if t is not None]
    for a, b in zip(run(n), run(100)):
        assert torch.equal(a, b)


def test_keys_and_values_of_wide_rows():
    """More K/V heads than a CTA's shared memory or one pass of its threads holds."""
    n, H, Hkv, D, B = 3, 150, 75, 128, 16
    q, k, v = inputs(n, H, Hkv, D, torch.float32, "plain", 61)
    nb, slots, pos, tab = make_case(n, H, Hkv, D, 64, B, 62)
    for rot in (0, 64, 128):
        tab = R.table(5000, rot).to(DEV) if rot else None
        k4, v4 = R.new_pool(nb, B, Hkv, D, DEV, fill=0), R.new_pool(nb, B, Hkv, D, DEV, fill=0)
        out4 = pa.rope_and_cache_q4(q, k, v, tab, pos if rot else None, k4, v4, slots)
        kc = torch.zeros(nb, B, Hkv, D, device=DEV)
        vc = torch.zeros_like(kc)
        out = pa.rope_and_cache(q, k, v, tab, pos if rot else None, kc, vc, slots)
        assert torch.equal(out, out4)
        k8, v8 = R.new_pool(nb, B, Hkv, D, DEV, fill=0), R.new_pool(nb, B, Hkv, D, DEV, fill=0)
        pairs = torch.arange(nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
        pa.quantize_blocks_q4(kc, vc, k8, v8, pairs)
        s = slots.cpu().numpy()
        for a, b, kind in ((k4, k8, "k"), (v4, v8, "v")):
            assert np.array_equal(R.values(a, kind, B, D).reshape(-1, Hkv, D)[s], R.values(b, kind, B, D).reshape(-1, Hkv, D)[s])


def test_a_captured_step_follows_its_buffers():
    """Slot mapping, rotation with append, 4-bit decode and expansion in one graph, replayed with other tokens."""
    H, Hkv, D, B, S, mb = 8, 2, 128, 16, 3, 4
    nb = S * mb
    g = torch.Generator().manual_seed(70)
    bt = torch.randperm(nb, generator=g).int().view(S, mb).to(DEV)
    tab = R.table(64, D).to(DEV)
    qkv = torch.empty(S, (H + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, Hkv * D, Hkv * D], 1))
    start = torch.zeros(S, dtype=torch.int32, device=DEV)
    ctx = torch.ones(S, dtype=torch.int32, device=DEV)
    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(S, dtype=torch.int64, device=DEV)
    back = torch.stack([bt.flatten(), torch.arange(nb, device=DEV).int()], 1).contiguous()
    ws = torch.empty(pa.decode_q4_workspace_size(S, H, Hkv, D, B, mb), dtype=torch.uint8, device=DEV)

    def state():
        return dict(k4=R.new_pool(nb, B, Hkv, D, DEV, fill=0), v4=R.new_pool(nb, B, Hkv, D, DEV, fill=0),
                    qo=torch.zeros(S, H, D, dtype=torch.bfloat16, device=DEV), out=torch.zeros(S, H, D, dtype=torch.bfloat16, device=DEV),
                    wk=torch.zeros(nb, B, Hkv, D, dtype=torch.bfloat16, device=DEV), wv=torch.zeros(nb, B, Hkv, D, dtype=torch.bfloat16, device=DEV))

    def step(z):
        pa.compute_slot_mapping(bt, start, cu, nb, S, slot_mapping=slots)
        pa.rope_and_cache_q4(q, k, v, tab, start, z["k4"], z["v4"], slots, q_out=z["qo"])
        pa.decode_q4(z["qo"], z["k4"], z["v4"], bt, ctx, 0.09, out=z["out"], workspace=ws)
        pa.dequantize_blocks_q4(z["k4"], z["v4"], z["wk"], z["wv"], back)
    a, b = state(), state()
    step(a)
    a = state()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step(a)
    torch.cuda.synchronize()
    for t in range(40):
        qkv.copy_(torch.randn(qkv.shape, generator=g).to(DEV))
        start.fill_(t)
        ctx.fill_(t + 1)
        graph.replay()
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        assert torch.isfinite(a["out"].float()).all()
        for name in a:
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), (t, name)


def rows_with_edges(n, B, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, B, H, D, generator=g) * torch.exp(2 * torch.randn(n, B, H, 1, generator=g))
    f = x.view(-1, 32)
    f[0] = 0
    f[1, 3] = float("nan")
    f[2, 30] = float("-inf")
    f[3] = torch.linspace(-7, 7, 32) * 1e-39                 # subnormals
    f[4] = 1e-45
    f[5] = torch.arange(32).float() / 2 - 7                   # amax 8.5: codes around borders
    f[6] = (torch.arange(32).float() - 14) / 2                # scale 1 or so, exact ties
    f[6, 0] = 7.0
    f[7] = 3.3e38
    f[8, 1:] = 0
    f[9] = -0.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,D", [(16, 8, 128), (8, 1, 64), (32, 3, 64), (8, 5, 128), (32, 2, 128), (16, 7, 64)])
def test_block_conversion_is_bit_exact(B, H, D, dtype):
    n, m = 23, 29
    k, v = rows_with_edges(n, B, H, D, dtype, 31), rows_with_edges(n, B, H, D, dtype, 32)
    rng = np.random.default_rng(33)
    pairs = np.stack([rng.permutation(n)[:17], rng.permutation(m)[:17]], 1).astype(np.int32)
    pairs[4, 0], pairs[6, 1] = -1, -5
    start_k, start_v = R.new_pool(m, B, H, D, "cpu", seed=3), R.new_pool(m, B, H, D, "cpu", seed=4)
    k4, v4 = start_k.to(DEV), start_v.to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dp = torch.from_numpy(pairs).to(DEV)
    pa.quantize_blocks_q4(k.to(DEV), v.to(DEV), k4, v4, dp, dev_status=st)
    want_k, want_v = start_k.numpy().copy(), start_v.numpy().copy()
    for src, dst in pairs.tolist():
        if src < 0 or dst < 0:
            continue
        for tok in range(B):
            for h in range(H):
                R.store(want_k, "k", dst, h, tok, *R.quantize(k[src, tok, h].float().numpy()), B, D)
                R.store(want_v, "v", dst, h, tok, *R.quantize(v[src, tok, h].float().numpy()), B, D)
    assert np.array_equal(k4.cpu().numpy(), want_k) and np.array_equal(v4.cpu().numpy(), want_v)
    # and out again: (n - 8) s rounded once, whatever the bytes of the block are
    wk = torch.full((n, B, H, D), 3.0, dtype=dtype, device=DEV)
    wv = torch.full_like(wk, 4.0)
    pa.dequantize_blocks_q4(k4, v4, wk, wv, dp.flip(1).contiguous(), dev_status=st)
    assert pa.get_device_status(st) == 0
    with np.errstate(over="ignore"):
        for pool, got, kind, keep in ((want_k, wk, "k", 3.0), (want_v, wv, "v", 4.0)):
            want = torch.full((n, B, H, D), keep, dtype=dtype)
            vals = R.values(pool, kind, B, D).astype(np.float32)   # exact: at most 12 significant bits
            for src, dst in pairs.tolist():
                if src >= 0 and dst >= 0:
                    want[src] = torch.from_numpy(vals[dst]).to(dtype)
            g = got.cpu()
            assert torch.equal(torch.isnan(g), torch.isnan(want))
            ok = ~torch.isnan(want)
            assert torch.equal(g[ok], want[ok])


@pytest.mark.parametrize("quantize", [True, False])
def test_block_conversion_reports_pairs_past_the_pools(quantize):
    wide = torch.randn(5, 16, 2, 64, device=DEV).bfloat16()
    q4 = R.new_pool(4, 16, 2, 64, DEV, fill=0x11)
    for bad in ((5, 0), (0, 4)) if quantize else ((4, 0), (0, 5)):
        w1, w2, a, b = wide.clone(), wide.clone(), q4.clone(), q4.clone()
        pairs = torch.tensor([[1, 2], list(bad), [2, 1]], dtype=torch.int32, device=DEV)
        good = torch.tensor([[1, 2], [2, 1]], dtype=torch.int32, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        fn = (lambda p, s: pa.quantize_blocks_q4(w1, w2, a, b, p, dev_status=s)) if quantize else \
            (lambda p, s: pa.dequantize_blocks_q4(a, b, w1, w2, p, dev_status=s))
        fn(pairs, st)
        assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
        got = [t.clone() for t in (w1, w2, a, b)]
        for t, s in zip((w1, w2, a, b), (wide, wide, q4, q4)):
            t.copy_(s)
        fn(good, None)
        for x, y in zip(got, (w1, w2, a, b)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_no_pairs_and_no_tokens_launch_nothing():
    wide = torch.zeros(2, 16, 2, 64, device=DEV)
    q4 = R.new_pool(2, 16, 2, 64, DEV, fill=0)
    none = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    pa.quantize_blocks_q4(wide, wide, q4, q4, none)
    pa.dequantize_blocks_q4(q4, q4, wide, wide, none)
    e = torch.zeros(0, 2, 64, device=DEV)
    pa.rope_and_cache(e, e, e, R.table(4, 64).to(DEV), torch.zeros(0, dtype=torch.int32, device=DEV), wide, wide,
                      torch.zeros(0, dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()


def test_copy_blocks_moves_4_bit_blocks():
    B, H, D = 16, 3, 128
    a, b = R.new_pool(9, B, H, D, DEV, seed=5), R.new_pool(9, B, H, D, DEV, seed=6)
    c, d = R.new_pool(6, B, H, D, DEV, fill=0), R.new_pool(6, B, H, D, DEV, fill=0)
    assert a[0].numel() == pa.q4_block_bytes(B, H, D)
    pa.copy_blocks(a, b, c, d, torch.tensor([[8, 0], [2, 5]], dtype=torch.int32, device=DEV))
    assert torch.equal(c[0], a[8]) and torch.equal(c[5], a[2]) and torch.equal(d[5], b[2]) and not c[1].any()


def test_far_slots_past_32_bits_of_bytes():
    """A 4-bit pool of more than 4 GiB: the last blocks are written and read back."""
    B, H, D = 32, 32, 128
    nb = (5 << 30) // (H * R.slab_bytes(B, D))
    k4 = torch.zeros(nb, H, R.slab_bytes(B, D), dtype=torch.uint8, device=DEV)
    v4 = torch.zeros_like(k4)
    n = 3
    q, k, v = inputs(n, 32, H, D, torch.bfloat16, "plain", 8)
    slots = torch.tensor([nb * B - 1, 0, nb * B - B], dtype=torch.int64, device=DEV)
    tab, pos = R.table(64, D).to(DEV), torch.tensor([63, 1, 2], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.rope_and_cache_q4(q, k, v, tab, pos, k4, v4, slots, dev_status=st)
    wk = torch.zeros(2, B, H, D, dtype=torch.bfloat16, device=DEV)
    wv = torch.zeros_like(wk)
    pa.dequantize_blocks_q4(k4, v4, wk, wv, torch.tensor([[nb - 1, 0], [0, 1]], dtype=torch.int32, device=DEV), dev_status=st)
    assert pa.get_device_status(st) == 0
    nib, sb = R.quantize(v.float().cpu().numpy())
    want = ((nib.astype(np.float64) - 8).reshape(n, H, -1, 32)
            * (sb.astype(np.uint32) << 16).view(np.float32)[..., None]).reshape(n, H, D)
    want = torch.from_numpy(want).float().bfloat16()
    assert torch.equal(wv[0, B - 1].cpu(), want[0]) and torch.equal(wv[1, 0].cpu(), want[1])
    assert torch.equal(wv[0, 0].cpu(), want[2]) and not wv[0, 1:B - 1].any() and not wv[1, 1:].any()
