"""GPU tests of rotated rows that hold infinities, or whose turned values pass the largest fp32."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative
INF = float("inf")
PAIRS = [(INF, 1.0), (1.0, -INF), (INF, INF), (-INF, INF), (3e38, 3e38), (-3e38, 3e38), (3e38, -1.0), (float("nan"), 1.0)]
TURNS = [(0.8, 0.6), (0.8, -0.6), (1.0, 0.0), (0.0, 1.0), (-0.6, 0.8), (1.5, 0.5)]   # (cos, sin) of the positions


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_kv_cache_reshape_gb300 import build
    build.build()
    pa.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def place(D, rot, inter):
    i = min(3, rot // 2 - 1)
    return (i, i + rot // 2) if not inter else (2 * i, 2 * i + 1)


def forms(x, tab, pos, rot, inter):
    """The definition in fp32 and in 64 bits (either is allowed where products overflow), both as fp32 values."""
    r = rot // 2
    i = np.arange(r)
    one, two = (2 * i, 2 * i + 1) if inter else (i, i + r)
    out = []
    for t in (np.float32, np.float64):
        y, cs = R.f64(x).astype(t), R.f64(tab).astype(t)[pos][:, None]
        c, s, a, b = cs[..., :r], cs[..., r:], y[..., one], y[..., two]
        z = y.copy()
        with np.errstate(all="ignore"):
            z[..., one], z[..., two] = a * c - b * s, b * c + a * s
            out.append((z, z.astype(np.float32)))
    return out[0][1], out[1][1], out[1][0]


def check(got, x, tab, pos, rot, inter, what):
    dtype, g = got.dtype, R.f64(got)
    f32, near, exact = forms(x, tab, pos, rot, inter)
    with np.errstate(all="ignore"):
        def same(a):
            a = R.f64(torch.from_numpy(a).to(dtype))
            return (g == a) | (np.isnan(g) & np.isnan(a))
        mag = R.rotate(torch.nan_to_num(x.float(), 0.0, 0.0, 0.0), tab, pos, rot, inter)[1]
        close = np.isfinite(g) & (np.abs(g - exact) <= HALF[dtype] * (1 + 2 ** -8) * np.abs(exact) + 3 * 2.0 ** -24 * mag)
        ok = close | (~np.isfinite(g) & (same(f32) | same(near)))
    assert ok.all(), f"{what}: {g[~ok][:4]} where {exact[~ok][:4]} are due"


SHAPES = [(128, 128), (64, 32), (96, 64), (128, 72), (40, 14)]   # the last two go element by element


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("long", [False, True])
def test_infinities_and_overflow_follow_the_formula(D, rot, inter, dtype, long):
    n, H, Hkv, B = len(PAIRS) * len(TURNS), 2, 2, 16
    g = torch.Generator().manual_seed(D + rot)
    x = torch.randn(n, H + 2 * Hkv, D, generator=g)
    a, b = place(D, rot, inter)
    for t in range(n):
        x[t, 0, a], x[t, 0, b] = PAIRS[t % len(PAIRS)]             # the first query row
        x[t, H, a], x[t, H, b] = PAIRS[t % len(PAIRS)]             # the first key row
        x[t, H + Hkv + 1, a] = PAIRS[t % len(PAIRS)][0]            # a value row: not turned
    x = x.to(dtype).to(DEV)
    pos = np.arange(n) // len(PAIRS)
    if long:   # two tokens a CTA
        x, pos = x.repeat(28, 1, 1), np.tile(pos, 28)
        n = n * 28
    q, k, v = x[:, :H].contiguous(), x[:, H:H + Hkv].contiguous(), x[:, H + Hkv:].contiguous()
    r = rot // 2
    tab = torch.tensor([[c] * r + [s] * r for c, s in TURNS], device=DEV)
    dpos = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    nb = n // B + 2
    slots = torch.randperm(nb * B, generator=g)[:n].to(DEV)
    kc, vc = (torch.zeros(nb, B, Hkv, D, dtype=dtype, device=DEV) for _ in "kv")
    out = pa.rope_and_cache(q, k, v, tab, dpos, kc, vc, slots, interleaved=inter)
    check(out, q, tab, pos, rot, inter, "q_out")
    got = kc.view(nb * B, Hkv, D)[slots]
    check(got, k, tab, pos, rot, inter, "k_cache")
    kind = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(vc.view(nb * B, Hkv, D)[slots].view(kind), v.view(kind))
    if D not in (64, 128) or long:
        return
    # and into 4 bits: what quantising those rows gives, a group that is not finite as a NaN
    k4, v4 = R.new_pool(nb, B, Hkv, D, DEV, fill=0), R.new_pool(nb, B, Hkv, D, DEV, fill=0)
    pa.rope_and_cache_q4(q, k, v, tab, dpos, k4, v4, slots, interleaved=inter)
    want = np.zeros(tuple(k4.shape), np.uint8)
    rows = got.float().cpu().numpy()
    for t, s in enumerate(slots.tolist()):
        for h in range(Hkv):
            R.store(want, "k", s // B, h, s % B, *R.quantize(rows[t, h]), B, D)
    assert np.array_equal(k4.cpu().numpy(), want)
