"""Keys with infinities, whose logits are minus infinity over whole tiles, units or pieces: such keys have weight 0 and
take no part in the maximum, however small the other logits are; where no key is left the result is NaN."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

from shared_prefix_checks import DEV, HALF, Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
ids = dict(ids=lambda v: str(v).replace("torch.", ""))
INF = float("inf")


def lowered(c, low=-2000.0):
    """Dim 0 of the queries is positive, so that a key's dim 0 of -inf makes its logit -inf; dim 1 is 1 and every key's
    dim 1 is `low`: all logits lie about low / sqrt(D) * log2(e) below 0, -255 in powers of two at 128 dims."""
    c.q[..., 0] = c.q[..., 0].abs() + 0.25
    c.q[..., 1] = 1.0
    c.k[..., 1] = torch.where(torch.isnan(c.k[..., 1]), c.k[..., 1], torch.full_like(c.k[..., 1], low))
    return c


def drop(c, s, first, last, head):
    """Tokens first .. last - 1 of sequence s: keys of kv-head `head` with -inf in dim 0."""
    t = torch.arange(first, last, device=DEV)
    c.k[c.bt[s].long()[t // c.B], t % c.B, head, 0] = -INF


def check(c, out, rows):
    """out against the definition in 64 bits over the keys whose logit is not -inf.

    As shared_prefix_checks states it: a logit's error is 2 (D + 8) 2^-24 mag, mag the largest sum of |scale q k| of
    those keys; the exponential's 2^-21, sums and joins (2 n + 600) 2^-24; one rounding of the weights to bf16, one of
    the result."""
    half, bf, G = HALF[c.dtype], c.dtype == torch.bfloat16, c.H // c.Hkv
    for s in rows:
        n = c.lens[s]
        blocks = c.bt[s, :-(-n // c.B)].long()
        k, v = (t[blocks].reshape(-1, c.Hkv, c.D)[:n].double().transpose(0, 1) for t in (c.k, c.v))
        q = c.q[s].double().view(c.Hkv, G, c.D)
        for h in range(c.Hkv):
            keep = torch.isfinite(k[h]).all(-1)
            got = out[s].double().view(c.Hkv, G, c.D)[h]
            if not bool(keep.any()):
                assert torch.isnan(got).all(), f"row {s}, kv-head {h}: no key is left"
                continue
            kk, vv = k[h][keep], v[h][keep]
            w = torch.softmax(q[h] @ kk.T * c.scale, -1)
            mag = (q[h].abs() @ kk.abs().T * abs(c.scale)).amax(-1, keepdim=True)
            ref, spread = w @ vv, w @ vv.abs()
            e_w = 2 * (c.D + 8) * 2.0 ** -24 * mag + 2.0 ** -21 + (2 * n + 600) * 2.0 ** -24
            tol = 2 * e_w * spread + half * ref.abs() + (half * spread if bf else 0.0) + 1e-30
            err = (got - ref).abs()
            assert bool((err <= tol).all()), f"row {s}, kv-head {h} ({n} tokens): {float((err / tol).max()):.3g} of the bound"


# H, Hkv, D, B, sequences of the group: two kv-heads at a time, an odd number of kv-heads, more rows than an M-tile,
# a group over several items
SHARED = [(8, 2, 128, 16, 20), (6, 3, 64, 8, 9), (32, 8, 128, 16, 48), (16, 1, 64, 32, 70), (5, 5, 128, 32, 200)]


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B,n", SHARED)
@pytest.mark.parametrize("first,last", [(0, 64), (0, 128), (0, 300), (128, 384), (0, 2047), (0, 2048), (1, 2048), (640, 2048)])
def test_shared_keys(first, last, H, Hkv, D, B, n, dtype):
    """The shared part's first tile, several, tiles in its middle, all of its keys but one, all of them."""
    c = lowered(Case([(n, 2048)], [30, 7, 200], H, Hkv, D, B, dtype, seed=D + n, anchor=True))
    head = Hkv - 1
    drop(c, 0, first, last, head)
    check(c, c.run(), sorted({0, 1, n // 2, n - 1}))


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", [(8, 2, 128, 16), (33, 3, 64, 8), (32, 8, 128, 32), (4, 4, 64, 16)])
def test_own_keys(H, Hkv, D, B, dtype):
    """A sequence's own part: its first keys, its last, all of them; with the shared ones gone too, no key is left."""
    c = lowered(Case([(20, 2048)], [30, 700, 1500], H, Hkv, D, B, dtype, seed=3, anchor=True))
    for s, (a, b) in ((0, (0, 16)), (1, (0, 200)), (2, (0, 1500)), (3, (0, 30)), (4, (16, 700)), (5, (1, 1500))):
        drop(c, s, 2048 + a, 2048 + b, 0)
    check(c, c.run(), range(8))
    drop(c, 0, 0, 2048, 0)
    check(c, c.run(), range(8))


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", [(8, 2, 128, 16), (33, 3, 64, 8), (32, 8, 128, 32), (4, 4, 64, 16)])
@pytest.mark.parametrize("own", [[16, 17, 40], [700, 5000, 33], [20000, 40]])
def test_decode(own, H, Hkv, D, B, dtype):
    """pa.decode: sequences in one piece and in many; units of 16 keys and whole pieces without a finite logit."""
    c = lowered(Case([(2 * len(own), 0)], own, H, Hkv, D, B, dtype, seed=4))
    for i, n in enumerate(own):
        drop(c, i, 0, 16, 0)                         # the first unit
        drop(c, i, n * 2 // 3 // 16 * 16, n - 1, 0)  # whole pieces, up to the last key
        drop(c, len(own) + i, 0, n - 1, Hkv - 1)     # all but the last key
    check(c, pa.decode(c.q, c.k, c.v, c.bt, c.ctx, c.scale), range(c.S))
    drop(c, 0, 0, own[0], 0)
    check(c, pa.decode(c.q, c.k, c.v, c.bt, c.ctx, c.scale), range(c.S))


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("own", [[40], [5000], [20000, 40]])
def test_a_piece_of_nan_logits_stays_nan(own, dtype):
    """Keys that are NaN over whole units and pieces, or everywhere: their rows are NaN, the other kv-head's are not."""
    c = Case([(2 * len(own), 0)], own, 8, 2, 128, 16, dtype, seed=5)
    want = pa.decode(c.q, c.k, c.v, c.bt, c.ctx, c.scale)
    n = own[0]
    for first, last in ((0, 16), (0, n // 2 // 16 * 16), (n // 2 // 16 * 16, n), (0, n)):
        k = c.k.clone()
        t = torch.arange(first, last, device=DEV)
        k[c.bt[0].long()[t // 16], t % 16, 1, 5] = float("nan")
        for out in (pa.decode(c.q, k, c.v, c.bt, c.ctx, c.scale), c.run(k_cache=k)):
            assert torch.isnan(out[0, 4:]).all(), (first, last)
            assert not torch.isnan(out[0, :4]).any() and not torch.isnan(out[1:]).any()
    assert not torch.isnan(want).any()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B,n", SHARED)
def test_shared_keys_that_are_nan(H, Hkv, D, B, n, dtype):
    """Over one tile, several or all: every row of the group is NaN at that kv-head, all others are not."""
    c = Case([(n, 2048), (3, 0)], [30, 7, 200], H, Hkv, D, B, dtype, seed=D + n, anchor=True)
    G = H // Hkv
    for first, last in ((0, 128), (256, 900), (0, 2048)):
        k = c.k.clone()
        t = torch.arange(first, last, device=DEV)
        k[c.bt[0].long()[t // B], t % B, Hkv - 1, 5] = float("nan")
        out = torch.isnan(c.run(k_cache=k))
        assert out[:n, H - G:].all(), (first, last)
        assert not out[:n, :H - G].any() and not out[n:].any()


@pytest.mark.parametrize("H,Hkv,D,B", [(8, 2, 128, 16), (16, 1, 64, 32), (4, 4, 64, 8)])
@pytest.mark.parametrize("cached,rows", [(0, 300), (700, 40), (2000, 257)])
def test_prefill(cached, rows, H, Hkv, D, B):
    """pa.varlen_prefill of one chunk behind `cached` tokens, its first keys without a finite logit."""
    dtype, n = torch.bfloat16, cached + rows
    c = lowered(Case([(1, 0)], [n], H, Hkv, D, B, dtype, seed=6))
    q = torch.randn(rows, H, D, generator=torch.Generator().manual_seed(7)).to(dtype).to(DEV)
    q[..., 0] = q[..., 0].abs() + 0.25
    q[..., 1] = 1.0
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    for last in (128, 256, 301):
        drop(c, 0, 0, min(last, n), 0)
        out = pa.varlen_prefill(q, cu, c.k, c.v, c.bt, c.ctx, c.scale, rows)
        for r in sorted({0, 1, 127, 128, rows - 1} & set(range(rows))):
            row = Case.__new__(Case)
            row.__dict__.update(c.__dict__, q=q[r:r + 1], lens=[cached + r + 1])
            check(row, out[r:r + 1], [0])
