"""4-bit decode with queries over the whole range of their type, and with logits past the usual."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R
from q4_decode_checks import check
from test_gpu_decode_q4 import Case, _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def refill(c, factor, seed=7):
    """Pools anew: K ~ N(0, 1) factor, V ~ N(0, 1)."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(c.nb, c.B, c.Hkv, c.D, generator=g).to(DEV) for _ in "kv")
    ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
    pa.quantize_blocks_q4(k * factor, v, c.k4, c.v4, ident)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D", [(8, 128), (32, 64)])
@pytest.mark.parametrize("e", [-118, -100, 100, 118, 121, 124])
def test_queries_and_keys_of_opposite_size(e, H, D, dtype):
    """q 2^e over K 2^-e: ordinary logits."""
    c = Case([40, 500], H, 2, D, 16, dtype, seed=81)
    refill(c, 2.0 ** -e)
    c.q *= 2.0 ** e
    check(c, c.run(), what=f"2^{e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [-124, -110, 0, 110, 123])
def test_keys_along_the_query(e, dtype):
    """Keys of the queries' signs: every product of a row adds to the one sum, and the codes are the largest."""
    c = Case([40, 500], 2, 2, 128, 16, dtype, seed=86)
    c.q[:] = c.q[0]
    c.q *= 2.0 ** e
    g = torch.Generator().manual_seed(87)
    size = 0.7 + 0.3 * torch.rand(c.nb, 16, 2, 1, generator=g).to(DEV)
    k = torch.sign(c.q[0].float()) * size * 2.0 ** -e
    v = torch.randn(c.nb, 16, 2, 128, generator=g).to(DEV)
    ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
    pa.quantize_blocks_q4(k, v, c.k4, c.v4, ident)
    check(c, c.run(), what=f"2^{e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_heads_of_all_sizes_side_by_side(dtype):
    """Heads of one kv-head whose queries differ by powers of two up to 2^224: logits from nothing to several units."""
    c = Case([300], 8, 1, 128, 16, dtype, seed=82)
    refill(c, 2.0 ** -122)
    c.q *= torch.exp2(torch.tensor([122.0, 0.0, 121.0, -100.0, 118.0, 110.0, 124.0, 60.0], device=DEV))[None, :, None].to(dtype)
    check(c, c.run(), what="mixed")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [30, 60, 110, 121])
def test_huge_logits_take_the_largest_one(e, dtype):
    """Logits of 2^e: one token takes all the weight (they lie 2^e 2^-24 apart at least, or they are the same)."""
    ctx = [1, 40, 300, 900]
    c = Case(ctx, 8, 2, 128, 16, dtype, seed=83)
    refill(c, 1.0)
    c.q *= 2.0 ** e
    out = c.run()
    assert torch.isfinite(out).all()
    k, v = R.values(c.k4, "k", 16, 128), R.values(c.v4, "v", 16, 128)
    seen = 0
    for s, n in enumerate(ctx):
        ids = c.bt[s, :-(-n // 16)].cpu().numpy()
        kr, vr = k[ids].reshape(-1, 2, 128)[:n], v[ids].reshape(-1, 2, 128)[:n]
        for h in range(8):
            x = kr[:, h // 4] @ R.f64(c.q[s, h])
            top = np.argsort(x)[::-1]
            # a sum's error: 16 fp32 steps of five times the products' magnitudes, as in the other tests
            far = 2 * 5 * 16 * 2.0 ** -23 * (np.abs(kr[:, h // 4]) @ np.abs(R.f64(c.q[s, h]))).max()
            if n > 1 and x[top[0]] - x[top[1]] < far + 2.0 ** 12:
                continue
            seen += 1
            want = torch.from_numpy(vr[top[0], h // 4]).to(dtype)   # (n - 8) s, rounded once
            assert torch.equal(out[s, h].cpu(), want), (s, h)
    assert seen >= 24


@pytest.mark.parametrize("D", [64, 128])
def test_small_elements_beside_a_large_one(D):
    """bf16 queries are held in fp16: elements 2^-30 of the head's largest are exact in the dims 0, 2, 4, 6 (mod 8) and
    2^-26 of it in the others.  The large element meets keys of zero, so the small ones decide."""
    c = Case([40, 500], 8, 2, D, 16, torch.bfloat16, seed=84)
    g = torch.Generator().manual_seed(85)
    k, v = (torch.randn(c.nb, 16, 2, D, generator=g).to(DEV) for _ in "kv")
    k[..., :32] = 0                                     # group 0: scale 0
    ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
    pa.quantize_blocks_q4(k, v, c.k4, c.v4, ident)
    for odd in (0, 1):
        q = torch.zeros(2, 8, D, device=DEV)
        small = torch.randn(2, 8, D // 2, generator=g).clamp(-2, 2).to(DEV)
        small = torch.where(small.abs() < 1, torch.copysign(torch.ones_like(small), small), small)   # 1 .. 2
        q[..., odd::2] = small.bfloat16().float() * 2.0 ** (-26 if odd else -30)
        q[..., :32] = 0
        q[..., 5] = 1.0
        c.q = q.bfloat16()
        c.scale = 0.1 * 2.0 ** (26 if odd else 30)
        check(c, c.run(), what=f"odd {odd}", exact_q=True)
