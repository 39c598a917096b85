"""GPU tests of the rotary cache writes at head sizes whose rows do not divide a CTA, and at infinities."""
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
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check_rows(got, ref, mag, dtype, what):
    """One rounding to the type (through fp32), and two roundings of fp32 products and one of their sum."""
    err = np.abs(R.f64(got) - ref)
    tol = HALF[dtype] * (1 + 2 ** -8) * np.abs(ref) + 3 * 2.0 ** -24 * mag
    assert np.all(err <= tol), f"{what}: {float((err - tol).max()):.3e} over the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,H,Hkv,D,rot,inter", [
    (1301, 32, 32, 96, 96, False), (1301, 16, 8, 96, 32, True), (1301, 32, 16, 80, 80, False),
    (1301, 16, 8, 160, 160, False), (1301, 32, 8, 192, 128, False), (1301, 16, 16, 192, 192, True),
    (1301, 32, 16, 112, 112, False), (1301, 32, 16, 48, 48, False), (1301, 9, 4, 240, 16, False),
    (3, 91, 31, 80, 80, False), (3, 69, 20, 112, 48, True)])
def test_rows_that_do_not_divide_a_cta(n, H, Hkv, D, rot, inter, dtype):
    """head_dim / 16 lanes a row, a number that does not divide the threads of a CTA: in long batches (two tokens a
    CTA), and with more rows than one pass of a CTA holds (one token).  Against the formula, and the same bytes as
    calls of 100 tokens give."""
    B = 16
    g = torch.Generator().manual_seed(D + H)
    x = torch.randn(n, (H + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([H * D, Hkv * D, Hkv * D], 1))
    rng = np.random.default_rng(D)
    nb = n // B + 3
    slots = torch.from_numpy(rng.permutation(nb * B)[:n].astype(np.int64)).to(DEV)
    p = rng.integers(0, 2000, n).astype(np.int32)
    pos, tab = torch.from_numpy(p).to(DEV), R.table(2000, rot).to(DEV)

    def run(step):
        kc = torch.full((nb, B, Hkv, D), 5.0, dtype=dtype, device=DEV)
        vc, out = torch.full_like(kc, 6.0), torch.full((n, H, D), 9.0, dtype=dtype, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        for i in range(0, n, step):
            j = slice(i, i + step)
            pa.rope_and_cache(q[j], k[j], v[j], tab, pos[j], kc, vc, slots[j], interleaved=inter, q_out=out[j],
                              dev_status=st)
        assert pa.get_device_status(st) == 0
        return kc, vc, out
    a, b = run(n), run(100)
    for s, t in zip(a, b):
        assert torch.equal(bits(s), bits(t))
    check_rows(a[2], *R.rotate(q, tab, p, rot, inter), dtype, "q_out")
    check_rows(a[0].view(nb * B, Hkv, D)[slots], *R.rotate(k, tab, p, rot, inter), dtype, "k_cache")
    assert torch.equal(a[1].view(nb * B, Hkv, D)[slots], v)
