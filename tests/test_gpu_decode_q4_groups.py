"""4-bit decode where the groups of V's dims differ in size: no group's weights depend on another's scales."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

from q4_decode_checks import check
from test_gpu_decode_q4 import Case, _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def refill(c, exps):
    """Pools anew: K ~ N(0, 1), V ~ N(0, 1) 2^exps, exps broadcast against [blocks, B, heads, D / 32]."""
    g = torch.Generator().manual_seed(7)
    k = torch.randn(c.nb, c.B, c.Hkv, c.D, generator=g).to(DEV)
    v = torch.randn(c.nb, c.B, c.Hkv, c.D, generator=g).to(DEV)
    v = (v.unflatten(3, (-1, 32)) * torch.exp2(exps.to(DEV).float())[..., None]).flatten(3)
    ident = torch.arange(c.nb, dtype=torch.int32, device=DEV)[:, None].repeat(1, 2).contiguous()
    pa.quantize_blocks_q4(k, v, c.k4, c.v4, ident)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctx,H,Hkv,D,B,exps", [
    ([700], 8, 2, 128, 16, (0, -24, -28, -32)), ([700], 8, 2, 128, 16, (-32, -28, -24, 0)),
    ([5, 300, 4097], 4, 1, 64, 8, (20, -20)), ([5, 300, 4097], 4, 1, 64, 32, (-32, 0)),
    ([3000, 17], 16, 1, 128, 16, (0, -40, 40, -90)), ([20000], 4, 1, 128, 16, (-30, 0, 0, -60)),
    ([20000], 32, 1, 64, 16, (0, -30)), ([100] * 80, 8, 8, 64, 16, (0, -32)), ([33], 8, 8, 128, 8, (-90, 90, -60, 3))],
    ids=str)
def test_groups_of_v_far_apart(ctx, H, Hkv, D, B, exps, dtype):
    c = Case(ctx, H, Hkv, D, B, dtype, seed=71)
    refill(c, torch.tensor(exps))
    check(c, c.run(), what=str(exps))


def test_groups_at_the_ends_of_the_range():
    c = Case([33, 3], 8, 8, 128, 8, torch.bfloat16, seed=75)
    refill(c, torch.tensor([-118, 100, 0, 3]))
    check(c, c.run(), what="ends")


@pytest.mark.parametrize("H,Hkv", [(8, 2), (16, 1)])
def test_groups_that_rise_and_fall_along_the_sequence(H, Hkv):
    """Scales over forty powers of two, two groups rising along the sequence and two falling."""
    n, B = 700, 16
    c = Case([n], H, Hkv, 128, B, torch.bfloat16, seed=72)
    at = torch.zeros(c.nb, B, 1, 4)
    t = torch.zeros(44 * B)
    t[:n] = torch.linspace(-20.0, 20.0, n)
    at[c.bt[0, :44].long().cpu()] = t.view(44, B, 1, 1) * torch.tensor([1.0, -1.0, -1.0, 1.0])
    refill(c, at)
    check(c, c.run(), what="rising and falling")


def test_a_group_of_zeros_stays_zero():
    c = Case([5, 700], 8, 2, 128, 16, torch.bfloat16, seed=73)
    refill(c, torch.tensor([0.0, float("-inf"), -30.0, float("-inf")]))
    out = c.run()
    check(c, out, what="zeros")
    z = out.view(2, 8, 4, 32)
    assert not z[:, :, 1].any() and not z[:, :, 3].any()


def test_a_nan_scale_stays_in_its_group():
    c = Case([90], 4, 2, 128, 16, torch.bfloat16, seed=74)
    exps = torch.tensor([0.0, -30.0, 3.0, -12.0])
    refill(c, exps)
    ref = c.run()
    at = 16 * 64 + 3 * 8 + 2 * 2                       # token 3, group 2
    c.v4[int(c.bt[0, 2]), 0, at:at + 2] = 0xff
    out, ref = c.run().view(4, 4, 32).float(), ref.view(4, 4, 32).float()
    assert torch.isnan(out[:2, 2]).all() and torch.equal(out[2:], ref[2:])
    for g in (0, 1, 3):   # the reference of the weights may have moved elsewhere: roundings of weights and result
        assert torch.allclose(out[:2, g], ref[:2, g], rtol=2.0 ** -7, atol=1e-3 * 2.0 ** float(exps[g]))
