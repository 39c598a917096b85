"""Argument checks of the rotary cache writes with several position axes: returned before any launch, so they run
without a GPU."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import build as B
from pagedattention_kv_cache_reshape_gb300 import pa

INV, UNS = pa.ERR_INVALID_ARG, pa.ERR_UNSUPPORTED

# addresses that are never read: the calls below return before a launch
ARGS = dict(q_out=1 << 30, q=2 << 30, key=3 << 30, value=4 << 30, qs=4096, ks=1024, vs=1024, cs=5 << 30, pos=6 << 30,
            pstride=16, axis=10 << 30, axes=3, max_pos=4096, rot=128, inter=0, k=7 << 30, v=8 << 30, slot=9 << 30, n=16,
            h=32, hkv=8, d=128, b=16, nb=64, dt=pa.DTYPE_BF16, st=None, stream=None)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pa.load()


def mrope(lib, q4=False, **kw):
    return (lib.pa_mrope_and_cache_q4 if q4 else lib.pa_mrope_and_cache)(*{**ARGS, **kw}.values())


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(axes=0), INV), (dict(axes=-1), INV), (dict(axes=5), UNS), (dict(pstride=-1), INV), (dict(axis=None), INV),
    (dict(axis=(10 << 30) + 2), INV), (dict(pos=None), INV), (dict(cs=None), INV), (dict(pos=(6 << 30) + 1), INV),
    (dict(rot=3), INV), (dict(rot=130), INV), (dict(max_pos=0), INV), (dict(ks=1023), INV), (dict(dt=9), INV),
    (dict(q_out=(2 << 30) + 64), INV), (dict(n=-1), INV),
    (dict(n=0, axes=5), UNS), (dict(n=0, pos=None, axis=None, cs=None, key=None), pa.OK),
])
def test_mrope_refuses(lib, q4, kw, want):
    assert mrope(lib, q4, **kw) == want


def test_mrope_shapes_of_the_4_bit_pools(lib):
    assert mrope(lib, True, d=96, rot=96) == UNS
    assert mrope(lib, True, b=24) == UNS


class NoLaunch:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,error", [
    (dict(positions=torch.zeros(3, dtype=torch.int32)), "axes, tokens"),
    (dict(positions=torch.zeros(3, 2, dtype=torch.int32)), "entry per token"),
    (dict(positions=torch.zeros(4, 3, dtype=torch.int32).T), "contiguous along"),
    (dict(positions=torch.zeros(3, 4, dtype=torch.int64)), "positions must be torch.int32"),
    (dict(pair_axis=torch.zeros(63, dtype=torch.int32)), "pair_axis"),
    (dict(pair_axis=torch.zeros(64, 1, dtype=torch.int32)), "pair_axis"),
    (dict(pair_axis=torch.zeros(64, dtype=torch.int64)), "pair_axis must be torch.int32"),
    (dict(pair_axis=torch.zeros(128, dtype=torch.int32)[::2]), "pair_axis must be contiguous"),
    (dict(pair_axis=None), "are needed"), (dict(positions=None), "are needed"), (dict(cos_sin=None), "are needed"),
    (dict(cos_sin=torch.zeros(9, 128).double()), "cos_sin"), (dict(slot_mapping=torch.zeros(3, dtype=torch.int64)), "slot"),
])
def test_the_binding_refuses(q4, kw, error, monkeypatch):
    """torch gives CPU tensors the device number -1, which stands in for the current device; a launch fails the test."""
    B.build()
    pa.load()
    monkeypatch.setattr(pa, "_lib", NoLaunch())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(pa, "_refuse", lambda dev, *specs: _check(specs))
    shape, dtype = ((4, 2, 16 * 72), torch.uint8) if q4 else ((4, 16, 2, 128), torch.bfloat16)
    pools = [torch.zeros(shape, dtype=dtype) for _ in "kv"]
    args = dict(q=None, key=torch.zeros(4, 2, 128).bfloat16(), value=torch.zeros(4, 2, 128).bfloat16(),
                cos_sin=torch.zeros(9, 128), positions=torch.zeros(3, 4, dtype=torch.int32),
                pair_axis=torch.zeros(64, dtype=torch.int32), k_cache=pools[0], v_cache=pools[1],
                slot_mapping=torch.zeros(4, dtype=torch.int64))
    with pytest.raises((ValueError, TypeError), match=error):
        (pa.mrope_and_cache_q4 if q4 else pa.mrope_and_cache)(**{**args, **kw})


def _check(specs):
    """_refuse without its checks of the device, which CPU tensors never pass."""
    for t, name, dtype in specs:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
