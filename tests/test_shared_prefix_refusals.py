"""Argument checks of the shared-prefix decode: returned before any launch, so they run without a GPU."""
import ctypes

import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import build as B
from pagedattention_kv_cache_reshape_gb300 import pa

INV, UNS, WS = pa.ERR_INVALID_ARG, pa.ERR_UNSUPPORTED, pa.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pa.load()


# addresses that are never read: the calls below return before a launch
ARGS = dict(out=1 << 30, q=2 << 30, k=3 << 30, v=4 << 30, bt=5 << 30, ctx=6 << 30, starts=7 << 30, prefix=8 << 30, n=6,
            groups=2, h=8, hkv=4, d=128, b=16, mb=4, nb=8, scale=ctypes.c_float(0.1), dt=pa.DTYPE_BF16, ws=9 << 30,
            wsb=1 << 40, st=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(groups=-1), INV), (dict(groups=0), INV), (dict(h=6), INV), (dict(h=0), INV),
    (dict(mb=0), INV), (dict(nb=0), INV), (dict(dt=3), INV), (dict(scale=ctypes.c_float(float("nan"))), INV),
    (dict(d=96), UNS), (dict(b=4), UNS), (dict(b=64), UNS), (dict(h=4 * 33), UNS), (dict(out=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(bt=None), INV), (dict(ctx=None), INV),
    (dict(starts=None), INV), (dict(prefix=None), INV), (dict(q=(2 << 30) + 1), INV), (dict(k=(3 << 30) + 1), INV),
    (dict(bt=(5 << 30) + 1), INV), (dict(ctx=(6 << 30) + 2), INV), (dict(starts=(7 << 30) + 2), INV),
    (dict(prefix=(8 << 30) + 3), INV), (dict(ws=None), WS), (dict(ws=(9 << 30) + 8), WS), (dict(wsb=0), WS),
    (dict(mb=1 << 28), INV), (dict(mb=(1 << 27) - 8), UNS), (dict(n=1 << 28), UNS), (dict(groups=1 << 28), UNS),
    (dict(n=0, groups=0, out=None, q=None, k=None, v=None, bt=None, ctx=None, starts=None, prefix=None, ws=None, wsb=0), pa.OK),
    (dict(n=0, groups=-1), INV),
])
def test_decode_shared_prefix_refuses(lib, kw, want):
    assert lib.pa_decode_shared_prefix(*{**ARGS, **kw}.values()) == want


@pytest.mark.parametrize("dt", [pa.DTYPE_BF16, pa.DTYPE_F32])
def test_it_wants_its_whole_workspace(lib, dt):
    need = pa.decode_shared_prefix_workspace_size(6, 2, 8, 4, 128, 16, 4)
    assert need > 0 and pa.decode_shared_prefix_workspace_size(0, 0, 0, 0, 0, 0, 0) > 0
    assert pa.decode_shared_prefix_workspace_size(-1, -1, -1, -1, -1, -1, -1) > 0
    assert lib.pa_decode_shared_prefix(*{**ARGS, "wsb": need - 1, "dt": dt}.values()) == WS


class NoLaunch:
    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(self.lib, name)

        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


i32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("kw,error", [
    (dict(v_cache=torch.zeros(4, 16, 2, 64).bfloat16()), "pools"), (dict(k_cache=torch.zeros(4, 16, 128).bfloat16()), "pools"),
    (dict(block_tables=torch.zeros(3, 2, **i32)), "a row per sequence"), (dict(context_lens=torch.zeros(3, **i32)), "a row per"),
    (dict(group_starts=torch.zeros(2, **i32)), "one entry more"), (dict(prefix_lens=torch.zeros(3, **i32)), "one entry more"),
    (dict(q=torch.zeros(4, 4, 128).half()), "unsupported dtype"), (dict(out=torch.zeros(4, 4, 64).bfloat16()), "out must"),
    (dict(k_cache=torch.zeros(4, 16, 2, 128)), "k_cache"), (dict(group_starts=torch.zeros(3)), "group_starts"),
    (dict(prefix_lens=torch.zeros(2, dtype=torch.int64)), "prefix_lens"),
    (dict(group_starts=torch.zeros(6, **i32)[::2]), "group_starts"),
])
def test_the_binding_refuses(lib, kw, error, monkeypatch):
    """torch gives CPU tensors the device number -1, which stands in for the current device; a launch fails the test."""
    monkeypatch.setattr(pa, "_lib", NoLaunch(lib))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)

    def refuse(dev, *specs):
        for t, name, dtype in specs:
            if not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
                raise ValueError(name)
    monkeypatch.setattr(pa, "_refuse", refuse)
    pool = torch.zeros(4, 16, 2, 128).bfloat16()
    args = dict(q=torch.zeros(4, 4, 128).bfloat16(), k_cache=pool, v_cache=pool, block_tables=torch.zeros(4, 2, **i32),
                context_lens=torch.zeros(4, **i32), group_starts=torch.zeros(3, **i32), prefix_lens=torch.zeros(2, **i32),
                scale=0.1)
    with pytest.raises((ValueError, TypeError), match=error):
        pa.decode_shared_prefix(**{**args, **kw})


def test_tensors_off_the_current_device_are_refused(lib, monkeypatch):
    monkeypatch.setattr(pa, "_lib", NoLaunch(lib))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    pool = torch.zeros(4, 16, 2, 128).bfloat16()
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.decode_shared_prefix(torch.zeros(4, 4, 128).bfloat16(), pool, pool, torch.zeros(4, 2, **i32),
                                torch.zeros(4, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32), 0.1)
