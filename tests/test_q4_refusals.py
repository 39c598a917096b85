"""Argument checks of the rotary and 4-bit cache calls: returned before any launch, so they run without a GPU."""
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
ROPE = dict(q_out=1 << 30, q=2 << 30, key=3 << 30, value=4 << 30, qs=4096, ks=1024, vs=1024, cs=5 << 30, pos=6 << 30,
            max_pos=4096, rot=128, inter=0, k=7 << 30, v=8 << 30, slot=9 << 30, n=16, h=32, hkv=8, d=128, b=16, nb=64,
            dt=pa.DTYPE_BF16, st=None, stream=None)


def rope(lib, q4=False, **kw):
    return (lib.pa_rope_and_cache_q4 if q4 else lib.pa_rope_and_cache)(*{**ROPE, **kw}.values())


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw", [
    dict(dt=7), dict(n=-1), dict(h=-1), dict(hkv=0), dict(d=0), dict(b=0), dict(nb=0), dict(rot=-2), dict(rot=3),
    dict(rot=130), dict(max_pos=0), dict(inter=2), dict(inter=-1), dict(ks=1023), dict(vs=1023), dict(qs=4095),
    dict(key=None), dict(value=None), dict(k=None), dict(v=None), dict(slot=None), dict(q=None), dict(q_out=None),
    dict(cs=None), dict(pos=None), dict(key=(3 << 30) + 1), dict(k=(7 << 30) + 1), dict(cs=(5 << 30) + 2),
    dict(pos=(6 << 30) + 1), dict(slot=(9 << 30) + 4), dict(q=(2 << 30) + 1), dict(q_out=(1 << 30) + 1),
    dict(q_out=(2 << 30) + 64),                          # half on q
    dict(q_out=2 << 30, qs=6144),                        # on q, whose rows are not contiguous
    dict(q_out=(3 << 30) - 64), dict(q_out=(4 << 30) + 1024),   # on key, on value
])
def test_rope_refuses(lib, q4, kw):
    assert rope(lib, q4, **kw) == INV


def test_rope_shapes_of_the_4_bit_pools(lib):
    assert rope(lib, True, d=96, rot=96) == UNS
    assert rope(lib, True, b=24) == UNS
    assert rope(lib, True, k=(7 << 30) + 8) == INV       # 4-bit pools start on 16 bytes


@pytest.mark.parametrize("q4", [False, True])
def test_rope_of_no_tokens_does_nothing(lib, q4):
    assert rope(lib, q4, n=0, key=None, value=None, q=None, q_out=None, k=None, v=None, slot=None, pos=None,
                cs=None) == pa.OK
    assert rope(lib, q4, n=0, rot=5) == INV              # shape checks come first


BLK = dict(sk=1 << 30, sv=2 << 30, dk=3 << 30, dv=4 << 30, b=16, hkv=8, d=128, ns=9, nd=9, pairs=5 << 30, n=3,
           dt=pa.DTYPE_BF16, st=None, stream=None)


@pytest.mark.parametrize("fn", ["pa_quantize_blocks_q4", "pa_dequantize_blocks_q4"])
@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), INV), (dict(n=-1), INV), (dict(ns=-1), INV), (dict(nd=-1), INV), (dict(hkv=0), INV),
    (dict(d=0), INV), (dict(b=0), INV), (dict(b=4), UNS), (dict(b=64), UNS), (dict(d=32), UNS), (dict(d=256), UNS),
    (dict(sk=None), INV), (dict(sv=None), INV), (dict(dk=None), INV), (dict(dv=None), INV), (dict(pairs=None), INV),
    (dict(sk=(1 << 30) + 8), INV), (dict(dv=(4 << 30) + 2), INV), (dict(pairs=(5 << 30) + 2), INV),
    (dict(n=0, sk=None, sv=None, dk=None, dv=None, pairs=None), pa.OK),
])
def test_block_conversion_refuses(lib, fn, kw, want):
    assert getattr(lib, fn)(*{**BLK, **kw}.values()) == want


DEC = dict(out=1 << 30, q=2 << 30, k=3 << 30, v=4 << 30, bt=5 << 30, ctx=6 << 30, n=2, h=8, hkv=4, d=128, b=16, mb=4,
           nb=8, scale=ctypes.c_float(0.1), dt=pa.DTYPE_BF16, ws=7 << 30, wsb=1 << 40, st=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(h=6), INV), (dict(h=0), INV), (dict(mb=0), INV), (dict(nb=0), INV), (dict(dt=3), INV),
    (dict(scale=ctypes.c_float(float("nan"))), INV), (dict(d=96), UNS), (dict(b=4), UNS), (dict(b=64), UNS),
    (dict(h=4 * 33), UNS), (dict(out=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(bt=None), INV), (dict(ctx=None), INV), (dict(q=(2 << 30) + 1), INV), (dict(k=(3 << 30) + 8), INV),
    (dict(v=(4 << 30) + 2), INV), (dict(bt=(5 << 30) + 1), INV), (dict(ws=None), WS), (dict(ws=(7 << 30) + 8), WS),
    (dict(wsb=0), WS), (dict(mb=1 << 28), INV),
    (dict(n=0, out=None, q=None, k=None, v=None, bt=None, ctx=None, ws=None, wsb=0), pa.OK),
])
def test_decode_q4_refuses(lib, kw, want):
    assert lib.pa_decode_q4(*{**DEC, **kw}.values()) == want


def test_decode_q4_wants_its_whole_workspace(lib):
    need = pa.decode_q4_workspace_size(2, 8, 4, 128, 16, 4)
    assert need > 0
    assert lib.pa_decode_q4(*{**DEC, "wsb": need - 1}.values()) == WS


def test_q4_block_bytes(lib):
    for b in (8, 16, 32):
        for h in (1, 5, 32):
            for d in (64, 128):
                assert pa.q4_block_bytes(b, h, d) == b * h * d * 9 // 16
    assert pa.q4_block_bytes(4, 1, 64) == -1 and pa.q4_block_bytes(16, 0, 64) == -1
    assert pa.q4_block_bytes(16, 1, 96) == -1


def test_binding_refuses_wrong_tensors(lib):
    pool = torch.zeros(4, 2, 16 * 72, dtype=torch.uint8)
    q = torch.zeros(3, 4, 128)
    with pytest.raises(ValueError):
        pa.decode_q4(q, pool[:, :, :1000], pool[:, :, :1000], torch.zeros(3, 1, dtype=torch.int32),
                     torch.ones(3, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        pa.decode_q4(q, pool, pool[:2], torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        pa.rope_and_cache_q4(None, torch.zeros(3, 4, 128), torch.zeros(3, 4, 128), None, None, pool, pool,
                             torch.zeros(3, dtype=torch.int64))
    wide = torch.zeros(4, 16, 2, 128)
    with pytest.raises(ValueError):
        pa.rope_and_cache(None, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), None, None, wide, wide,
                          torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        pa.rope_and_cache(None, torch.zeros(3, 2, 128).bfloat16(), torch.zeros(3, 2, 128).bfloat16(), None, None, wide,
                          wide, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        pa.quantize_blocks_q4(wide, wide, pool[:, :1], pool[:, :1], torch.zeros(1, 2, dtype=torch.int32))
