"""What the Python binding of the rotary and 4-bit calls refuses before the library is called.  Without a GPU: torch
gives CPU tensors the device number -1, which stands in for the current device here, and a launch would fail the test."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import build as B
from pagedattention_kv_cache_reshape_gb300 import pa


class NoLaunch:
    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(self.lib, name)

        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def _stand_in(monkeypatch):
    B.build()
    lib = pa.load()
    monkeypatch.setattr(pa, "_lib", NoLaunch(lib))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)


def rows(n, h, d=128):
    return torch.zeros(n, h, d, dtype=torch.bfloat16)


def wide():
    return [torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16) for _ in "kv"]


def q4():
    return [torch.zeros(4, 2, 16 * 72, dtype=torch.uint8) for _ in "kv"]


@pytest.mark.parametrize("call,pools", [("rope_and_cache", wide), ("rope_and_cache_q4", q4)])
def test_a_table_without_positions_is_refused(call, pools):
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="positions"):
        getattr(pa, call)(None, rows(3, 2), rows(3, 2), torch.zeros(9, 128), None, *pools(), slots)


class Elsewhere:
    """A status word on another GPU."""
    is_cuda, dtype, device = True, torch.int32, "cuda:1"

    def get_device(self):
        return 1

    def data_ptr(self):
        raise AssertionError("its address was taken")


def status_calls():
    pairs = torch.zeros(1, 2, dtype=torch.int32)
    slots, pos, tab = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), torch.zeros(9, 128)
    bt, ctx = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    ws = torch.zeros(pa.decode_q4_workspace_size(3, 4, 2, 128, 16, 1), dtype=torch.uint8)
    return {
        "rope_and_cache": lambda st: pa.rope_and_cache(None, rows(3, 2), rows(3, 2), tab, pos, *wide(), slots, dev_status=st),
        "rope_and_cache_q4": lambda st: pa.rope_and_cache_q4(None, rows(3, 2), rows(3, 2), tab, pos, *q4(), slots,
                                                             dev_status=st),
        "quantize_blocks_q4": lambda st: pa.quantize_blocks_q4(*wide(), *q4(), pairs, dev_status=st),
        "dequantize_blocks_q4": lambda st: pa.dequantize_blocks_q4(*q4(), *wide(), pairs, dev_status=st),
        "decode_q4": lambda st: pa.decode_q4(rows(3, 4), *q4(), bt, ctx, 0.1, out=rows(3, 4), workspace=ws, dev_status=st),
    }


@pytest.mark.parametrize("name", ["rope_and_cache", "rope_and_cache_q4", "quantize_blocks_q4", "dequantize_blocks_q4",
                                  "decode_q4"])
def test_a_status_word_on_another_device_is_refused(name):
    with pytest.raises(ValueError, match="dev_status"):
        status_calls()[name](Elsewhere())
