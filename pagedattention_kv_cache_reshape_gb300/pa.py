"""Thin Python binding of the C ABI in include/pa.h (ctypes).

Argument marshalling only: torch tensors supply device pointers, the current
CUDA stream supplies the stream, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback: if ``libpa.so`` is missing
or a call fails, an exception is raised.

The functions keep the C names without the ``pa_`` prefix.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_OUT_OF_RANGE, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(7)
DTYPE_F32, DTYPE_BF16 = 0, 1

EXPORTS = (
    "pa_status_string", "pa_version", "pa_num_blocks_needed", "pa_compute_slot_mapping",
    "pa_reshape_and_cache", "pa_decode_workspace_size", "pa_decode",
    "pa_varlen_prefill_workspace_size", "pa_varlen_prefill", "pa_get_device_status",
    "pa_reset_device_status", "pa_set_timing_events", "pa_decode_static_scratch", "pa_decode_step",
    "pa_copy_blocks", "pa_varlen_encode", "pa_varlen_step",
    "pa_block_manager_create", "pa_block_manager_destroy", "pa_block_manager_num_free",
    "pa_block_manager_refcount", "pa_allocate_slots", "pa_free_sequence", "pa_share_prefix",
    "pa_block_manager_tables", "pa_validate_inputs", "pa_allocate_slots_batch", "pa_set_wait_test",
    "pa_rope_and_cache", "pa_q4_block_bytes", "pa_rope_and_cache_q4", "pa_quantize_blocks_q4",
    "pa_dequantize_blocks_q4", "pa_decode_q4_workspace_size", "pa_decode_q4",
)
STATIC_SCRATCH_BYTES = 24 << 20
STALL_NONE, STALL_PRODUCER, STALL_CONSUMER = 0, 1, 2
WAIT_DECODE_PRODUCER, WAIT_DECODE_CONSUMER = 1, 2
WAIT_PREFILL_PRODUCER, WAIT_PREFILL_MMA, WAIT_PREFILL_SOFTMAX = 4, 8, 16


class PAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libpa.so (built by __graft_entry__.build() or build.py)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build the CUDA library first "
                              "(python -m pagedattention_kv_cache_reshape_gb300.build)")
        L = ctypes.CDLL(path)
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_status_string.argtypes = [i32]
        L.pa_version.restype = i32
        L.pa_num_blocks_needed.restype = i32
        L.pa_num_blocks_needed.argtypes = [i32, i32]
        L.pa_compute_slot_mapping.restype = i32
        L.pa_compute_slot_mapping.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp]
        L.pa_reshape_and_cache.restype = i32
        L.pa_reshape_and_cache.argtypes = [vp, vp, i64, i64, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
        L.pa_decode_workspace_size.restype = sz
        L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.pa_decode.restype = i32
        L.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                vp, sz, vp, vp]
        L.pa_varlen_prefill_workspace_size.restype = sz
        L.pa_varlen_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.pa_varlen_prefill.restype = i32
        L.pa_varlen_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                        i32, i32, f32, i32, vp, sz, vp, vp]
        L.pa_block_manager_create.restype = vp
        L.pa_block_manager_create.argtypes = [i32, i32, i32]
        L.pa_block_manager_destroy.restype = None
        L.pa_block_manager_destroy.argtypes = [vp]
        L.pa_block_manager_num_free.restype = i32
        L.pa_block_manager_num_free.argtypes = [vp]
        L.pa_block_manager_refcount.restype = i32
        L.pa_block_manager_refcount.argtypes = [vp, i32]
        L.pa_allocate_slots.restype = i32
        L.pa_allocate_slots.argtypes = [vp, i64, i32]
        L.pa_allocate_slots_batch.restype = i32
        L.pa_allocate_slots_batch.argtypes = [vp, vp, vp, i32, vp]
        L.pa_free_sequence.restype = i32
        L.pa_free_sequence.argtypes = [vp, i64]
        L.pa_share_prefix.restype = i32
        L.pa_share_prefix.argtypes = [vp, i64, i64, i32]
        L.pa_block_manager_tables.restype = i32
        L.pa_block_manager_tables.argtypes = [vp, vp, i32, vp, i32, vp]
        L.pa_varlen_encode.restype = i32
        L.pa_varlen_encode.argtypes = L.pa_varlen_prefill.argtypes
        L.pa_get_device_status.restype = i32
        L.pa_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
        L.pa_reset_device_status.restype = i32
        L.pa_reset_device_status.argtypes = [vp, vp]
        L.pa_set_timing_events.restype = i32
        L.pa_set_timing_events.argtypes = [vp, vp]
        L.pa_set_wait_test.restype = i32
        L.pa_set_wait_test.argtypes = [ctypes.c_uint64, i32, i32, vp]
        L.pa_copy_blocks.restype = i32
        L.pa_copy_blocks.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp, i32, vp, vp]
        L.pa_decode_step.restype = i32
        L.pa_decode_step.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32,
                                     i32, i32, i32, i32, f32, i32, vp, sz, vp, vp]
        L.pa_varlen_step.restype = i32
        L.pa_varlen_step.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                     i32, i32, i32, i32, i32, f32, i32, vp, sz, vp, vp]
        L.pa_decode_static_scratch.restype = i32
        L.pa_decode_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                               f32, i32, vp, vp]
        L.pa_rope_and_cache.restype = i32
        L.pa_rope_and_cache.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, i32, i32, i32, vp, vp, vp, i32, i32,
                                        i32, i32, i32, i32, i32, vp, vp]
        L.pa_rope_and_cache_q4.restype = i32
        L.pa_rope_and_cache_q4.argtypes = L.pa_rope_and_cache.argtypes
        L.pa_q4_block_bytes.restype = i64
        L.pa_q4_block_bytes.argtypes = [i32, i32, i32]
        L.pa_quantize_blocks_q4.restype = i32
        L.pa_quantize_blocks_q4.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, i32, vp, vp]
        L.pa_dequantize_blocks_q4.restype = i32
        L.pa_dequantize_blocks_q4.argtypes = L.pa_quantize_blocks_q4.argtypes
        L.pa_decode_q4_workspace_size.restype = sz
        L.pa_decode_q4_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.pa_decode_q4.restype = i32
        L.pa_decode_q4.argtypes = L.pa_decode.argtypes
        L.pa_validate_inputs.restype = i32
        L.pa_validate_inputs.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_int64)]
        _lib = L
        return L


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise PAError(rc, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream) -> int:
    if stream is None:   # the current stream's handle, no torch.cuda.Stream is made
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream, result: bool = False):
    """Memory that a call on `stream` makes itself.  torch's allocator hands freed memory out again in the order of the
    stream that it was taken on, so it is taken on the call's own stream.  A result is also marked as used by the
    current stream, where the caller may read it (after waiting for `stream`)."""
    if stream is None or device.type != "cuda":   # (tensors off the GPU are refused before the launch)
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    handle = _stream(stream)
    if handle == here.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):   # 0 and 1 are names of the default stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(here)
    return t


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _contig(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _dev(t, name, dtype)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _opt(t) -> int:
    return 0 if t is None else _dev(t, "dev_status", torch.int32)


# ------------------------------------------------------------------ calls

def version() -> int:
    return int(load().pa_version())


def num_blocks_needed(num_tokens: int, block_size: int) -> int:
    return int(load().pa_num_blocks_needed(int(num_tokens), int(block_size)))


def compute_slot_mapping(block_tables, seq_start, cu_seqlens_q, num_blocks: int, total_new: int,
                         block_size: int = 16, slot_mapping=None, dev_status=None, stream=None):
    """pa_compute_slot_mapping; returns the int64 slot_mapping tensor."""
    num_seqs, max_blocks = block_tables.shape
    if slot_mapping is None:
        slot_mapping = _empty(total_new, torch.int64, block_tables.device, stream, result=True)
    rc = load().pa_compute_slot_mapping(
        _contig(block_tables, "block_tables", torch.int32), num_seqs, max_blocks,
        _contig(seq_start, "seq_start", torch.int32), _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32),
        int(total_new), int(block_size), int(num_blocks),
        _contig(slot_mapping, "slot_mapping", torch.int64), _opt(dev_status), _stream(stream))
    _check(rc, "pa_compute_slot_mapping")
    return slot_mapping


def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, dev_status=None, stream=None):
    """pa_reshape_and_cache; key/value may be token-strided views (rows contiguous)."""
    num_blocks, block_size, hkv, d = k_cache.shape
    for name, t in (("key", key), ("value", value)):
        if t.dim() != 3 or t.shape[1:] != (hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [tokens, {hkv}, {d}] with contiguous rows")
    if key.shape[0] != value.shape[0] or slot_mapping.numel() < key.shape[0]:
        raise ValueError("key, value and slot_mapping disagree on the token count")
    if not (key.dtype == value.dtype == k_cache.dtype == v_cache.dtype):
        raise TypeError("key, value and the pools must share one dtype")
    rc = load().pa_reshape_and_cache(
        _dev(key, "key"), _dev(value, "value"), key.stride(0), value.stride(0),
        _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(slot_mapping, "slot_mapping", torch.int64), int(key.shape[0]), hkv, d,
        block_size, num_blocks, _dtype_code(k_cache), _opt(dev_status), _stream(stream))
    _check(rc, "pa_reshape_and_cache")


def decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                               block_size, max_blocks))


def varlen_prefill_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim, block_size,
                                  max_blocks) -> int:
    return int(load().pa_varlen_prefill_workspace_size(num_seqs, total_q, num_heads, num_kv_heads,
                                                       head_dim, block_size, max_blocks))


def _ws(workspace, nbytes, device, stream):
    if workspace is None:
        workspace = _empty(max(nbytes, 16), torch.uint8, device, stream)
    return workspace


def decode(q, k_cache, v_cache, block_tables, context_lens, scale: float, out=None,
           workspace=None, dev_status=None, stream=None):
    """pa_decode: q [num_seqs, H, D] -> out [num_seqs, H, D]."""
    num_seqs, H, D = q.shape
    num_blocks, block_size, hkv, d = k_cache.shape
    max_blocks = block_tables.shape[1]
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    need = decode_workspace_size(num_seqs, H, hkv, D, block_size, max_blocks)
    workspace = _ws(workspace, need, q.device, stream)
    rc = load().pa_decode(
        _contig(out, "out"), _contig(q, "q"), _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(block_tables, "block_tables", torch.int32), _contig(context_lens, "context_lens", torch.int32),
        num_seqs, H, hkv, D, block_size, max_blocks, num_blocks, float(scale), _dtype_code(q),
        _contig(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _opt(dev_status), _stream(stream))
    _check(rc, "pa_decode")
    return out


def decode_step(q, key, value, k_cache, v_cache, block_tables, context_lens, seq_start, cu_seqlens_new,
                scale: float, out=None, slot_mapping=None, workspace=None, dev_status=None, stream=None):
    """pa_decode_step: slot mapping + cache write of the new tokens + decode, in one call.
    Returns (slot_mapping, out)."""
    num_seqs, H, D = q.shape
    num_blocks, block_size, hkv, d = k_cache.shape
    max_blocks = block_tables.shape[1]
    total_new = int(key.shape[0])
    for name, t in (("key", key), ("value", value)):
        if t.dim() != 3 or t.shape[1:] != (hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [tokens, {hkv}, {d}] with contiguous rows")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    if slot_mapping is None:
        slot_mapping = _empty(total_new, torch.int64, q.device, stream, result=True)
    need = decode_workspace_size(num_seqs, H, hkv, D, block_size, max_blocks)
    workspace = _ws(workspace, need, q.device, stream)
    rc = load().pa_decode_step(
        _contig(out, "out"), _contig(q, "q"), _dev(key, "key"), _dev(value, "value"), key.stride(0),
        value.stride(0), _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(block_tables, "block_tables", torch.int32), _contig(context_lens, "context_lens", torch.int32),
        _contig(seq_start, "seq_start", torch.int32), _contig(cu_seqlens_new, "cu_seqlens_new", torch.int32),
        total_new, _contig(slot_mapping, "slot_mapping", torch.int64), num_seqs, H, hkv, D, block_size,
        max_blocks, num_blocks, float(scale), _dtype_code(q), _contig(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt(dev_status), _stream(stream))
    _check(rc, "pa_decode_step")
    return slot_mapping, out


def copy_blocks(src_k, src_v, dst_k, dst_v, pairs, dev_status=None, stream=None):
    """pa_copy_blocks: whole blocks src -> dst between pools of equal block shape.
    Pools may be device tensors or pinned host tensors (reachable from the device);
    pairs is a device int32 tensor [n, 2]."""
    if src_k.shape[1:] != dst_k.shape[1:] or src_k.dtype != dst_k.dtype:
        raise ValueError("source and destination pools must share block shape and dtype")
    for name, t in (("src_k", src_k), ("src_v", src_v), ("dst_k", dst_k), ("dst_v", dst_v)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    pairs = pairs.reshape(-1, 2)
    block_bytes = src_k[0].numel() * src_k.element_size()
    rc = load().pa_copy_blocks(src_k.data_ptr(), src_v.data_ptr(), dst_k.data_ptr(), dst_v.data_ptr(),
                               block_bytes, int(src_k.shape[0]), int(dst_k.shape[0]),
                               _contig(pairs, "pairs", torch.int32), int(pairs.shape[0]), _opt(dev_status),
                               _stream(stream))
    _check(rc, "pa_copy_blocks")


def varlen_prefill(q, cu_seqlens_q, k_cache, v_cache, block_tables, context_lens, scale: float,
                   max_q_len: int, out=None, workspace=None, dev_status=None, stream=None,
                   causal: bool = True):
    """pa_varlen_prefill (causal) or pa_varlen_encode (causal=False) over a
    concatenated super-sequence: q [total_q, H, D]."""
    total_q, H, D = q.shape
    num_blocks, block_size, hkv, d = k_cache.shape
    num_seqs, max_blocks = block_tables.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    need = varlen_prefill_workspace_size(num_seqs, total_q, H, hkv, D, block_size, max_blocks)
    workspace = _ws(workspace, need, q.device, stream)
    fn = load().pa_varlen_prefill if causal else load().pa_varlen_encode
    rc = fn(
        _contig(out, "out"), _contig(q, "q"), _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32),
        _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(block_tables, "block_tables", torch.int32), _contig(context_lens, "context_lens", torch.int32),
        num_seqs, total_q, int(max_q_len), H, hkv, D, block_size, max_blocks, num_blocks, float(scale),
        _dtype_code(q), _contig(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _opt(dev_status), _stream(stream))
    _check(rc, "pa_varlen_prefill" if causal else "pa_varlen_encode")
    return out


def varlen_step(q, key, value, k_cache, v_cache, cu_seqlens_q, block_tables, context_lens, seq_start,
                scale: float, max_q_len: int, out=None, slot_mapping=None, workspace=None, dev_status=None,
                stream=None):
    """pa_varlen_step: slot mapping + cache write of the step's query tokens + causal varlen
    attention over the super-sequence, in one call.  Returns (slot_mapping, out)."""
    total_q, H, D = q.shape
    num_blocks, block_size, hkv, d = k_cache.shape
    num_seqs, max_blocks = block_tables.shape
    for name, t in (("key", key), ("value", value)):
        if t.dim() != 3 or t.shape[0] != total_q or t.shape[1:] != (hkv, d) or t.stride(2) != 1 \
                or t.stride(1) != d:
            raise ValueError(f"{name} must be [{total_q}, {hkv}, {d}] with contiguous rows")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    if slot_mapping is None:
        slot_mapping = _empty(total_q, torch.int64, q.device, stream, result=True)
    need = varlen_prefill_workspace_size(num_seqs, total_q, H, hkv, D, block_size, max_blocks)
    workspace = _ws(workspace, need, q.device, stream)
    rc = load().pa_varlen_step(
        _contig(out, "out"), _contig(q, "q"), _dev(key, "key"), _dev(value, "value"), key.stride(0),
        value.stride(0), _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(cu_seqlens_q, "cu_seqlens_q", torch.int32), _contig(block_tables, "block_tables", torch.int32),
        _contig(context_lens, "context_lens", torch.int32), _contig(seq_start, "seq_start", torch.int32),
        _contig(slot_mapping, "slot_mapping", torch.int64), num_seqs, total_q, int(max_q_len), H, hkv, D,
        block_size, max_blocks, num_blocks, float(scale), _dtype_code(q), _contig(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt(dev_status), _stream(stream))
    _check(rc, "pa_varlen_step")
    return slot_mapping, out


_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _refuse(dev: int, *specs):
    """Raises what is wrong with the first wrong tensor of (tensor, name, dtype or None); the calls below come here
    only when their one combined check fails.  Launches go to the current device's stream, so a tensor of another
    device is refused, not reached across."""
    for t, name, dtype in specs:
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _status(t, dev: int) -> int:
    """The status word's address; like the other tensors it is the current device's."""
    if t.is_cuda and t.get_device() != dev:
        raise ValueError(f"dev_status must be on the current device cuda:{dev}, got {t.device}")
    return _opt(t)


def _rows(name: str, t, shape, dtype, dev: int) -> None:
    """Raises what is wrong with a token-strided view [tokens, heads, d]."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} with contiguous rows")
    if t.dtype != dtype:
        raise TypeError("q, key, value and the 16/32-bit pools must share one dtype")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on the current device cuda:{dev}, got {t.device}")
    tokens, heads, d = shape
    _, sh, sd = t.stride()
    if tokens and ((sd != 1 and d > 1) or (sh != d and heads > 1)):
        raise ValueError(f"{name} must be {list(shape)} with contiguous rows")


def _q4_pool_shape(k_cache, v_cache, head_dim: int):
    """(num_blocks, block_size, num_kv_heads) of a pair of 4-bit pools."""
    if k_cache.dim() != 3 or k_cache.shape != v_cache.shape:
        raise ValueError("4-bit pools must be uint8 [num_blocks, num_kv_heads, slab] of one shape")
    num_blocks, hkv, slab = k_cache.shape
    row = head_dim // 2 + head_dim // 32 * 2
    if row <= 0 or slab % row:
        raise ValueError(f"a slab of {slab} bytes does not hold token rows of head_dim {head_dim}")
    return num_blocks, slab // row, hkv


def _rope(fn, q, key, value, cos_sin, positions, k_cache, v_cache, pool_dtype, num_blocks, block_size, slot_mapping,
          interleaved, q_out, dev_status, stream):
    shape, dtype, dev = key.shape, key.dtype, torch.cuda.current_device()
    n, hkv, d = shape
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    (ks, k1, k2), (vs, v1, v2) = key.stride(), value.stride()
    if not (value.shape == shape and value.dtype == dtype and k2 == 1 and v2 == 1 and k1 == d and v1 == d
            and key.get_device() == dev and value.get_device() == dev):
        _rows("key", key, shape, dtype, dev)     # (strides of single rows and heads may be anything)
        _rows("value", value, shape, dtype, dev)
    heads = qs = q_ptr = out_ptr = 0
    if q is not None:
        q_shape = q.shape
        heads = q_shape[1] if len(q_shape) == 3 else 0
        if q_out is None:
            q_out = _empty((n, heads, d), dtype, q.device, stream, result=True)
        qs, q1, q2 = q.stride() if heads else (0, 0, 0)
        if not (q_shape == q_out.shape == (n, heads, d) and q.dtype == q_out.dtype == dtype and q2 == 1 and q1 == d
                and q.get_device() == dev and q_out.get_device() == dev):
            _rows("q", q, (n, heads, d), dtype, dev)
            _rows("q_out", q_out, (n, heads, d), dtype, dev)
        if not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    if n == 1:   # torch may report any token stride for one token
        qs, ks, vs = heads * d, hkv * d, hkv * d
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and slot_mapping.is_contiguous()
            and k_cache.get_device() == v_cache.get_device() == slot_mapping.get_device() == dev
            and k_cache.dtype == v_cache.dtype == pool_dtype and slot_mapping.dtype == torch.int64):
        _refuse(dev, (k_cache, "k_cache", pool_dtype), (v_cache, "v_cache", pool_dtype),
                (slot_mapping, "slot_mapping", torch.int64))
    rot = max_pos = table_ptr = pos_ptr = 0
    if cos_sin is not None:
        if positions is None:
            raise ValueError("positions are needed with cos_sin")
        max_pos, rot = cos_sin.shape
        if not (cos_sin.is_contiguous() and positions.is_contiguous()
                and cos_sin.get_device() == positions.get_device() == dev
                and cos_sin.dtype == torch.float32 and positions.dtype == torch.int32):
            _refuse(dev, (cos_sin, "cos_sin", torch.float32), (positions, "positions", torch.int32))
        if positions.numel() < n:
            raise ValueError("positions must have an entry per token")
        table_ptr, pos_ptr = cos_sin.data_ptr(), positions.data_ptr()
    if slot_mapping.numel() < n:
        raise ValueError("slot_mapping must have an entry per token")
    rc = getattr(_lib or load(), fn)(
        out_ptr, q_ptr, key.data_ptr(), value.data_ptr(), qs, ks, vs, table_ptr, pos_ptr, max_pos, rot,
        1 if interleaved else 0, k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), n, heads, hkv, d,
        block_size, num_blocks, code, 0 if dev_status is None else _status(dev_status, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc != OK:
        raise PAError(rc, fn)
    return q_out


def rope_and_cache(q, key, value, cos_sin, positions, k_cache, v_cache, slot_mapping, interleaved: bool = False,
                   q_out=None, dev_status=None, stream=None):
    """pa_rope_and_cache: q [tokens, H, D] (or None) and key rotated by position, K/V rows written to the pools;
    returns q_out.  q, key and value may be token-strided views; cos_sin is fp32 [max_position, rot_dim] (None: no
    rotation) and positions int32 [tokens]."""
    pool, rows, dtype = k_cache.shape, key.shape, key.dtype
    if len(pool) != 4 or v_cache.shape != pool or len(rows) != 3 or rows[1] != pool[2] or rows[2] != pool[3]:
        raise ValueError("key, value and the pools disagree on heads or head_dim")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError("q, key, value and the 16/32-bit pools must share one dtype")
    return _rope("pa_rope_and_cache", q, key, value, cos_sin, positions, k_cache, v_cache, dtype, pool[0],
                 pool[1], slot_mapping, interleaved, q_out, dev_status, stream)


def q4_block_bytes(block_size: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().pa_q4_block_bytes(int(block_size), int(num_kv_heads), int(head_dim)))


def rope_and_cache_q4(q, key, value, cos_sin, positions, k_cache, v_cache, slot_mapping, interleaved: bool = False,
                      q_out=None, dev_status=None, stream=None):
    """pa_rope_and_cache_q4: rope_and_cache into 4-bit pools (uint8 [num_blocks, num_kv_heads,
    q4_block_bytes(block_size, 1, head_dim)])."""
    if key.dim() != 3:
        raise ValueError("key must be [tokens, num_kv_heads, head_dim]")
    num_blocks, block_size, hkv = _q4_pool_shape(k_cache, v_cache, key.shape[2])
    if key.shape[1] != hkv:
        raise ValueError("key and the pools disagree on num_kv_heads")
    return _rope("pa_rope_and_cache_q4", q, key, value, cos_sin, positions, k_cache, v_cache, torch.uint8, num_blocks,
                 block_size, slot_mapping, interleaved, q_out, dev_status, stream)


def _q4_blocks(fn, wide_k, wide_v, q4_k, q4_v, quantize, pairs, dev_status, stream):
    num_wide, block_size, hkv, d = wide_k.shape
    num_q4, b4, h4 = _q4_pool_shape(q4_k, q4_v, d)
    if wide_k.shape != wide_v.shape or b4 != block_size or h4 != hkv:
        raise ValueError("the 16/32-bit and 4-bit pools must share block size, heads and head_dim")
    dtype, dev = wide_k.dtype, torch.cuda.current_device()
    if wide_v.dtype != dtype:
        raise TypeError("the 16/32-bit pools must share one dtype")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    if not (wide_k.is_contiguous() and wide_v.is_contiguous() and q4_k.is_contiguous() and q4_v.is_contiguous()
            and pairs.is_contiguous() and pairs.dtype == torch.int32 and q4_k.dtype == q4_v.dtype == torch.uint8
            and wide_k.get_device() == wide_v.get_device() == q4_k.get_device() == q4_v.get_device()
            == pairs.get_device() == dev):
        _refuse(dev, (wide_k, "16/32-bit pool", None), (wide_v, "16/32-bit pool", None),
                (q4_k, "4-bit pool", torch.uint8), (q4_v, "4-bit pool", torch.uint8), (pairs, "pairs", torch.int32))
    n = pairs.numel()
    if n % 2:
        raise ValueError("pairs must be [n, 2]")
    wide, q4 = (wide_k.data_ptr(), wide_v.data_ptr()), (q4_k.data_ptr(), q4_v.data_ptr())
    src, dst = (wide, q4) if quantize else (q4, wide)
    n_src, n_dst = (num_wide, num_q4) if quantize else (num_q4, num_wide)
    rc = getattr(_lib or load(), fn)(src[0], src[1], dst[0], dst[1], block_size, hkv, d, n_src, n_dst,
                                     pairs.data_ptr(), n // 2, code, 0 if dev_status is None else _status(dev_status, dev),
                                     _raw_stream(dev) if stream is None else _stream(stream))
    if rc != OK:
        raise PAError(rc, fn)


def quantize_blocks_q4(src_k, src_v, dst_k, dst_v, pairs, dev_status=None, stream=None):
    """pa_quantize_blocks_q4: blocks of 16/32-bit pools [n, B, Hkv, D] into 4-bit pools; pairs device int32 [n, 2]."""
    _q4_blocks("pa_quantize_blocks_q4", src_k, src_v, dst_k, dst_v, True, pairs, dev_status, stream)


def dequantize_blocks_q4(src_k, src_v, dst_k, dst_v, pairs, dev_status=None, stream=None):
    """pa_dequantize_blocks_q4: blocks of 4-bit pools into 16/32-bit pools [n, B, Hkv, D]; pairs device int32 [n, 2]."""
    _q4_blocks("pa_dequantize_blocks_q4", dst_k, dst_v, src_k, src_v, False, pairs, dev_status, stream)


def decode_q4_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks) -> int:
    return int(load().pa_decode_q4_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                  max_blocks))


def decode_q4(q, k_cache, v_cache, block_tables, context_lens, scale: float, out=None, workspace=None,
              dev_status=None, stream=None):
    """pa_decode_q4: q [num_seqs, H, D] over 4-bit pools -> out [num_seqs, H, D]."""
    num_seqs, H, D = q.shape
    num_blocks, block_size, hkv = _q4_pool_shape(k_cache, v_cache, D)
    n, max_blocks = block_tables.shape
    if n != num_seqs or context_lens.numel() != num_seqs:
        raise ValueError("block_tables and context_lens must have a row per sequence")
    dtype, dev = q.dtype, torch.cuda.current_device()
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    elif out.shape != q.shape or out.dtype != dtype:
        raise ValueError("out must have q's shape and dtype")
    if workspace is None:
        workspace = _ws(None, decode_q4_workspace_size(num_seqs, H, hkv, D, block_size, max_blocks), q.device, stream)
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous() and workspace.is_contiguous()
            and k_cache.dtype == v_cache.dtype == torch.uint8
            and block_tables.dtype == context_lens.dtype == torch.int32
            and q.get_device() == out.get_device() == k_cache.get_device() == v_cache.get_device()
            == block_tables.get_device() == context_lens.get_device() == workspace.get_device() == dev):
        _refuse(dev, (q, "q", None), (out, "out", None), (k_cache, "k_cache", torch.uint8),
                (v_cache, "v_cache", torch.uint8), (block_tables, "block_tables", torch.int32),
                (context_lens, "context_lens", torch.int32), (workspace, "workspace", None))
    rc = (_lib or load()).pa_decode_q4(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), num_seqs, H, hkv, D, block_size, max_blocks, num_blocks, scale, code,
        workspace.data_ptr(), workspace.nbytes, 0 if dev_status is None else _status(dev_status, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc != OK:
        raise PAError(rc, "pa_decode_q4")
    return out


def validate_inputs(block_tables, context_lens, slot_mapping, block_size: int, num_blocks: int):
    """pa_validate_inputs on host (CPU) tensors.  Returns (status, check, index):
    status PA_OK or the error code, check the failed check (1-5, 0 when OK) and
    index the offending row or slot index (-1 when OK).  context_lens and
    slot_mapping may be None."""
    def host(t, dtype, name):
        if t is None:
            return None, None
        t = torch.as_tensor(t)
        if t.device.type != "cpu" or t.dtype != dtype:
            raise TypeError(f"{name}: expected a CPU {dtype} tensor")
        t = t.contiguous()
        return t, t.data_ptr()
    bt, bt_p = host(block_tables, torch.int32, "block_tables")
    ctx, ctx_p = host(context_lens, torch.int32, "context_lens")
    sl, sl_p = host(slot_mapping, torch.int64, "slot_mapping")
    num_seqs, max_blocks = (bt.shape[0], bt.shape[1]) if bt is not None else (0, 0)
    check, index = ctypes.c_int(-1), ctypes.c_int64(-2)
    rc = load().pa_validate_inputs(bt_p, num_seqs, max_blocks, ctx_p, sl_p,
                                   0 if sl is None else sl.numel(), block_size, num_blocks,
                                   ctypes.byref(check), ctypes.byref(index))
    return int(rc), int(check.value), int(index.value)


def get_device_status(dev_status, stream=None) -> int:
    host = ctypes.c_int32(-1)
    rc = load().pa_get_device_status(_dev(dev_status, "dev_status", torch.int32), ctypes.byref(host),
                                     _stream(stream))
    _check(rc, "pa_get_device_status")
    return int(host.value)


def reset_device_status(dev_status, stream=None) -> None:
    _check(load().pa_reset_device_status(_dev(dev_status, "dev_status", torch.int32), _stream(stream)),
           "pa_reset_device_status")


def set_timing_events(ev_begin=None, ev_end=None) -> None:
    """pa_set_timing_events with torch.cuda.Event objects (or None, None)."""
    def handle(ev):
        if ev is None:
            return None
        if ev.cuda_event == 0:      # torch creates the CUDA event on first record
            ev.record()
        return ev.cuda_event
    _check(load().pa_set_timing_events(handle(ev_begin), handle(ev_end)), "pa_set_timing_events")


def set_wait_test(limit_ns: int = 0, stall: int = STALL_NONE, after: int = 0, sites=None) -> None:
    """pa_set_wait_test: the bounded in-kernel waits' limit (0 = one second) and
    the test stall for later calls from this thread; sites is an optional
    device int32 tensor that receives the WAIT_* bits of the waits that ran out."""
    _check(load().pa_set_wait_test(int(limit_ns), int(stall), int(after),
                                   None if sites is None else _dev(sites, "sites", torch.int32)),
           "pa_set_wait_test")


def decode_static_scratch(q, k_cache, v_cache, block_tables, context_lens, scale: float, out=None,
                          dev_status=None, stream=None):
    """pa_decode_static_scratch: pa_decode with the library's fixed scratch array
    (for callers that cannot allocate device memory)."""
    num_seqs, H, D = q.shape
    num_blocks, block_size, hkv, d = k_cache.shape
    max_blocks = block_tables.shape[1]
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, result=True)
    rc = load().pa_decode_static_scratch(
        _contig(out, "out"), _contig(q, "q"), _contig(k_cache, "k_cache"), _contig(v_cache, "v_cache"),
        _contig(block_tables, "block_tables", torch.int32), _contig(context_lens, "context_lens", torch.int32),
        num_seqs, H, hkv, D, block_size, max_blocks, num_blocks, float(scale), _dtype_code(q),
        _opt(dev_status), _stream(stream))
    _check(rc, "pa_decode_static_scratch")
    return out


class BlockManager:
    """Host block pool (pa_block_manager_*): allocate_slots, free, shared prefixes,
    and the int32 block tables / token counts the kernels consume."""

    def __init__(self, num_blocks: int, block_size: int = 16, max_blocks_per_seq: int = 4096):
        self._L = load()
        self._h = self._L.pa_block_manager_create(num_blocks, block_size, max_blocks_per_seq)
        if not self._h:
            raise ValueError("invalid block manager arguments")
        self.num_blocks, self.block_size, self.max_blocks_per_seq = num_blocks, block_size, max_blocks_per_seq

    def close(self):
        if self._h:
            self._L.pa_block_manager_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def num_free(self) -> int:
        return int(self._L.pa_block_manager_num_free(self._h))

    def refcount(self, block: int) -> int:
        return int(self._L.pa_block_manager_refcount(self._h, int(block)))

    def allocate_slots(self, seq_id: int, num_new_tokens: int) -> int:
        """Returns the status (OK, ERR_OUT_OF_RANGE when the pool is short, ...)."""
        return int(self._L.pa_allocate_slots(self._h, int(seq_id), int(num_new_tokens)))

    def allocate_slots_batch(self, seq_ids, num_new_tokens, statuses=None) -> int:
        """pa_allocate_slots_batch on host int64 seq_ids / int32 counts (numpy
        or CPU tensors); fills statuses (int32, same length) when given."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        cnt = np.ascontiguousarray(num_new_tokens, dtype=np.int32)
        if ids.shape != cnt.shape:
            raise ValueError("seq_ids and num_new_tokens must have the same length")
        st_ptr = None
        if statuses is not None:
            if not (isinstance(statuses, np.ndarray) and statuses.dtype == np.int32 and statuses.flags.c_contiguous
                    and statuses.shape == ids.shape):
                raise ValueError("statuses must be a contiguous int32 numpy array of the same length")
            st_ptr = statuses.ctypes.data
        return int(self._L.pa_allocate_slots_batch(self._h, ids.ctypes.data, cnt.ctypes.data, int(ids.size),
                                                   st_ptr))

    def free(self, seq_id: int) -> int:
        return int(self._L.pa_free_sequence(self._h, int(seq_id)))

    def share_prefix(self, parent_id: int, child_id: int, num_tokens: int) -> int:
        return int(self._L.pa_share_prefix(self._h, int(parent_id), int(child_id), int(num_tokens)))

    def tables(self, seq_ids, max_blocks: int):
        """(block_tables int32 [n, max_blocks], num_tokens int32 [n]) as CPU tensors."""
        ids = torch.tensor(list(seq_ids), dtype=torch.int64)
        bt = torch.empty((ids.numel(), max_blocks), dtype=torch.int32)
        nt = torch.empty(ids.numel(), dtype=torch.int32)
        rc = self._L.pa_block_manager_tables(self._h, ids.data_ptr(), ids.numel(), bt.data_ptr(),
                                             int(max_blocks), nt.data_ptr())
        _check(rc, "pa_block_manager_tables")
        return bt, nt
