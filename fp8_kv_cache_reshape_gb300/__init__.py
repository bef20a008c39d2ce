"""Python binding of libkvq (include/kvq.h): FP8 E4M3 KV-cache quantization
and attention over a paged FP8 / BF16 KV cache on GB300 (sm_103a).

The functions below carry the C ABI's names and only marshal arguments:
shapes and device pointers are read from torch tensors, the current CUDA
stream is passed through, and a non-zero status raises KvqError with the
library's message.  Every step runs in the library's CUDA kernels; there is
no fallback.  PyTorch provides device memory and streams.

Build the library first (``python -c "import __graft_entry__ as g; g.build()"``
or ``python fp8_kv_cache_reshape_gb300/_build.py``); importing this module
without it raises ImportError.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_CUDA = 3
KVQ_ERR_DEVICE_FAULT = 4

KVQ_DTYPE_FP8_E4M3 = 0
KVQ_DTYPE_BF16 = 1
KVQ_DTYPE_FP8_E5M2 = 2
KVQ_DTYPE_FP4_E2M1 = 3

KVQ_ACC_TWO_LEVEL = 0
KVQ_ACC_SINGLE_LEVEL = 1

KVQ_DEV_BAD_SLOT = 0x1
KVQ_DEV_BAD_BLOCK = 0x2
KVQ_DEV_BAD_SEQLEN = 0x4
KVQ_DEV_TIMEOUT = 0x8
KVQ_DEV_BAD_QROWS = 0x10
KVQ_DEV_BAD_GROUP = 0x20
KVQ_DEV_BAD_AXIS = 0x40

PAGE = 16

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libkvq.so is not built ({LIB_PATH}); run fp8_kv_cache_reshape_gb300/_build.py")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_f = ctypes.c_float
_sz = ctypes.c_size_t

lib.kvq_version.restype = _i
lib.kvq_version.argtypes = []
lib.kvq_last_error_string.restype = ctypes.c_char_p
lib.kvq_last_error_string.argtypes = []
lib.kvq_debug_set_stall_ns.restype = None
lib.kvq_debug_set_stall_ns.argtypes = [ctypes.c_uint64]
lib.kvq_reshape_and_cache.restype = _i
lib.kvq_reshape_and_cache.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i64, _i, _p, _p]
lib.kvq_quantize_query.restype = _i
lib.kvq_quantize_query.argtypes = [_p, _p, _p, _i64, _p]
lib.kvq_decode_num_splits.restype = _i
lib.kvq_decode_num_splits.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.kvq_decode_workspace_size.restype = _sz
lib.kvq_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
lib.kvq_paged_decode_attention.restype = _i
lib.kvq_paged_decode_attention.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _f,
                                           _i, _i, _i, _p, _sz, _p, _p]
lib.kvq_decode_static_scratch_bytes.restype = _sz
lib.kvq_decode_static_scratch_bytes.argtypes = []
lib.kvq_paged_decode_attention_static_scratch.restype = _i
lib.kvq_paged_decode_attention_static_scratch.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i,
                                                          _i64, _f, _i, _i, _i, _p, _p]
lib.kvq_reshape_and_cache_per_token.restype = _i
lib.kvq_reshape_and_cache_per_token.argtypes = [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i64, _i, _p, _p]
lib.kvq_paged_decode_attention_per_token.restype = _i
lib.kvq_paged_decode_attention_per_token.argtypes = [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64,
                                                     _f, _i, _i, _i, _p, _sz, _p, _p]
lib.kvq_paged_decode_attention_append.restype = _i
lib.kvq_paged_decode_attention_append.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i,
                                                  _i64, _f, _i, _i, _i, _p, _sz, _p, _p]
lib.kvq_paged_decode_attention_acc.restype = _i
lib.kvq_paged_decode_attention_acc.argtypes = lib.kvq_paged_decode_attention.argtypes + [_i]
lib.kvq_prefill_attention_acc.restype = _i
lib.kvq_prefill_attention_acc.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _i,
                                          _f, _i, _p, _p, _i]
lib.kvq_prefill_attention_dtype.restype = _i
lib.kvq_prefill_attention_dtype.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _i,
                                            _f, _i, _p, _p, _i]
lib.kvq_prefill_attention_per_token.restype = _i
lib.kvq_prefill_attention_per_token.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _i,
                                                _f, _i, _i, _p, _p]
lib.kvq_prefill_attention.restype = _i
lib.kvq_prefill_attention.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _i,
                                      _f, _i, _p, _p]
lib.kvq_shared_prefix_workspace_size.restype = _sz
lib.kvq_shared_prefix_workspace_size.argtypes = [_i] * 8
lib.kvq_paged_decode_attention_shared_prefix.restype = _i
lib.kvq_paged_decode_attention_shared_prefix.argtypes = [_p] * 11 + [_i] * 8 + [_i64, _f, _i, _p, _sz, _p, _p]
lib.kvq_decode_weights_workspace_size.restype = _sz
lib.kvq_decode_weights_workspace_size.argtypes = [_i] * 8
lib.kvq_paged_decode_attention_weights.restype = _i
lib.kvq_paged_decode_attention_weights.argtypes = [_p] * 9 + [_i64, _f, _i, _i, _i, _i, _i, _i, _i64, _f, _i, _i, _i,
                                                              _i, _p, _sz, _p, _p]
lib.kvq_evict_tokens.restype = _i
lib.kvq_evict_tokens.argtypes = [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _i64, _p, _p, _i, _i, _i, _i, _i, _i, _i64, _i,
                                 _i, _i, _i, _p, _p]


class _Rotary(ctypes.Structure):
    _fields_ = [("positions", _p), ("positions_stride", _i64), ("inv_freq", _p), ("pair_axis", _p), ("num_axes", _i),
                ("rot_dim", _i), ("interleaved", _i), ("scale", _f)]


class _HeadNorm(ctypes.Structure):
    _fields_ = [("q_weight", _p), ("k_weight", _p), ("eps", _f)]


_rot, _norm = ctypes.POINTER(_Rotary), ctypes.POINTER(_HeadNorm)
lib.kvq_qk_norm_rope.restype = _i
lib.kvq_qk_norm_rope.argtypes = [_p, _i64, _p, _i64, _norm, _rot, _p, _i64, _p, _i64, _i, _i, _i, _i, _p, _p]
lib.kvq_rope_and_cache.restype = _i
lib.kvq_rope_and_cache.argtypes = [_p, _i64, _p, _i64, _p, _i64, _norm, _rot, _p, _p, _p, _p, _p, _p, _i64, _p, _p, _i, _i,
                                   _i, _i, _i, _i64, _i, _i, _p, _p]
lib.kvq_gather_cache.restype = _i
lib.kvq_gather_cache.argtypes = [_p] * 7 + [_i, _i, _i, _i, _i64, _i, _i, _p, _p]
lib.kvq_decode_fp4_workspace_size.restype = _sz
lib.kvq_decode_fp4_workspace_size.argtypes = [_i] * 6
lib.kvq_paged_decode_attention_fp4.restype = _i
lib.kvq_paged_decode_attention_fp4.argtypes = [_p] * 8 + [_i] * 6 + [_i64, _f, _i, _p, _sz, _p, _p]


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.kvq_last_error_string().decode(errors="replace")
        super().__init__(f"{where}: status {status}: {msg}")
        self.status = status


def _check(status: int, where: str):
    if status != KVQ_OK:
        raise KvqError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkvq takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libkvq takes contiguous tensors only")
    return t.data_ptr()


# the current device's current stream as a raw handle; torch.cuda.current_stream()
# builds a Python object around it, several microseconds a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(cache_dtype: str) -> int:
    if cache_dtype in ("fp8", "fp8_e4m3", KVQ_DTYPE_FP8_E4M3):
        return KVQ_DTYPE_FP8_E4M3
    if cache_dtype in ("bf16", "bfloat16", KVQ_DTYPE_BF16):
        return KVQ_DTYPE_BF16
    if cache_dtype in ("fp8_e5m2", KVQ_DTYPE_FP8_E5M2):
        return KVQ_DTYPE_FP8_E5M2
    if cache_dtype in ("fp4", "fp4_e2m1", KVQ_DTYPE_FP4_E2M1):
        return KVQ_DTYPE_FP4_E2M1
    raise ValueError(f"unknown cache dtype {cache_dtype!r}")


def _acc_code(accumulation) -> int:
    if accumulation in ("two_level", KVQ_ACC_TWO_LEVEL):
        return KVQ_ACC_TWO_LEVEL
    if accumulation in ("single_level", KVQ_ACC_SINGLE_LEVEL):
        return KVQ_ACC_SINGLE_LEVEL
    raise ValueError(f"unknown accumulation mode {accumulation!r}")


def version() -> int:
    return lib.kvq_version()


def kvq_debug_set_stall_ns(ns: int):
    """Failure-path test hook (include/kvq.h): > 0 makes later decode and
    prefill launches fail one bounded wait after `ns` nanoseconds; 0 = off."""
    lib.kvq_debug_set_stall_ns(int(ns))


# per-token scale tail of a V page: 16 K scales and 16 V scales, float32
SCALE_TAIL_BYTES = 2 * PAGE * 4


def _page_bytes(head_dim, dt):
    """Bytes of a K page: FP4 codes and their block scales, FP8 codes or bf16."""
    if dt == KVQ_DTYPE_FP4_E2M1:
        return PAGE * (head_dim // 2 + head_dim // 16)
    return PAGE * head_dim * (2 if dt == KVQ_DTYPE_BF16 else 1)


def alloc_kv_cache(num_blocks: int, kv_heads: int, head_dim: int, cache_dtype="fp8_e4m3",
                   device="cuda", fill=None, per_token=False, paired=False):
    """Allocate (k_cache, v_cache) as uint8 tensors in the library's paged
    format ([num_blocks][Hkv][P][D] and [num_blocks][Hkv][D][P] elements).
    per_token: each V page also carries its scale tail (FP8 only).
    "fp4_e2m1": 4-bit codes and a block scale per 16 dims (head dims 64, 128).
    paired: one allocation [num_blocks][Hkv][K page | V page]; k_cache is it
    and v_cache a flat view starting one K page in (the library recognizes
    the layout from the pointers and moves each pair with one copy)."""
    dt = _dtype_code(cache_dtype)
    if per_token and dt not in (KVQ_DTYPE_FP8_E4M3, KVQ_DTYPE_FP8_E5M2):
        raise ValueError("per-token scales need an FP8 cache")
    if dt == KVQ_DTYPE_FP4_E2M1 and head_dim not in (64, 128):
        raise ValueError("an FP4 cache has head dim 64 or 128")
    kpage = _page_bytes(head_dim, dt)
    vpage = kpage + (SCALE_TAIL_BYTES if per_token else 0)
    make = (lambda shape: torch.empty(shape, dtype=torch.uint8, device=device)) if fill is None else \
        (lambda shape: torch.full(shape, fill, dtype=torch.uint8, device=device))
    if paired:
        buf = make((num_blocks, kv_heads, kpage + vpage))
        return buf, buf.view(-1)[kpage:]
    return make((num_blocks, kv_heads, kpage)), make((num_blocks, kv_heads, vpage))


def _is_paired(k_cache, v_cache, kpage):
    return v_cache.data_ptr() == k_cache.data_ptr() + kpage


def _is_one_page(k_cache, v_cache, kpage, vpage):
    """Separate tensors of one page each, which may lie side by side: the same bytes as a pair."""
    return k_cache.nbytes == kpage and v_cache.nbytes == vpage


def _num_blocks(k_cache, v_cache, Hkv, kpage):
    """Blocks of a cache from its K tensor: [num_blocks][Hkv][...] (separate
    or paired), or flat separate pages."""
    if k_cache.dim() >= 2 or _is_paired(k_cache, v_cache, kpage):
        return k_cache.shape[0]
    return k_cache.numel() // (Hkv * kpage)


def kvq_reshape_and_cache(k, v, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None,
                          cache_dtype="fp8_e4m3", dev_status=None, stream=None):
    """Quantize (or copy) new tokens k, v (bf16 [T][Hkv][D]) into the cache."""
    T, Hkv, D = k.shape
    dt = _dtype_code(cache_dtype)
    if dt == KVQ_DTYPE_FP4_E2M1:
        _check_dense(k, torch.bfloat16, (T, Hkv, D), "k")
        _check_dense(v, torch.bfloat16, (T, Hkv, D), "v")
        _check_dense(slot_mapping, torch.int64, (T,), "slot_mapping")
        num_blocks = _check_dense_cache(k_cache, v_cache, k_scale, v_scale, Hkv, D, dt, False, None)
        *ptrs, status = _addresses(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, dev_status)
        _check(lib.kvq_reshape_and_cache(*ptrs, T, Hkv, D, PAGE, num_blocks, dt, status, _stream(stream)),
               "kvq_reshape_and_cache")
        return
    num_blocks = _num_blocks(k_cache, v_cache, Hkv, _page_bytes(D, dt))
    _check(lib.kvq_reshape_and_cache(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(k_scale), _ptr(v_scale), T, Hkv, D, PAGE, num_blocks, dt,
                                     _ptr(dev_status), _stream(stream)), "kvq_reshape_and_cache")


def _check_per_token_cache(k_cache, v_cache, Hkv, D):
    kpage, vpage = PAGE * D, PAGE * D + SCALE_TAIL_BYTES
    if _is_paired(k_cache, v_cache, kpage):
        nb = k_cache.shape[0]
        ok = k_cache.numel() == nb * Hkv * (kpage + vpage) or nb * Hkv == 1 and _is_one_page(k_cache, v_cache, kpage, vpage)
    else:
        nb = k_cache.numel() // (Hkv * kpage)
        ok = k_cache.numel() == nb * Hkv * kpage and v_cache.numel() == nb * Hkv * vpage
    if not ok:
        raise ValueError("per-token caches must be alloc_kv_cache(..., per_token=True) tensors")
    return nb


def kvq_reshape_and_cache_per_token(k, v, slot_mapping, k_cache, v_cache, cache_dtype="fp8_e4m3",
                                    dev_status=None, stream=None):
    """Quantize new tokens k, v (bf16 [T][Hkv][D]) with one dynamic scale per
    token and head; the scales go to the scale tails of the V pages."""
    T, Hkv, D = k.shape
    num_blocks = _check_per_token_cache(k_cache, v_cache, Hkv, D)
    _check(lib.kvq_reshape_and_cache_per_token(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                               T, Hkv, D, PAGE, num_blocks, _dtype_code(cache_dtype),
                                               _ptr(dev_status), _stream(stream)),
           "kvq_reshape_and_cache_per_token")


def kvq_quantize_query(q, q8, q_scale, stream=None):
    """q8 = E4M3(q / q_scale), per tensor."""
    _check(lib.kvq_quantize_query(_ptr(q), _ptr(q8), _ptr(q_scale), q.numel(), _stream(stream)),
           "kvq_quantize_query")


def _window(window):
    """A window as a C int, which ctypes would make of any integer's last 32 bits."""
    return max(-2, min(window, 2**31 - 1))


def kvq_decode_num_splits(B, Hkv, max_blocks, window=-1, num_splits=0, head_dim=128):
    return lib.kvq_decode_num_splits(B, Hkv, head_dim, PAGE, max_blocks, _window(window), num_splits)


def kvq_decode_workspace_size(B, Hq, Hkv, D, max_blocks, window=-1, num_splits=0):
    return lib.kvq_decode_workspace_size(B, Hq, Hkv, D, PAGE, max_blocks, _window(window), num_splits)


def _workspace(need, like, stream):
    """A workspace for one call, from the memory of the call's own stream: work
    queued on another one neither still uses it nor reuses it while the call runs."""
    if stream is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device) if isinstance(stream, int) else stream):
        return torch.empty(max(need, 16), dtype=torch.uint8, device=like.device)


def kvq_paged_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out,
                               num_blocks=None, sm_scale=None, window=-1, cache_dtype="fp8_e4m3",
                               num_splits=0, workspace=None, dev_status=None, stream=None, accumulation=None):
    """One decode step over the paged cache; writes out (bf16 [B][Hq][D]).

    workspace: a uint8 CUDA tensor of at least kvq_decode_workspace_size()
    bytes (allocated here when omitted).  accumulation: None (the default,
    two-level) or "two_level" / "single_level" through
    kvq_paged_decode_attention_acc."""
    B, Hq, D = q.shape
    max_blocks = block_table.shape[1]
    dt = _dtype_code(cache_dtype)
    Hkv = k_cache.shape[1] if k_cache.dim() >= 3 else None
    if Hkv is None:
        raise ValueError("k_cache must be [num_blocks][Hkv][...]")
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    need = kvq_decode_workspace_size(B, Hq, Hkv, D, max_blocks, window, num_splits)
    if workspace is None:
        workspace = _workspace(need, q, stream)
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
            _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, PAGE, max_blocks, num_blocks, float(sm_scale), _window(window), dt,
            num_splits, _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    if accumulation is None:
        _check(lib.kvq_paged_decode_attention(*args), "kvq_paged_decode_attention")
    else:
        _check(lib.kvq_paged_decode_attention_acc(*args, _acc_code(accumulation)), "kvq_paged_decode_attention_acc")
    return out


def kvq_paged_decode_attention_append(q, k_new, v_new, slot_new, k_cache, v_cache, k_scale, v_scale, block_table,
                                      seq_lens, out, num_blocks=None, sm_scale=None, window=-1,
                                      cache_dtype="fp8_e4m3", num_splits=0, workspace=None, dev_status=None,
                                      stream=None):
    """One decode step that also writes the step's new token (k_new, v_new:
    bf16 [B][Hkv][D], slot_new: int64 [B]) into the cache, as
    kvq_reshape_and_cache followed by kvq_paged_decode_attention would."""
    B, Hq, D = q.shape
    max_blocks = block_table.shape[1]
    Hkv = k_cache.shape[1]
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    for t in (k_new, v_new):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hkv, D):
            raise ValueError("k_new / v_new must be bf16 [B][Hkv][D]")
    if slot_new.dtype != torch.int64 or slot_new.numel() != B:
        raise ValueError("slot_new must be int64 [B]")
    need = kvq_decode_workspace_size(B, Hq, Hkv, D, max_blocks, window, num_splits)
    if workspace is None:
        workspace = _workspace(need, q, stream)
    _check(lib.kvq_paged_decode_attention_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_new), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, PAGE, max_blocks, num_blocks,
        float(sm_scale), _window(window), _dtype_code(cache_dtype), num_splits, _ptr(workspace), workspace.numel(),
        _ptr(dev_status), _stream(stream)), "kvq_paged_decode_attention_append")
    return out


def kvq_paged_decode_attention_per_token(q, k_cache, v_cache, block_table, seq_lens, out, num_blocks=None,
                                         sm_scale=None, window=-1, cache_dtype="fp8_e4m3", num_splits=0,
                                         workspace=None, dev_status=None, stream=None):
    """Decode over a cache written by kvq_reshape_and_cache_per_token."""
    B, Hq, D = q.shape
    max_blocks = block_table.shape[1]
    Hkv = k_cache.shape[1]
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    need = kvq_decode_workspace_size(B, Hq, Hkv, D, max_blocks, window, num_splits)
    if workspace is None:
        workspace = _workspace(need, q, stream)
    _check(lib.kvq_paged_decode_attention_per_token(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, PAGE, max_blocks, num_blocks, float(sm_scale), _window(window),
        _dtype_code(cache_dtype), num_splits, _ptr(workspace), workspace.numel(), _ptr(dev_status),
        _stream(stream)), "kvq_paged_decode_attention_per_token")
    return out


def kvq_prefill_attention(q8, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_q,
                          seq_lens, out, max_q_tokens, num_blocks=None, sm_scale=None, causal=True,
                          dev_status=None, stream=None, accumulation=None, cache_dtype="fp8_e4m3"):
    """Chunked causal prefill over the FP8 cache; writes out (bf16 [Tq][Hq][D]).
    accumulation: None (two-level) or "two_level" / "single_level" through
    kvq_prefill_attention_acc.  cache_dtype "fp8_e5m2" goes through
    kvq_prefill_attention_dtype (with the default accumulation)."""
    Tq, Hq, D = q8.shape
    B = cu_seqlens_q.numel() - 1
    Hkv = k_cache.shape[1]
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    args = (_ptr(q8), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_table), _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, PAGE,
            block_table.shape[1], num_blocks, int(max_q_tokens), float(sm_scale), 1 if causal else 0,
            _ptr(dev_status), _stream(stream))
    dt = _dtype_code(cache_dtype)
    if dt != KVQ_DTYPE_FP8_E4M3:
        if accumulation is not None:
            raise ValueError("an explicit accumulation mode takes an E4M3 cache")
        _check(lib.kvq_prefill_attention_dtype(*args, dt), "kvq_prefill_attention_dtype")
    elif accumulation is None:
        _check(lib.kvq_prefill_attention(*args), "kvq_prefill_attention")
    else:
        _check(lib.kvq_prefill_attention_acc(*args, _acc_code(accumulation)), "kvq_prefill_attention_acc")
    return out


def kvq_prefill_attention_per_token(q8, q_scale, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens, out,
                                    max_q_tokens, num_blocks=None, sm_scale=None, causal=True,
                                    cache_dtype="fp8_e4m3", dev_status=None, stream=None):
    """Chunked causal prefill over a cache written by
    kvq_reshape_and_cache_per_token; writes out (bf16 [Tq][Hq][D])."""
    Tq, Hq, D = q8.shape
    B = cu_seqlens_q.numel() - 1
    Hkv = k_cache.shape[1]
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    _check_per_token_cache(k_cache, v_cache, Hkv, D)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    _check(lib.kvq_prefill_attention_per_token(
        _ptr(q8), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(cu_seqlens_q),
        _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, PAGE, block_table.shape[1], num_blocks, int(max_q_tokens),
        float(sm_scale), 1 if causal else 0, _dtype_code(cache_dtype), _ptr(dev_status), _stream(stream)),
        "kvq_prefill_attention_per_token")
    return out


def _check_tensor(t, dtype, shape, name):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


def _check_cache(k_cache, v_cache, Hkv, D, dt, per_token, num_blocks):
    """The caches' bytes against what the head dim and format say (a wrong one
    would read and write past a page); returns the block count."""
    kpage = _page_bytes(D, dt)
    vpage = kpage + (SCALE_TAIL_BYTES if per_token else 0)
    nb = k_cache.shape[0]
    if v_cache.data_ptr() == k_cache.data_ptr() + kpage:
        ok = k_cache.nbytes == nb * Hkv * (kpage + vpage) or nb * Hkv == 1 and _is_one_page(k_cache, v_cache, kpage, vpage)
    else:
        ok = k_cache.nbytes == nb * Hkv * kpage and v_cache.nbytes == nb * Hkv * vpage
    if not ok:
        raise ValueError("k_cache and v_cache must be alloc_kv_cache() tensors of this head dim and cache dtype")
    if num_blocks is None:
        return nb
    if num_blocks > nb:
        raise ValueError(f"num_blocks {num_blocks} > the caches' {nb}")
    return num_blocks


def _check_scales(k_scale, v_scale, Hkv):
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None:
            _check_tensor(t, torch.float32, (Hkv,), name)


def _device_ptrs(*tensors):
    """Addresses of contiguous tensors on the current device (None for None)."""
    if not tensors[0].is_cuda:
        raise ValueError("libkvq takes CUDA tensors only")
    current = torch.cuda.current_device()
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != current:
            if not t.is_cuda:
                raise ValueError("libkvq takes CUDA tensors only")
            raise ValueError(f"the tensors' device (cuda:{t.get_device()}) must be the current one (cuda:{current})")
        if not t.is_contiguous():
            raise ValueError("libkvq takes contiguous tensors only")
        out.append(t.data_ptr())
    return out


def kvq_shared_prefix_workspace_size(B, G, Hq, Hkv, D, max_prefix_blocks, max_blocks):
    return lib.kvq_shared_prefix_workspace_size(B, G, Hq, Hkv, D, PAGE, max_prefix_blocks, max_blocks)


def kvq_paged_decode_attention_shared_prefix(q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_lens,
                                             group_starts, block_table, seq_lens, out, num_blocks=None, sm_scale=None,
                                             cache_dtype="fp8_e4m3", workspace=None, dev_status=None, stream=None):
    """One decode step of a batch whose sequences share prefixes: sequences
    group_starts[i] .. group_starts[i + 1] - 1 attend to the first
    prefix_lens[i] tokens of prefix_table[i] (read once for the whole group)
    and to their own seq_lens[b] tokens of block_table[b]."""
    B, Hq, D = q.shape
    G, max_prefix = prefix_table.shape
    Hkv = k_cache.shape[1]
    _check_tensor(q, torch.bfloat16, (B, Hq, D), "q")
    _check_tensor(out, torch.bfloat16, (B, Hq, D), "out")
    _check_tensor(prefix_table, torch.int32, (G, max_prefix), "prefix_table")
    _check_tensor(prefix_lens, torch.int32, (G,), "prefix_lens")
    _check_tensor(group_starts, torch.int32, (G + 1,), "group_starts")
    _check_tensor(block_table, torch.int32, (B, block_table.shape[1]), "block_table")
    _check_tensor(seq_lens, torch.int32, (B,), "seq_lens")
    max_blocks = block_table.shape[1]
    dt = _dtype_code(cache_dtype)
    _check_scales(k_scale, v_scale, Hkv)
    num_blocks = _check_cache(k_cache, v_cache, Hkv, D, dt, False, num_blocks)
    if workspace is None:
        workspace = _workspace(kvq_shared_prefix_workspace_size(B, G, Hq, Hkv, D, max_prefix, max_blocks), q, stream)
    *ptrs, ws, status = _device_ptrs(q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_lens, group_starts,
                                     block_table, seq_lens, out, workspace, dev_status)
    _check(lib.kvq_paged_decode_attention_shared_prefix(
        *ptrs, B, G, Hq, Hkv, D, PAGE, max_prefix, max_blocks, num_blocks,
        1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), dt, ws, workspace.nbytes, status,
        _stream(stream)), "kvq_paged_decode_attention_shared_prefix")
    return out


def kvq_decode_weights_workspace_size(B, Hq, Hkv, D, max_blocks, window=-1, num_splits=0):
    return lib.kvq_decode_weights_workspace_size(B, Hq, Hkv, D, PAGE, max_blocks, _window(window), num_splits)


def kvq_paged_decode_attention_weights(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, weights,
                                       decay=1.0, num_blocks=None, sm_scale=None, window=-1, cache_dtype="fp8_e4m3",
                                       per_token=False, num_splits=0, workspace=None, dev_status=None, stream=None):
    """kvq_paged_decode_attention that also accumulates each cached token's
    attention weight: weights (float32 [B][Hkv][>= max_blocks * 16]) becomes
    decay * weights + the sum over the KV head's query heads, for the first
    seq_lens[b] tokens.  per_token: a per-token-scaled cache (k_scale and
    v_scale None)."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    max_blocks = block_table.shape[1]
    _check_tensor(q, torch.bfloat16, (B, Hq, D), "q")
    _check_tensor(out, torch.bfloat16, (B, Hq, D), "out")
    _check_tensor(block_table, torch.int32, (B, max_blocks), "block_table")
    _check_tensor(seq_lens, torch.int32, (B,), "seq_lens")
    _check_tensor(weights, torch.float32, (B, Hkv, weights.shape[-1]), "weights")
    dt = _dtype_code(cache_dtype)
    _check_scales(k_scale, v_scale, Hkv)
    num_blocks = _check_cache(k_cache, v_cache, Hkv, D, dt, per_token, num_blocks)
    if workspace is None:
        workspace = _workspace(kvq_decode_weights_workspace_size(B, Hq, Hkv, D, max_blocks, window, num_splits), q, stream)
    *ptrs, ws, status = _device_ptrs(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, weights, workspace,
                                     dev_status)
    _check(lib.kvq_paged_decode_attention_weights(
        *ptrs, weights.shape[-1], float(decay), B, Hq, Hkv, D, PAGE, max_blocks, num_blocks,
        1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale), _window(window), dt, 1 if per_token else 0, num_splits, ws,
        workspace.nbytes, status, _stream(stream)), "kvq_paged_decode_attention_weights")
    return out


def kvq_evict_tokens(weights, k_cache, v_cache, block_table, seq_lens, keep_lens, dst_block_table, dst_weights,
                     dst_seq_lens, kept, head_dim, sink=0, recent=0, num_blocks=None, cache_dtype="fp8_e4m3",
                     per_token=False, dev_status=None, stream=None):
    """Cut each sequence's cache to its keep_lens[b] heaviest tokens per KV
    head (the first `sink` and last `recent` always stay), copied in order
    into the pages dst_block_table[b]; dst_weights (float32 [B][Hkv][...]),
    dst_seq_lens (int32 [B]) and kept (int32 [B][Hkv][max_dst_blocks * 16],
    source positions) are written."""
    B, max_blocks = block_table.shape
    max_dst = dst_block_table.shape[1]
    Hkv = k_cache.shape[1]
    _check_tensor(weights, torch.float32, (B, Hkv, weights.shape[-1]), "weights")
    _check_tensor(block_table, torch.int32, (B, max_blocks), "block_table")
    _check_tensor(seq_lens, torch.int32, (B,), "seq_lens")
    _check_tensor(keep_lens, torch.int32, (B,), "keep_lens")
    _check_tensor(dst_block_table, torch.int32, (B, max_dst), "dst_block_table")
    _check_tensor(dst_weights, torch.float32, (B, Hkv, dst_weights.shape[-1]), "dst_weights")
    _check_tensor(dst_seq_lens, torch.int32, (B,), "dst_seq_lens")
    _check_tensor(kept, torch.int32, (B, Hkv, max_dst * PAGE), "kept")
    dt = _dtype_code(cache_dtype)
    num_blocks = _check_cache(k_cache, v_cache, Hkv, head_dim, dt, per_token, num_blocks)
    (w, kc, vc, bt, lens, keep, dst, dst_w, dst_lens, src, status) = _device_ptrs(
        weights, k_cache, v_cache, block_table, seq_lens, keep_lens, dst_block_table, dst_weights, dst_seq_lens, kept,
        dev_status)
    _check(lib.kvq_evict_tokens(
        w, weights.shape[-1], kc, vc, bt, lens, keep, dst, dst_w, dst_weights.shape[-1], dst_lens, src, B, Hkv, head_dim,
        PAGE, max_blocks, max_dst, num_blocks, min(sink, 2**31 - 1), min(recent, 2**31 - 1), dt, 1 if per_token else 0,
        status, _stream(stream)), "kvq_evict_tokens")
    return dst_seq_lens


def _rows(t, T, D, name):
    """Heads and token stride (in elements) of tokens' heads, bf16 [T][heads][D]
    with any stride between tokens."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be bf16 [T][heads][{D}], got {t.dtype} {list(t.shape)}")
    tokens, heads, dim = t.shape
    stride, head_stride, dim_stride = t.stride()
    if dim != D:
        raise ValueError(f"{name} must be bf16 [T][heads][{D}], got {t.dtype} {list(t.shape)}")
    if tokens != T:
        raise ValueError(f"{name} must have {T} tokens like the others, got {tokens}")
    if dim_stride != 1 or (heads > 1 and head_stride != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return heads, stride if T > 1 else heads * D


def _addresses(*tensors):
    """Addresses of tensors on the current device, whose strides their user has
    checked (None for None)."""
    current = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.get_device() == current:
            out.append(t.data_ptr())
        elif t.get_device() < 0:
            raise ValueError("libkvq takes CUDA tensors only")
        else:
            raise ValueError(f"the tensors' device (cuda:{t.get_device()}) must be the current one (cuda:{current})")
    return out


def _check_dense(t, dtype, shape, name):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: libkvq takes contiguous tensors only")


def _check_turn(positions, inv_freq, pair_axis, q_weight, k_weight, T, D):
    """The shapes of the rotation's and norms' tensors; (axes, stride between
    their positions, pairs)."""
    if q_weight is not None:
        _check_dense(q_weight, torch.bfloat16, (D,), "q_weight")
    if k_weight is not None:
        _check_dense(k_weight, torch.bfloat16, (D,), "k_weight")
    if positions is None:
        if inv_freq is not None or pair_axis is not None:
            raise ValueError("inv_freq and pair_axis need positions")
        return 0, 0, 0
    shape, strides = positions.shape, positions.stride()
    axes = shape[0] if len(shape) == 2 else 1
    if positions.dtype is not torch.int64 or not 1 <= len(shape) <= 2 or shape[-1] != T:
        raise ValueError(f"positions must be int64 [{T}] or [axes][{T}], got {positions.dtype} {list(shape)}")
    if strides[-1] != 1 and T > 1:
        raise ValueError("positions: an axis's tokens must be contiguous")
    if inv_freq is None:
        raise ValueError("positions need inv_freq")
    pairs = inv_freq.numel()
    _check_dense(inv_freq, torch.float32, (pairs,), "inv_freq")
    if pair_axis is not None:
        _check_dense(pair_axis, torch.int32, (pairs,), "pair_axis")
    elif axes > 1:
        raise ValueError("several position axes need pair_axis")
    return axes, strides[0] if axes > 1 else T, pairs


def kvq_qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, pair_axis=None,
                     interleaved=False, rope_scale=1.0, dev_status=None, stream=None):
    """Head norms and rotary positions of queries and keys in one pass.

    q, k: bf16 [T][heads][D] with any stride between tokens (a slice of the
    projection's output), either may be None; q_out, k_out: alike, and may be q
    and k.  positions: int64 [T], or [axes][T] with pair_axis (int32 [pairs])
    naming each pair's axis; None: no rotation.  inv_freq: float32 [pairs],
    2 * pairs dims of each head are turned, pairs of dims pairs apart or
    (interleaved) neighbours.  q_weight, k_weight: bf16 [D] norm weights, None:
    no norm."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    T, _, D = x.shape
    Hq = qs = qos = Hkv = ks = kos = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        Hq, qs = _rows(q, T, D, "q")
        heads, qos = _rows(q_out, T, D, "q_out")
        if heads != Hq:
            raise ValueError("q_out must be shaped like q")
    if k is not None:
        if k_out is None:
            raise ValueError("k needs k_out")
        Hkv, ks = _rows(k, T, D, "k")
        heads, kos = _rows(k_out, T, D, "k_out")
        if heads != Hkv:
            raise ValueError("k_out must be shaped like k")
    axes, stride, pairs = _check_turn(positions, inv_freq, pair_axis, q_weight, k_weight, T, D)
    qp, kp, qop, kop, pos, freq, axis, qw, kw, status = _addresses(
        q, k, q_out if Hq else None, k_out if Hkv else None, positions, inv_freq, pair_axis, q_weight, k_weight, dev_status)
    norm = _HeadNorm(qw, kw, eps) if qw or kw else None
    rotary = _Rotary(pos, stride, freq, axis, axes, 2 * pairs, 1 if interleaved else 0, rope_scale) if axes else None
    _check(lib.kvq_qk_norm_rope(qp, qs, kp, ks, norm, rotary, qop, qos, kop, kos, T, Hq, Hkv, D, status, _stream(stream)),
           "kvq_qk_norm_rope")
    return q_out, k_out


def kvq_rope_and_cache(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None, q_out=None,
                       q8=None, q_scale=None, q_weight=None, k_weight=None, eps=1e-6, pair_axis=None, interleaved=False,
                       rope_scale=1.0, num_blocks=None, cache_dtype="fp8_e4m3", per_token=False, dev_status=None,
                       stream=None):
    """Head norms and rotary positions of q and k as kvq_qk_norm_rope, then k
    and v into the cache (any dtype of alloc_kv_cache, per_token: dynamic
    scales) and q out as bf16 (q_out, may be q) or E4M3 codes (q8 with q_scale)
    or both, in one launch.  q may be None."""
    T, _, D = k.shape
    Hkv, ks = _rows(k, T, D, "k")
    heads, vs = _rows(v, T, D, "v")
    if heads != Hkv:
        raise ValueError("v must be shaped like k")
    Hq = qs = qos = 0
    if q is not None:
        Hq, qs = _rows(q, T, D, "q")
        if q_out is not None:
            heads, qos = _rows(q_out, T, D, "q_out")
            if heads != Hq:
                raise ValueError("q_out must be shaped like q")
        elif q8 is None:
            raise ValueError("q needs q_out or q8")
        if q8 is not None:
            _check_dense(q8, torch.uint8, (T, Hq, D), "q8")
            if q_scale is None or q_scale.dtype is not torch.float32 or q_scale.numel() != 1:
                raise ValueError("q8 needs q_scale, float32 [1]")
    elif q_out is not None or q8 is not None:
        raise ValueError("q_out and q8 need q")
    _check_dense(slot_mapping, torch.int64, (T,), "slot_mapping")
    dt = _dtype_code(cache_dtype)
    num_blocks = _check_dense_cache(k_cache, v_cache, k_scale, v_scale, Hkv, D, dt, per_token, num_blocks)
    axes, stride, pairs = _check_turn(positions, inv_freq, pair_axis, q_weight, k_weight, T, D)
    qp, kp, vp, pos, freq, axis, qw, kw, slots, kc, vc, ksc, vsc, qop, q8p, qsc, status = _addresses(
        q, k, v, positions, inv_freq, pair_axis, q_weight, k_weight, slot_mapping, k_cache, v_cache, k_scale, v_scale, q_out,
        q8, q_scale, dev_status)
    norm = _HeadNorm(qw, kw, eps) if qw or kw else None
    rotary = _Rotary(pos, stride, freq, axis, axes, 2 * pairs, 1 if interleaved else 0, rope_scale) if axes else None
    _check(lib.kvq_rope_and_cache(qp, qs, kp, ks, vp, vs, norm, rotary, slots, kc, vc, ksc, vsc, qop, qos, q8p, qsc, T, Hq, Hkv,
                                  D, PAGE, num_blocks, dt, 1 if per_token else 0, status, _stream(stream)),
           "kvq_rope_and_cache")
    return q_out if q_out is not None else q8


def _check_dense_cache(k_cache, v_cache, k_scale, v_scale, Hkv, D, dt, per_token, num_blocks):
    """_check_scales and _check_cache for callers that take addresses as they
    are; returns the block count."""
    if k_scale is not None:
        _check_dense(k_scale, torch.float32, (Hkv,), "k_scale")
    if v_scale is not None:
        _check_dense(v_scale, torch.float32, (Hkv,), "v_scale")
    if not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("libkvq takes contiguous tensors only")
    return _check_cache(k_cache, v_cache, Hkv, D, dt, per_token, num_blocks)


def kvq_gather_cache(slot_mapping, k_cache, v_cache, k_out, v_out, k_scale=None, v_scale=None, num_blocks=None,
                     cache_dtype="fp8_e4m3", per_token=False, dev_status=None, stream=None):
    """The reverse of the cache writes: the tokens in the slots slot_mapping
    (int64 [T]) as bf16 k_out, v_out [T][Hkv][D]; rows of negative slots stay
    as they were."""
    T, Hkv, D = k_out.shape
    _check_dense(k_out, torch.bfloat16, (T, Hkv, D), "k_out")
    _check_dense(v_out, torch.bfloat16, (T, Hkv, D), "v_out")
    _check_dense(slot_mapping, torch.int64, (T,), "slot_mapping")
    dt = _dtype_code(cache_dtype)
    num_blocks = _check_dense_cache(k_cache, v_cache, k_scale, v_scale, Hkv, D, dt, per_token, num_blocks)
    *ptrs, status = _addresses(slot_mapping, k_cache, v_cache, k_scale, v_scale, k_out, v_out, dev_status)
    _check(lib.kvq_gather_cache(*ptrs, T, Hkv, D, PAGE, num_blocks, dt, 1 if per_token else 0, status, _stream(stream)),
           "kvq_gather_cache")
    return k_out, v_out


def kvq_decode_fp4_workspace_size(B, Hq, Hkv, D, max_blocks):
    return lib.kvq_decode_fp4_workspace_size(B, Hq, Hkv, D, PAGE, max_blocks)


def kvq_paged_decode_attention_fp4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, num_blocks=None,
                                   sm_scale=None, window=-1, workspace=None, dev_status=None, stream=None):
    """One decode step over a 4-bit cache (alloc_kv_cache(..., "fp4_e2m1"));
    writes out (bf16 [B][Hq][D]).  workspace: a uint8 CUDA tensor of at least
    kvq_decode_fp4_workspace_size() bytes (allocated here when omitted)."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    max_blocks = block_table.shape[1]
    _check_dense(q, torch.bfloat16, (B, Hq, D), "q")
    _check_dense(out, torch.bfloat16, (B, Hq, D), "out")
    _check_dense(block_table, torch.int32, (B, max_blocks), "block_table")
    _check_dense(seq_lens, torch.int32, (B,), "seq_lens")
    num_blocks = _check_dense_cache(k_cache, v_cache, k_scale, v_scale, Hkv, D, KVQ_DTYPE_FP4_E2M1, False, num_blocks)
    if workspace is None:
        workspace = _workspace(kvq_decode_fp4_workspace_size(B, Hq, Hkv, D, max_blocks), q, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace: libkvq takes contiguous tensors only")
    *ptrs, ws, status = _addresses(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, workspace, dev_status)
    _check(lib.kvq_paged_decode_attention_fp4(
        *ptrs, B, Hq, Hkv, D, PAGE, max_blocks, num_blocks, 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale),
        _window(window), ws, workspace.nbytes, status, _stream(stream)), "kvq_paged_decode_attention_fp4")
    return out
