"""Paged KV-cache decode attention for NVIDIA B200 (sm_100a).

A thin ctypes binding of ``libpagedkv.so`` (C ABI declared in ``include/pkv.h``).
Functions here only check and marshal torch tensors (device pointers, sizes,
dtypes, the current CUDA stream); every step of the computation runs in the
library's CUDA kernels. There is no CPU fallback: without the built library
(``python -m paged_kv_cache_462_b200.build``) every call raises.

Entry points (same names as the C ABI):

* ``reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, ...)`` — append
  the decode step's new K/V rows into their cache slots.
* ``paged_attention_decode(out, q, k_cache, v_cache, block_tables, seq_lens,
  scale, ...)`` — single-query grouped attention for every sequence, reading
  K/V block by block through the block table.
* ``qk_norm_rope`` / ``qk_norm_rope_and_cache`` — per-head RMS norm of queries and
  keys with the position rotation, and the append in the same pass.
* ``reshape_and_cache_block_scales`` / ``paged_attention_decode_block_scales`` — an
  8-bit cache with one scale for each block and KV head.
* ``update_key_bounds``, ``select_blocks``, ``paged_attention_decode_sparse`` — decode
  attention over the blocks a cheap score selects for each query.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpagedkv.so")

F32, BF16, FP8_E4M3, FP8_E5M2, INT8 = 0, 1, 2, 3, 4
DEVERR_BLOCK_ID, DEVERR_SEQ_LEN, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_PLAN = 1, 2, 4, 8, 16
DEVERR_ROWS, DEVERR_POSITION, DEVERR_SELECTION = 32, 64, 128

# uint8 caches hold E4M3 codes; E5M2 caches are passed as torch.float8_e5m2 tensors
_TORCH_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.uint8: FP8_E4M3, torch.float8_e4m3fn: FP8_E4M3,
                torch.float8_e5m2: FP8_E5M2, torch.int8: INT8}

_lib = None


class PkvError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


def load_library():
    """Load libpagedkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_462_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.paged_attention_workspace_size.restype = sz
    lib.pkv_workspace_init.argtypes = [P, sz, P]
    lib.pkv_workspace_init.restype = i32
    lib.paged_attention_decode.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32, i32,
                                           f32, f32, i32, P, sz, P]
    lib.paged_attention_decode.restype = i32
    lib.paged_decode_step.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32, i32,
                                      f32, f32, i32, P, sz, P, P, P, i32, P]
    lib.paged_decode_step.restype = i32
    lib.reshape_and_cache_head_scales.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, P]
    lib.reshape_and_cache_head_scales.restype = i32
    lib.paged_attention_decode_head_scales.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32,
                                                       i32, i32, P, P, i32, P, sz, P]
    lib.paged_attention_decode_head_scales.restype = i32
    lib.paged_attention_decode_mq.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                              i32, f32, f32, i32, P, sz, P]
    lib.paged_attention_decode_mq.restype = i32
    lib.pkv_test_decode_timeout.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32, i32,
                                            f32, f32, i32, P, sz, i32, P]
    lib.pkv_test_decode_timeout.restype = i32
    lib.reshape_and_cache.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, f32, f32, P, P]
    lib.reshape_and_cache.restype = i32
    lib.pkv_read_device_error.argtypes = [P, sz, ctypes.POINTER(ctypes.c_int32), i32, P]
    lib.pkv_read_device_error.restype = i32
    lib.pkv_default_partitions.argtypes = [i32, i32, i32, i32, i32]
    lib.pkv_default_partitions.restype = i32
    lib.pkv_set_fp8_kernel.argtypes = [i32]
    lib.pkv_set_fp8_kernel.restype = i32
    lib.paged_attention_shared_prefix_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.paged_attention_shared_prefix_workspace_size.restype = sz
    lib.paged_attention_decode_shared_prefix.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32,
                                                         i32, i32, f32, f32, P, P, P, P, P, i32, i32, i32, P, sz,
                                                         P]
    lib.paged_attention_decode_shared_prefix.restype = i32
    lib.paged_decode_step_shared_prefix.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                                    i32, f32, f32, P, P, P, P, P, i32, i32, i32, P, sz, P, P, P,
                                                    i32, P]
    lib.paged_decode_step_shared_prefix.restype = i32
    i64 = ctypes.c_int64
    lib.qk_norm_rope.argtypes = [P, P, P, P, P, P, f32, P, P, i32, i32, i32, i32, i32, i32, i32, i64, i64, i32, P, P]
    lib.qk_norm_rope.restype = i32
    lib.qk_norm_rope_and_cache.argtypes = [P, P, P, P, P, P, f32, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                           i32, i32, i64, i64, i64, i32, i32, f32, f32, P, P]
    lib.qk_norm_rope_and_cache.restype = i32
    lib.reshape_and_cache_block_scales.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i64,
                                                   i64, i32, i32, P, P]
    lib.reshape_and_cache_block_scales.restype = i32
    lib.paged_attention_decode_block_scales.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                                        i32, P, P, i32, P, sz, P]
    lib.paged_attention_decode_block_scales.restype = i32
    lib.update_key_bounds.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32, P, P, P]
    lib.update_key_bounds.restype = i32
    lib.pkv_select_workspace_size.argtypes = [i32, i32, i32]
    lib.pkv_select_workspace_size.restype = sz
    lib.select_blocks.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, P, sz, P]
    lib.select_blocks.restype = i32
    lib.paged_attention_decode_sparse.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                                  i32, i32, f32, f32, P, P, i32, P, sz, P]
    lib.paged_attention_decode_sparse.restype = i32
    lib.pkv_validate_tables.argtypes = [P, P, i32, i32, i32, i32, P, ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32)]
    lib.pkv_validate_tables.restype = i32
    lib.pkv_stream_recorded.argtypes = [P]
    lib.pkv_stream_recorded.restype = i32
    lib.pkv_status_string.argtypes = [i32]
    lib.pkv_status_string.restype = ctypes.c_char_p
    _bind_fast(lib)
    _lib = lib
    return lib


# The hot path of the operators that a serving loop calls once per layer (csrc/fastcall.cpp), where it
# is built: their C functions without ctypes' conversions, and the checks of a call's tensors in one
# go. What the module does not pass, the checks below look at one by one and explain.
_fast = None
_SPECS: dict = {}


def _bind_fast(lib) -> None:
    global _fast
    try:
        from . import _fastcall
    except ImportError:
        return
    if getattr(_fastcall, "torch_version", None) != torch.__version__:
        return
    for name in ("qk_norm_rope", "qk_norm_rope_and_cache", "reshape_and_cache_block_scales",
                 "paged_attention_decode_block_scales", "update_key_bounds", "select_blocks",
                 "paged_attention_decode_sparse", "pkv_stream_recorded"):
        _fastcall.bind(name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
        setattr(lib, name, getattr(_fastcall, name))
    caches = "k_cache:N,Hkv,B,D:c:K v_cache:N,Hkv,B,D:c:K"
    tables = "block_tables:S,M:c:i seq_lens:S:c:i"
    norm = ("q:T,Hq,D:rows:X k:T,Hkv,D:rows:X q_out:T,Hq,D:c:X q_weight:D:c:X k_weight:D:c:X cos_sin:P,R:c:f "
            "positions:T:c:l")
    decode = f"q:S,Hq,D:c:X out:S,Hq,D:c:X {caches} {tables}"
    _SPECS.update({name: _fastcall.spec(text) for name, text in {
        "norm": f"{norm} k_out:T,Hkv,D:c:X",
        "norm_cache": f"{norm} v:T,Hkv,D:rows:X {caches} slot_mapping:T:c:l",
        "append": f"k:T,Hkv,D:rows:X v:T,Hkv,D:rows:X {caches} k_scales:N,Hkv:c:f v_scales:N,Hkv:c:f {tables} "
                  "row_offsets:S+1:c:i",
        "decode": f"{decode} k_scales:N,Hkv:c:f v_scales:N,Hkv:c:f",
        "sparse": f"{decode} selected:S,Hkv,W:c:i ?k_scales:N,Hkv:c:f ?v_scales:N,Hkv:c:f",
        "bounds": f"key_bounds:N,Hkv,2,D:c:b k_cache:N,Hkv,B,D:c:K {tables} row_offsets:S+1:c:i ?k_scales:N,Hkv:c:f",
        "select": f"selected:S,Hkv,W:c:i q:S,Hq,D:c:b key_bounds:N,Hkv,2,D:c:b {tables}",
    }.items()})
    _fast = _fastcall


def _match(name, *tensors):
    """The pieces of a call's tensors (pointers, sizes in the spec's order, row strides, type codes, the
    device) if every check passes, else None."""
    load_library()
    return None if _fast is None else _fast.match(_SPECS[name], *tensors)


def status_string(status: int) -> str:
    return load_library().pkv_status_string(int(status)).decode()


def _check(fn, status):
    if status != 0:
        raise PkvError(fn, status)


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _TORCH_DTYPE[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _launch_device(name, t) -> int:
    """The current CUDA device (where the library launches), once `t` is known to be a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch.cuda.current_device()


def _cuda(name, t: torch.Tensor, dev: int | None = None):
    """Device pointer of a contiguous CUDA tensor on device `dev` (the current device, where the
    library launches; a tensor elsewhere would be read through a pointer this device cannot use)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev is not None and t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the current CUDA device is cuda:{dev}")
    return ctypes.c_void_p(t.data_ptr())


def workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, num_partitions=0) -> int:
    n = load_library().paged_attention_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, num_partitions)
    if n == 0:
        raise PkvError("paged_attention_workspace_size", 2)
    return int(n)


def new_workspace(num_seqs, num_heads, num_kv_heads, head_dim, num_partitions=0, device=None) -> torch.Tensor:
    """A zeroed (i.e. initialised) workspace tensor for paged_attention_decode."""
    n = workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, num_partitions)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check("pkv_workspace_init",
           load_library().pkv_workspace_init(_cuda("workspace", workspace), workspace.numel(), _stream_handle(stream)))


FP8_KERNEL_MMA = 0        # warp-level tensor cores on codes widened to f16 (the default)
FP8_KERNEL_TCGEN05 = 1    # fifth-generation tensor cores reading the 8-bit tiles (tcgen05.mma)


def set_fp8_kernel(which: int) -> int:
    """Process-wide kernel for FP8-cache decodes (pkv_set_fp8_kernel); returns the previous choice."""
    prev = load_library().pkv_set_fp8_kernel(int(which))
    if prev < 0:
        raise PkvError("pkv_set_fp8_kernel", -prev)
    return prev


def default_partitions(head_dim, block_size, num_heads, num_kv_heads, kv_dtype) -> int:
    code = kv_dtype if isinstance(kv_dtype, int) else _TORCH_DTYPE[kv_dtype]
    n = load_library().pkv_default_partitions(head_dim, block_size, num_heads, num_kv_heads, code)
    if n <= 0:
        raise PkvError("pkv_default_partitions", -n)
    return n


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                           k_scale=1.0, v_scale=1.0, num_partitions=0, workspace=None, stream=None) -> None:
    """out[s, g] = softmax(scale * q[s, g] . K) V over the seq_lens[s] cached tokens of sequence s.

    q, out: [num_seqs, num_heads, head_dim] (float32 or bfloat16);
    k_cache, v_cache: [num_blocks, num_kv_heads, block_size, head_dim]
    (float32, bfloat16, uint8/float8_e4m3fn E4M3 codes, float8_e5m2 codes or int8 codes, the
    8-bit ones with k_scale/v_scale);
    block_tables: int32 [num_seqs, max_blocks_per_seq]; seq_lens: int32 [num_seqs].
    """
    args, sizes, dev = _decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale,
                                    num_partitions)
    n = 0 if workspace is not None else workspace_size(*sizes, num_partitions)
    use = _workspace(workspace, n, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_attention_decode(*args, _cuda("workspace", ws, dev), ws.numel(),
                                                   _stream_handle(stream))
    _check("paged_attention_decode", st)


def _decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale, num_partitions):
    """Checked C arguments of a decode call, up to (not including) the workspace; the sizes that a
    workspace depends on; the device."""
    dev = _launch_device("q", q)
    S, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q/out and the caches")
    if out.dtype != q.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("out must match q's dtype and v_cache k_cache's")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    return ((_cuda("out", out, dev), _cuda("q", q, dev), _cuda("k_cache", k_cache, dev),
             _cuda("v_cache", v_cache, dev), _cuda("block_tables", block_tables, dev),
             _cuda("seq_lens", seq_lens, dev), S, Hq, Hkv, D, BS, float(scale),
             block_tables.shape[1], NB, _dtype_code(q), _dtype_code(k_cache), float(k_scale), float(v_scale),
             int(num_partitions)), (S, Hq, Hkv, D), dev)


def paged_attention_decode_mq(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale=1.0, v_scale=1.0,
                              num_partitions=0, workspace=None, stream=None) -> None:
    """q_len new tokens per sequence, causal within the chunk: q, out [num_seqs, q_len, num_heads, head_dim]
    (bf16); query j of sequence s sits at position seq_lens[s] - q_len + j and attends every token
    up to itself. The new tokens' K/V must already be in the cache."""
    dev = _launch_device("q", q)
    S, QL, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q/out and the caches")
    if out.dtype != q.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("out must match q's dtype and v_cache k_cache's")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    n = 0 if workspace is not None else workspace_size(S, Hq * QL, Hkv, D, num_partitions)
    use = _workspace(workspace, n, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_attention_decode_mq(
            _cuda("out", out, dev), _cuda("q", q, dev), _cuda("k_cache", k_cache, dev),
            _cuda("v_cache", v_cache, dev), _cuda("block_tables", block_tables, dev),
            _cuda("seq_lens", seq_lens, dev), S, QL, Hq, Hkv, D, BS, float(scale), block_tables.shape[1], NB,
            _dtype_code(q), _dtype_code(k_cache), float(k_scale), float(v_scale), int(num_partitions),
            _cuda("workspace", ws, dev), ws.numel(), _stream_handle(stream))
    _check("paged_attention_decode_mq", st)


def withheld_unit_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale, withheld_unit, workspace,
                        k_scale=1.0, v_scale=1.0, num_partitions=0, stream=None) -> None:
    """Failure-path test hook: paged_attention_decode with unit `withheld_unit`'s stage never handed
    to its consumers, so their bounded wait runs out and the workspace error word gets
    DEVERR_TIMEOUT (read it with read_device_error, then workspace_init before reuse)."""
    args, _, dev = _decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale,
                                num_partitions)
    st = load_library().pkv_test_decode_timeout(*args, _cuda("workspace", workspace, dev), workspace.numel(),
                                                int(withheld_unit), _stream_handle(stream))
    _check("pkv_test_decode_timeout", st)


def paged_decode_step(out, q, k_cache, v_cache, block_tables, seq_lens, new_k, new_v, slot_mapping, scale,
                      k_scale=1.0, v_scale=1.0, num_partitions=0, workspace=None, stream=None) -> None:
    """One decode step: append new_k/new_v row s at slot_mapping[s] (one new token per sequence,
    in its last block), then paged_attention_decode over the cache. One launch where the
    tensor-core decode kernel applies."""
    dev = _launch_device("q", q)
    S, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("shape mismatch between q/out and the caches")
    if tuple(new_k.shape) != (S, Hkv, D) or tuple(new_v.shape) != (S, Hkv, D) or new_v.dtype != new_k.dtype:
        raise ValueError("new_k/new_v must be [num_seqs, num_kv_heads, head_dim] of one dtype")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (S,):
        raise TypeError("slot_mapping must be int64 [num_seqs]")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    n = 0 if workspace is not None else workspace_size(S, Hq, Hkv, D, num_partitions)
    use = _workspace(workspace, n, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_decode_step(
            _cuda("out", out, dev), _cuda("q", q, dev), _cuda("k_cache", k_cache, dev),
            _cuda("v_cache", v_cache, dev), _cuda("block_tables", block_tables, dev),
            _cuda("seq_lens", seq_lens, dev), S, Hq, Hkv, D, BS, float(scale), block_tables.shape[1], NB,
            _dtype_code(q), _dtype_code(k_cache), float(k_scale), float(v_scale), int(num_partitions),
            _cuda("workspace", ws, dev), ws.numel(), _cuda("new_k", new_k, dev), _cuda("new_v", new_v, dev),
            _cuda("slot_mapping", slot_mapping, dev), _dtype_code(new_k), _stream_handle(stream))
    _check("paged_decode_step", st)


def reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, k_scale=1.0, v_scale=1.0,
                      device_error=None, stream=None) -> None:
    """Write k[t], v[t] ([num_tokens, num_kv_heads, head_dim]) into slot slot_mapping[t] of the caches."""
    dev = _launch_device("k", k)
    T, Hkv, D = k.shape
    NB, Hkv2, BS, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or tuple(v.shape) != tuple(k.shape) or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("shape mismatch between rows and caches")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise TypeError("slot_mapping must be int64 [num_tokens]")
    err = ctypes.c_void_p(_error_ptr(device_error, dev))
    st = load_library().reshape_and_cache(
        _cuda("k", k, dev), _cuda("v", v, dev), _cuda("k_cache", k_cache, dev), _cuda("v_cache", v_cache, dev),
        _cuda("slot_mapping", slot_mapping, dev), T, Hkv, D, BS, NB, _dtype_code(k), _dtype_code(k_cache),
        float(k_scale), float(v_scale), err, _stream_handle(stream))
    _check("reshape_and_cache", st)


def _head_scales(name, t, Hkv, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.shape != (Hkv,):
        raise TypeError(f"{name} must be a float32 tensor of num_kv_heads scales")
    return _cuda(name, t, dev)


def reshape_and_cache_head_scales(k, v, k_cache, v_cache, slot_mapping, k_head_scales, v_head_scales,
                                  device_error=None, stream=None) -> None:
    """reshape_and_cache into an 8-bit cache with one scale per KV head (float32 [num_kv_heads] tensors)."""
    dev = _launch_device("k", k)
    T, Hkv, D = k.shape
    NB, Hkv2, BS, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or tuple(v.shape) != tuple(k.shape) or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("shape mismatch between rows and caches")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise TypeError("slot_mapping must be int64 [num_tokens]")
    err = ctypes.c_void_p(_error_ptr(device_error, dev))
    st = load_library().reshape_and_cache_head_scales(
        _cuda("k", k, dev), _cuda("v", v, dev), _cuda("k_cache", k_cache, dev), _cuda("v_cache", v_cache, dev),
        _cuda("slot_mapping", slot_mapping, dev), T, Hkv, D, BS, NB, _dtype_code(k), _dtype_code(k_cache),
        _head_scales("k_head_scales", k_head_scales, Hkv, dev), _head_scales("v_head_scales", v_head_scales, Hkv, dev),
        err, _stream_handle(stream))
    _check("reshape_and_cache_head_scales", st)


def paged_attention_decode_head_scales(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_head_scales,
                                       v_head_scales, num_partitions=0, workspace=None, stream=None) -> None:
    """paged_attention_decode over an 8-bit cache with one scale per KV head."""
    args, sizes, dev = _decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, scale, 1.0, 1.0, num_partitions)
    Hkv = k_cache.shape[1]
    args = (*args[:16], _head_scales("k_head_scales", k_head_scales, Hkv, dev),
            _head_scales("v_head_scales", v_head_scales, Hkv, dev), *args[18:])
    n = 0 if workspace is not None else workspace_size(*sizes, num_partitions)
    use = _workspace(workspace, n, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_attention_decode_head_scales(*args, _cuda("workspace", ws, dev), ws.numel(),
                                                               _stream_handle(stream))
    _check("paged_attention_decode_head_scales", st)


def read_device_error(workspace: torch.Tensor | None = None, clear: bool = False, stream=None) -> int:
    """The workspace's device error word (PKV_DEVERR_* bits); synchronises the stream. Without a workspace:
    the bits of all that the binding keeps for calls on `stream` of the current device. Cleared after
    DEVERR_TIMEOUT, a kept workspace is initialised anew, as one of the caller's has to be. (Calls captured
    without a workspace have one of the graph's own, which is not among them: give those calls one.)"""
    if workspace is not None:
        return _error_word(workspace, clear, _stream_handle(stream))
    dev = torch.cuda.current_device()
    handle = _raw_stream(stream, dev)
    bits = 0
    for kept in ([k for (_, d, st), k in list(_op_ws.items()) if (d, st) == (dev, handle)] +
                 [k for (d, _, st), k in list(_ws_cache.items()) if (d, st or 0) == (dev, handle)]):
        with kept.lock:
            if kept.tensor is None:
                continue
            word = _error_word(kept.tensor, clear, ctypes.c_void_p(handle))
            if clear and word & DEVERR_TIMEOUT:
                workspace_init(kept.tensor, handle)
            bits |= word
    return bits


def _error_word(workspace, clear, handle) -> int:
    v = ctypes.c_int32(0)
    _check("pkv_read_device_error", load_library().pkv_read_device_error(
        _cuda("workspace", workspace), workspace.numel(), ctypes.byref(v), int(clear), handle))
    return int(v.value)


class DevicePrefixPlan:
    """A shared-prefix plan (``blocks.prefix_plan``'s result) copied to the device as the
    shared-prefix decode reads it: int32 members, offsets [groups + 1], tables [groups, max_blocks],
    lens [groups], shared [num_seqs]; ``max_group`` is the planner's group-size limit."""

    def __init__(self, plan, max_group: int, device=None):
        import numpy as np
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)
        self.num_groups = int(plan.num_groups)
        self.max_group = int(max_group)
        self.members = t(plan.members)
        self.offsets = t(plan.offsets[: self.num_groups + 1])
        self.tables = t(plan.tables[: self.num_groups])
        self.lens = t(plan.lens[: self.num_groups])
        self.shared = t(plan.shared)

    def tensors(self):
        return (self.members, self.offsets, self.tables, self.lens, self.shared)


def shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, num_partitions=0) -> int:
    n = load_library().paged_attention_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                                    num_groups, num_partitions)
    if n == 0:
        raise PkvError("paged_attention_shared_prefix_workspace_size", 2)
    return int(n)


def new_shared_prefix_workspace(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, num_partitions=0,
                                device=None) -> torch.Tensor:
    """A zeroed workspace for the shared-prefix decode."""
    n = shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, num_groups, num_partitions)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _plan_args(plan: DevicePrefixPlan, dev, S, MB):
    if not isinstance(plan, DevicePrefixPlan):
        raise TypeError("plan must be a DevicePrefixPlan")
    if plan.shared.shape != (S,) or (plan.num_groups and plan.tables.shape[1] != MB):
        raise ValueError("plan does not match the batch (shared [num_seqs], tables [groups, max_blocks])")
    ptr = lambda name, t: _cuda(name, t, dev) if t.numel() else ctypes.c_void_p(None)
    return (ptr("plan.members", plan.members), ptr("plan.offsets", plan.offsets), ptr("plan.tables", plan.tables),
            ptr("plan.lens", plan.lens), _cuda("plan.shared", plan.shared, dev), plan.num_groups, plan.max_group)


def _shared_prefix_workspace(workspace, S, Hq, Hkv, D, plan, num_partitions, dev, stream):
    n = 0 if workspace is not None else shared_prefix_workspace_size(S, Hq, Hkv, D, plan.num_groups, num_partitions)
    return _op_workspace(workspace, "shared_prefix", n, dev, _raw_stream(stream, dev)), n


def paged_attention_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, seq_lens, plan, scale,
                                         k_scale=1.0, v_scale=1.0, num_partitions=0, workspace=None,
                                         stream=None) -> None:
    """paged_attention_decode with the blocks a plan shares read once per group (a prefix pass over
    the groups' shared rows, a suffix pass over each sequence's own blocks, a log-sum-exp merge)."""
    dev = _launch_device("q", q)
    S, Hq, D = q.shape
    NB, Hkv, BS, _ = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape) or k_cache.shape[3] != D:
        raise ValueError("shape mismatch between q/out and the caches")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks] and seq_lens int32 [num_seqs]")
    use, n = _shared_prefix_workspace(workspace, S, Hq, Hkv, D, plan, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_attention_decode_shared_prefix(
            _cuda("out", out, dev), _cuda("q", q, dev), _cuda("k_cache", k_cache, dev),
            _cuda("v_cache", v_cache, dev), _cuda("block_tables", block_tables, dev),
            _cuda("seq_lens", seq_lens, dev), S, Hq, Hkv, D, BS, float(scale), block_tables.shape[1], NB,
            _dtype_code(q), _dtype_code(k_cache), float(k_scale), float(v_scale),
            *_plan_args(plan, dev, S, block_tables.shape[1]), int(num_partitions), _cuda("workspace", ws, dev),
            ws.numel(), _stream_handle(stream))
    _check("paged_attention_decode_shared_prefix", st)


def paged_decode_step_shared_prefix(out, q, k_cache, v_cache, block_tables, seq_lens, plan, new_k, new_v,
                                    slot_mapping, scale, k_scale=1.0, v_scale=1.0, num_partitions=0, workspace=None,
                                    stream=None) -> None:
    """paged_decode_step with the shared-prefix decode (the append rides in the suffix pass)."""
    dev = _launch_device("q", q)
    S, Hq, D = q.shape
    NB, Hkv, BS, _ = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape) or k_cache.shape[3] != D:
        raise ValueError("shape mismatch between q/out and the caches")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks] and seq_lens int32 [num_seqs]")
    if tuple(new_k.shape) != (S, Hkv, D) or tuple(new_v.shape) != (S, Hkv, D) or new_v.dtype != new_k.dtype:
        raise ValueError("new_k/new_v must be [num_seqs, num_kv_heads, head_dim] of one dtype")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (S,):
        raise TypeError("slot_mapping must be int64 [num_seqs]")
    use, n = _shared_prefix_workspace(workspace, S, Hq, Hkv, D, plan, num_partitions, dev, stream)
    with use.lock:
        ws = use.ready(n)
        st = load_library().paged_decode_step_shared_prefix(
            _cuda("out", out, dev), _cuda("q", q, dev), _cuda("k_cache", k_cache, dev),
            _cuda("v_cache", v_cache, dev), _cuda("block_tables", block_tables, dev),
            _cuda("seq_lens", seq_lens, dev), S, Hq, Hkv, D, BS, float(scale), block_tables.shape[1], NB,
            _dtype_code(q), _dtype_code(k_cache), float(k_scale), float(v_scale),
            *_plan_args(plan, dev, S, block_tables.shape[1]), int(num_partitions), _cuda("workspace", ws, dev),
            ws.numel(), _cuda("new_k", new_k, dev), _cuda("new_v", new_v, dev),
            _cuda("slot_mapping", slot_mapping, dev), _dtype_code(new_k), _stream_handle(stream))
    _check("paged_decode_step_shared_prefix", st)


def validate_tables(block_tables, seq_lens, block_size: int, num_blocks: int, slot_mapping=None):
    """Host check of a batch's tables (numpy or CPU tensors): (PKV_DEVERR_* bits found, first
    offending sequence or -1). See pkv_validate_tables."""
    import numpy as np
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    sm = None if slot_mapping is None else np.ascontiguousarray(slot_mapping, dtype=np.int64)
    if bt.ndim != 2 or bt.shape[0] != sl.shape[0] or (sm is not None and sm.shape != sl.shape):
        raise ValueError("block_tables [n, max_blocks], seq_lens [n], slot_mapping [n]")
    bits, first = ctypes.c_int32(0), ctypes.c_int32(-1)
    _check("pkv_validate_tables", load_library().pkv_validate_tables(
        bt.ctypes.data, sl.ctypes.data, sl.shape[0], max(1, bt.shape[1]), int(block_size), int(num_blocks),
        None if sm is None else sm.ctypes.data, ctypes.byref(bits), ctypes.byref(first)))
    return int(bits.value), int(first.value)


# The operators below are called once per layer and step: their checks read each property once.

def _current_raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return _current_raw_stream(dev)
    return int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)


def _ptr(name, t, dev):
    """Device pointer of a contiguous CUDA tensor on device `dev`, as _cuda checks it."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _cuda(name, t, dev).value


def _error_ptr(t, dev):
    """Pointer of the int32 word that a call sets its error bits in (None: none): four bytes, aligned."""
    if t is None:
        return None
    at = _ptr("device_error", t, dev)
    if t.dtype != torch.int32 or t.numel() < 1:
        raise TypeError("device_error must be an int32 tensor of one element or more")
    return at


def _rows(name, t, dev, heads=None, dim=None, dtype=None):
    """(device pointer, tokens, heads, head_dim, token stride) of rows [tokens, heads, head_dim] whose
    heads are contiguous; tokens may lie further apart (a view of a projection's output)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [num_tokens, heads, head_dim]")
    T, H, D = t.shape
    if (heads is not None and H != heads) or (dim is not None and D != dim):
        raise ValueError(f"{name} has another number of heads or another head_dim")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != dev and t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the current CUDA device is cuda:{dev}")
    s0, s1, s2 = t.stride()
    if T > 0 and (s2 != 1 or (H > 1 and s1 != D)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if T > 1 and s0 < H * D:
        raise ValueError(f"{name}: tokens must not share elements")
    return t.data_ptr(), T, H, D, (s0 if T > 1 else H * D)


def _norm_rope_args(q_out, q, k, q_weight, k_weight, cos_sin, positions, dev):
    """Checked pieces that qk_norm_rope and qk_norm_rope_and_cache share."""
    dt = q.dtype
    qp, T, Hq, D, qs = _rows("q", q, dev)
    kp, Tk, Hkv, _, ks = _rows("k", k, dev, dim=D, dtype=dt)
    if Tk != T or q_out.shape != (T, Hq, D):
        raise ValueError("shape mismatch between q, k and q_out")
    if q_out.dtype != dt or q_weight.dtype != dt or k_weight.dtype != dt:
        raise TypeError("q_out and the weights must have q's dtype")
    if q_weight.shape != (D,) or k_weight.shape != (D,):
        raise ValueError("the weights must be [head_dim]")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2:
        raise TypeError("cos_sin must be float32 [num_positions, rotary_dim]")
    if positions.dtype != torch.int64 or positions.shape != (T,):
        raise TypeError("positions must be int64 [num_tokens]")
    return (qp, kp, T, Hq, Hkv, D, qs, ks, _ptr("q_out", q_out, dev), _ptr("q_weight", q_weight, dev),
            _ptr("k_weight", k_weight, dev), _ptr("cos_sin", cos_sin, dev), _ptr("positions", positions, dev),
            *cos_sin.shape, _dtype_code(q))


def qk_norm_rope(q_out, k_out, q, k, q_weight, k_weight, eps, cos_sin, positions, interleaved=False,
                 device_error=None, stream=None) -> None:
    """q_out, k_out = rotate(rms_norm(q) * q_weight), rotate(rms_norm(k) * k_weight), head by head.

    q [num_tokens, num_heads, head_dim], k [num_tokens, num_kv_heads, head_dim] (float32 or bfloat16;
    views of a larger projection output are fine); q_out, k_out contiguous, or q and k themselves;
    weights [head_dim]; cos_sin float32 [num_positions, rotary_dim] (cosines, then sines);
    positions int64 [num_tokens]."""
    m = _match("norm", q, k, q_out, q_weight, k_weight, cos_sin, positions, k_out)
    if m is not None:
        qp, kp, qo, qw, kw, cs, pos, ko, T, Hq, D, Hkv, NP, R, qs, ks, dt, dev = m
    else:
        dev = _launch_device("q", q)
        qp, kp, T, Hq, Hkv, D, qs, ks, qo, qw, kw, cs, pos, NP, R, dt = _norm_rope_args(
            q_out, q, k, q_weight, k_weight, cos_sin, positions, dev)
        if k_out.shape != (T, Hkv, D) or k_out.dtype != q.dtype:
            raise ValueError("k_out must match k")
        ko = _ptr("k_out", k_out, dev)
    _check("qk_norm_rope", load_library().qk_norm_rope(
        qo, ko, qp, kp, qw, kw, float(eps), cs, pos, T, Hq, Hkv, D, R, NP, bool(interleaved), qs, ks, dt,
        _error_ptr(device_error, dev), _raw_stream(stream, dev)))


def qk_norm_rope_and_cache(q_out, q, k, v, q_weight, k_weight, eps, cos_sin, positions, k_cache, v_cache,
                           slot_mapping, interleaved=False, k_scale=1.0, v_scale=1.0, device_error=None,
                           stream=None) -> None:
    """qk_norm_rope with the append of reshape_and_cache in the same pass: the new keys and the rows
    of v go to slot slot_mapping[t] of the caches (a negative slot appends nothing)."""
    m = _match("norm_cache", q, k, q_out, q_weight, k_weight, cos_sin, positions, v, k_cache, v_cache, slot_mapping)
    if m is not None:
        (qp, kp, qo, qw, kw, cs, pos, vp, kc, vc, sm, T, Hq, D, Hkv, NP, R, NB, BS, qs, ks, vs, dt, kdt, dev) = m
    else:
        dev = _launch_device("q", q)
        qp, kp, T, Hq, Hkv, D, qs, ks, qo, qw, kw, cs, pos, NP, R, dt = _norm_rope_args(
            q_out, q, k, q_weight, k_weight, cos_sin, positions, dev)
        vp, Tv, _, _, vs = _rows("v", v, dev, heads=Hkv, dim=D, dtype=q.dtype)
        shape = k_cache.shape
        NB, Hkv2, BS, D2 = shape
        if Tv != T or Hkv2 != Hkv or D2 != D or v_cache.shape != shape:
            raise ValueError("shape mismatch between rows and caches")
        if v_cache.dtype != k_cache.dtype:
            raise TypeError("v_cache must have k_cache's dtype")
        if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
            raise TypeError("slot_mapping must be int64 [num_tokens]")
        kc, vc, kdt = _ptr("k_cache", k_cache, dev), _ptr("v_cache", v_cache, dev), _dtype_code(k_cache)
        sm = _ptr("slot_mapping", slot_mapping, dev)
    _check("qk_norm_rope_and_cache", load_library().qk_norm_rope_and_cache(
        qo, qp, kp, vp, qw, kw, float(eps), cs, pos, kc, vc, sm, T, Hq, Hkv, D, R, NP, BS, NB, bool(interleaved), qs,
        ks, vs, dt, kdt, float(k_scale), float(v_scale), _error_ptr(device_error, dev),
        _raw_stream(stream, dev)))


def _tables(block_tables, seq_lens, dev):
    """Checked (block_tables pointer, seq_lens pointer, num_seqs, max_blocks)."""
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    shape = block_tables.shape
    if len(shape) != 2 or seq_lens.shape != shape[:1]:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    return _ptr("block_tables", block_tables, dev), _ptr("seq_lens", seq_lens, dev), shape[0], shape[1]


def _block_scales(name, t, cache_shape, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.shape != cache_shape[:2]:
        raise TypeError(f"{name} must be a float32 tensor [num_blocks, num_kv_heads]")
    return _ptr(name, t, dev)


def _row_offsets(t, S, dev):
    if t.dtype != torch.int32 or t.shape != (S + 1,):
        raise TypeError("row_offsets must be int32 [num_seqs + 1]")
    return _ptr("row_offsets", t, dev)


def reshape_and_cache_block_scales(k, v, k_cache, v_cache, k_block_scales, v_block_scales, block_tables, seq_lens,
                                   row_offsets, device_error=None, stream=None) -> None:
    """Append rows to an 8-bit cache with one power-of-two scale for each (block, KV head).

    k, v [num_tokens, num_kv_heads, head_dim]: rows row_offsets[s] .. row_offsets[s + 1] - 1 are the
    newest tokens of sequence s, which has seq_lens[s] tokens with them. The scales (float32
    [num_blocks, num_kv_heads]) of the blocks they fall into are set, or grow (and the block's older
    codes with them) where the block already holds tokens of the sequence."""
    m = _match("append", k, v, k_cache, v_cache, k_block_scales, v_block_scales, block_tables, seq_lens, row_offsets)
    if m is not None:
        kp, vp, kc, vc, kbs, vbs, bt, sl, ro, T, Hkv, D, NB, BS, S, MB, ks, vs, dt, kdt, dev = m
    else:
        dev = _launch_device("k", k)
        kp, T, Hkv, D, ks = _rows("k", k, dev)
        vp, Tv, _, _, vs = _rows("v", v, dev, heads=Hkv, dim=D, dtype=k.dtype)
        shape = k_cache.shape
        NB, Hkv2, BS, D2 = shape
        if Tv != T or Hkv2 != Hkv or D2 != D or v_cache.shape != shape:
            raise ValueError("shape mismatch between rows and caches")
        if v_cache.dtype != k_cache.dtype:
            raise TypeError("v_cache must have k_cache's dtype")
        bt, sl, S, MB = _tables(block_tables, seq_lens, dev)
        ro = _row_offsets(row_offsets, S, dev)
        kbs = _block_scales("k_block_scales", k_block_scales, shape, dev)
        vbs = _block_scales("v_block_scales", v_block_scales, shape, dev)
        kc, vc = _ptr("k_cache", k_cache, dev), _ptr("v_cache", v_cache, dev)
        dt, kdt = _dtype_code(k), _dtype_code(k_cache)
    _check("reshape_and_cache_block_scales", load_library().reshape_and_cache_block_scales(
        kp, vp, kc, vc, kbs, vbs, bt, sl, ro, T, S, Hkv, D, BS, MB, NB, ks, vs, dt, kdt,
        _error_ptr(device_error, dev), _raw_stream(stream, dev)))


def _decode_shapes(out, q, k_cache, v_cache, block_tables, seq_lens, dev):
    """Checked sizes and pointers of a decode: (num_seqs, num_heads, head_dim, cache shape, out, q, k_cache,
    v_cache, block_tables, seq_lens, max_blocks)."""
    shape, cache = q.shape, k_cache.shape
    S, Hq, D = shape
    if cache[3] != D or v_cache.shape != cache or out.shape != shape:
        raise ValueError("shape mismatch between q/out and the caches")
    if out.dtype != q.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("out must match q's dtype and v_cache k_cache's")
    bt, sl, S2, MB = _tables(block_tables, seq_lens, dev)
    if S2 != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
    return (S, Hq, D, cache, _ptr("out", out, dev), _ptr("q", q, dev), _ptr("k_cache", k_cache, dev),
            _ptr("v_cache", v_cache, dev), bt, sl, MB)


def paged_attention_decode_block_scales(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_block_scales,
                                        v_block_scales, num_partitions=0, workspace=None, stream=None) -> None:
    """paged_attention_decode over an 8-bit cache with one scale for each (block, KV head):
    k_block_scales, v_block_scales float32 [num_blocks, num_kv_heads], positive."""
    m = _match("decode", q, out, k_cache, v_cache, block_tables, seq_lens, k_block_scales, v_block_scales)
    if m is not None:
        qp, op, kp, vp, bt, sl, ks, vs, S, Hq, D, NB, Hkv, BS, MB, dt, kdt, dev = m
    else:
        dev = _launch_device("q", q)
        S, Hq, D, cache, op, qp, kp, vp, bt, sl, MB = _decode_shapes(out, q, k_cache, v_cache, block_tables, seq_lens,
                                                                     dev)
        NB, Hkv, BS, _ = cache
        ks = _block_scales("k_block_scales", k_block_scales, cache, dev)
        vs = _block_scales("v_block_scales", v_block_scales, cache, dev)
        dt, kdt = _dtype_code(q), _dtype_code(k_cache)
    st = _raw_stream(stream, dev)
    n = 0 if workspace is not None else _sized(workspace_size, dev, S, Hq, Hkv, D, num_partitions)
    use = _op_workspace(workspace, "decode", n, dev, st)
    with use.lock:
        ws = use.ready(n)
        _check("paged_attention_decode_block_scales", load_library().paged_attention_decode_block_scales(
            op, qp, kp, vp, bt, sl, S, Hq, Hkv, D, BS, float(scale), MB, NB, dt, kdt, ks, vs, int(num_partitions),
            _ptr("workspace", ws, dev), ws.numel(), st))


def update_key_bounds(key_bounds, k_cache, block_tables, seq_lens, row_offsets, num_tokens, k_scale=1.0,
                      k_block_scales=None, device_error=None, stream=None) -> None:
    """Refresh key_bounds (bfloat16 [num_blocks, num_kv_heads, 2, head_dim]: maxima, minima over a
    block's keys) for the blocks that hold the num_tokens newest tokens of a batch, after their
    append; row_offsets as in reshape_and_cache_block_scales (int32 [num_seqs + 1])."""
    m = _match("bounds", key_bounds, k_cache, block_tables, seq_lens, row_offsets, k_block_scales)
    if m is not None:
        kb, kc, bt, sl, ro, scales, NB, Hkv, D, BS, S, MB, kdt, dev = m
    else:
        dev = _launch_device("k_cache", k_cache)
        shape = k_cache.shape
        NB, Hkv, BS, D = shape
        if key_bounds.dtype != torch.bfloat16 or key_bounds.shape != (NB, Hkv, 2, D):
            raise TypeError("key_bounds must be bfloat16 [num_blocks, num_kv_heads, 2, head_dim]")
        bt, sl, S, MB = _tables(block_tables, seq_lens, dev)
        ro = _row_offsets(row_offsets, S, dev)
        scales = None if k_block_scales is None else _block_scales("k_block_scales", k_block_scales, shape, dev)
        kb, kc, kdt = _ptr("key_bounds", key_bounds, dev), _ptr("k_cache", k_cache, dev), _dtype_code(k_cache)
    _check("update_key_bounds", load_library().update_key_bounds(
        kb, kc, bt, sl, ro, int(num_tokens), S, Hkv, D, BS, MB, NB, kdt, float(k_scale), scales or None,
        _error_ptr(device_error, dev), _raw_stream(stream, dev)))


def select_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq) -> int:
    n = load_library().pkv_select_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq)
    if n == 0:
        raise PkvError("pkv_select_workspace_size", 2)
    return int(n)


def new_select_workspace(num_seqs, num_kv_heads, max_blocks_per_seq, device=None) -> torch.Tensor:
    """A zeroed workspace for select_blocks."""
    n = select_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def select_blocks(selected, q, key_bounds, block_tables, seq_lens, block_size, num_sink_blocks=1,
                  num_recent_blocks=1, workspace=None, stream=None) -> None:
    """selected[s, h] (int32 [num_seqs, num_kv_heads, num_selected]) = the logical blocks KV head h's
    queries may need most, ascending, -1 behind where the sequence has fewer: the first
    num_sink_blocks, the last num_recent_blocks and the highest scores of the rest, a block's score
    being the bound that key_bounds sets to its keys' products with the group's queries (first of
    all, blocks with bounds that are not finite).
    q bfloat16 [num_seqs, num_heads, head_dim]."""
    m = _match("select", selected, q, key_bounds, block_tables, seq_lens)
    if m is not None:
        sel, qp, kb, bt, sl, S, Hkv, W, Hq, D, NB, MB, dev = m
    else:
        dev = _launch_device("q", q)
        S, Hq, D = q.shape
        NB, Hkv, two, D2 = key_bounds.shape
        if q.dtype != torch.bfloat16 or key_bounds.dtype != torch.bfloat16:
            raise TypeError("q and key_bounds must be bfloat16")
        if two != 2 or D2 != D:
            raise ValueError("key_bounds must be [num_blocks, num_kv_heads, 2, head_dim]")
        W = _selected_width(selected, S, Hkv)
        bt, sl, S2, MB = _tables(block_tables, seq_lens, dev)
        if S2 != S:
            raise ValueError("block_tables must be [num_seqs, max_blocks] and seq_lens [num_seqs]")
        sel, qp, kb = _ptr("selected", selected, dev), _ptr("q", q, dev), _ptr("key_bounds", key_bounds, dev)
    st = _raw_stream(stream, dev)
    n = 0 if workspace is not None else _sized(select_workspace_size, dev, S, Hkv, max(1, MB))
    use = _op_workspace(workspace, "select", n, dev, st)
    with use.lock:
        ws = use.ready(n)
        _check("select_blocks", load_library().select_blocks(
            sel, qp, kb, bt, sl, S, Hq, Hkv, D, int(block_size), MB, NB, W, int(num_sink_blocks),
            int(num_recent_blocks), _ptr("workspace", ws, dev), ws.numel(), st))


def _selected_width(selected, S, Hkv) -> int:
    shape = selected.shape
    if selected.dtype != torch.int32 or len(shape) != 3 or shape[0] != S or shape[1] != Hkv:
        raise TypeError("selected must be int32 [num_seqs, num_kv_heads, num_selected]")
    return shape[2]


def paged_attention_decode_sparse(out, q, k_cache, v_cache, block_tables, seq_lens, selected, scale, k_scale=1.0,
                                  v_scale=1.0, k_block_scales=None, v_block_scales=None, num_partitions=0,
                                  workspace=None, stream=None) -> None:
    """paged_attention_decode over the tokens of the listed blocks only: selected int32 [num_seqs,
    num_kv_heads, num_selected] (select_blocks' output), negative entries empty. 8-bit caches take
    per-tensor scales or both block scales."""
    if (k_block_scales is None) != (v_block_scales is None):
        raise ValueError("give both block scales or none")
    m = _match("sparse", q, out, k_cache, v_cache, block_tables, seq_lens, selected, k_block_scales, v_block_scales)
    if m is not None:
        qp, op, kp, vp, bt, sl, sel, ks, vs, S, Hq, D, NB, Hkv, BS, MB, W, dt, kdt, dev = m
    else:
        dev = _launch_device("q", q)
        S, Hq, D, cache, op, qp, kp, vp, bt, sl, MB = _decode_shapes(out, q, k_cache, v_cache, block_tables, seq_lens,
                                                                     dev)
        NB, Hkv, BS, _ = cache
        W = _selected_width(selected, S, Hkv)
        ks = vs = None
        if k_block_scales is not None:
            ks = _block_scales("k_block_scales", k_block_scales, cache, dev)
            vs = _block_scales("v_block_scales", v_block_scales, cache, dev)
        sel, dt, kdt = _ptr("selected", selected, dev), _dtype_code(q), _dtype_code(k_cache)
    st = _raw_stream(stream, dev)
    n = 0 if workspace is not None else _sized(workspace_size, dev, S, Hq, Hkv, D, num_partitions)
    use = _op_workspace(workspace, "decode", n, dev, st)
    with use.lock:
        ws = use.ready(n)
        _check("paged_attention_decode_sparse", load_library().paged_attention_decode_sparse(
            op, qp, kp, vp, bt, sl, sel, S, Hq, Hkv, D, BS, float(scale), MB, NB, W, dt, kdt, float(k_scale),
            float(v_scale), ks or None, vs or None, int(num_partitions), _ptr("workspace", ws, dev), ws.numel(), st))


_sizes: dict = {}


def _sized(size, dev, *args) -> int:
    """size(*args), remembered: a workspace's size depends on these numbers and the device alone."""
    n = _sizes.get((size, dev, args))
    if n is None:
        n = size(*args)
        if len(_sizes) < 4096:
            _sizes[(size, dev, args)] = n
    return n


class _Kept:
    """A workspace that the binding keeps for one stream, and its lock: a call holds it from the choice of the
    workspace until its launches are queued. They are two that hand over through the workspace, and the
    C call lets other threads run: their launches on the same stream would go in between."""
    __slots__ = ("tensor", "lock", "new", "args")

    def __init__(self, new, *args):
        self.tensor = None
        self.lock = threading.RLock()
        self.new, self.args = new, args

    def ready(self, n):
        """The workspace, of n bytes at least (the lock is held)."""
        if self.tensor is None or self.tensor.numel() < n:
            self.tensor = self.new(n, self.tensor, *self.args)
        return self.tensor


class _Given:
    """A workspace that one call alone uses, or that its caller answers for."""
    __slots__ = ("tensor",)
    lock = contextlib.nullcontext()

    def __init__(self, tensor):
        self.tensor = tensor

    def ready(self, n):
        return self.tensor


def _kept(table, key, new, *args) -> _Kept:
    """What `table` keeps under `key`; new(n, old, *args) makes its workspaces."""
    kept = table.get(key)
    return kept if kept is not None else table.setdefault(key, _Kept(new, *args))


def _recorded(stream, current) -> bool:
    """Whether calls on `stream` are being recorded into a graph. If either it or the current stream is, but not
    both as one, a workspace could come from the wrong place: memory of the graph that eager calls
    keep, or kept memory that the graph would go on using after a larger workspace has replaced it."""
    recorded = load_library().pkv_stream_recorded
    here = recorded(current) != 0
    if stream != current and (here or recorded(stream) != 0):
        raise ValueError("pass a workspace to capture on another stream than the current one")
    return here


_op_ws: dict = {}
_HEADER = 512        # what a workspace needs cleared before its first call: header and first arrival counters


def _op_workspace(workspace, kind, n, dev, stream):
    """The caller's workspace, or one of at least n bytes with a clear header, kept per (kind, device,
    stream), so that calls on different streams never share one. It is allocated and cleared on the
    stream that uses it. While that stream is being captured every call gets its own, from the
    graph's memory and cleared inside the graph: two graphs, or a graph and later eager calls, never
    meet in one."""
    if workspace is not None:
        return _Given(workspace)
    if _recorded(stream, _current_raw_stream(dev)):
        return _Given(_new_op_workspace(n, None, dev, stream))
    return _kept(_op_ws, (kind, dev, stream), _new_op_workspace, dev, stream)


def _new_op_workspace(n, _, dev, stream):
    here = stream == _current_raw_stream(dev)
    with torch.cuda.stream(torch.cuda.current_stream() if here else torch.cuda.ExternalStream(stream, device=dev)):
        ws = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev))
    _check("pkv_workspace_init", load_library().pkv_workspace_init(_ptr("workspace", ws, dev), min(n, _HEADER),
                                                                   stream))
    return ws


_ws_cache: dict = {}


def _workspace(workspace, n, parts, dev, stream):
    """The caller's workspace, or one kept per (device, partitions, stream), so calls on different streams
    never share one; a new one is zeroed by the library on the stream that will use it. While that
    stream is being captured every call gets its own, as in _op_workspace."""
    if workspace is not None:
        return _Given(workspace)
    handle = _stream_handle(stream)
    if _recorded(handle.value or 0, torch.cuda.current_stream().cuda_stream):
        return _Given(_new_op_workspace(n, None, dev, handle.value or 0))
    return _kept(_ws_cache, (dev, parts, handle.value), _new_workspace, dev, handle)


def _new_workspace(n, old, dev, handle):
    ws = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev))
    # the smaller one may still be in use on its stream, and what the current stream has queued may
    # still use the memory that it gave for a call on another one
    if torch.cuda.is_initialized() and (old is not None or handle.value != _stream_handle(None).value):
        torch.cuda.synchronize(dev)
    _check("pkv_workspace_init", load_library().pkv_workspace_init(_cuda("workspace", ws), n, handle))
    return ws


__all__ = [
    "paged_attention_decode", "paged_decode_step", "paged_attention_decode_mq", "paged_attention_decode_head_scales",
    "reshape_and_cache", "reshape_and_cache_head_scales", "workspace_size", "new_workspace", "workspace_init",
    "read_device_error", "default_partitions", "status_string", "load_library", "PkvError",
    "paged_attention_decode_shared_prefix", "paged_decode_step_shared_prefix", "DevicePrefixPlan",
    "shared_prefix_workspace_size", "new_shared_prefix_workspace", "validate_tables",
    "qk_norm_rope", "qk_norm_rope_and_cache", "reshape_and_cache_block_scales", "paged_attention_decode_block_scales",
    "update_key_bounds", "select_blocks", "select_workspace_size", "new_select_workspace",
    "paged_attention_decode_sparse",
    "F32", "BF16", "FP8_E4M3", "FP8_E5M2", "INT8",
]
