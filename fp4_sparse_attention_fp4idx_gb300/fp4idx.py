"""ctypes binding of libfp4idx.so (argument marshalling only).

Importing this module loads the CUDA library and raises ImportError if it is
missing: there is no CPU path.  Build it with
``python -m fp4_sparse_attention_fp4idx_gb300.build``.

Two layers:
  * ``lib()`` -- the raw C ABI (names and argument order of include/fp4idx.h,
    include/fp4idx_attention.h and include/fp4idx_step.h, plain integers for
    pointers).
  * torch wrappers with the same names (minus the ``fp4idx_`` prefix) that
    check dtypes/devices, allocate outputs with torch, pass ``data_ptr()``s
    and the current CUDA stream (or ``stream=``, on which outputs that are not
    given are then allocated), and raise ``Fp4idxError`` on a non-OK
    status.  Every step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
import threading
from typing import Any, NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp4idx.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp4idx.h")
ATTENTION_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp4idx_attention.h")
STEP_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp4idx_step.h")

ROPE_NEOX = 0
ROPE_INTERLEAVED = 1
HEAD_DIM = 128
PAGE_BYTES = 4352
ERRFLAG_POSITION = 0x1
ERRFLAG_SLOT = 0x2
ERRFLAG_TIMEOUT = 0x4
ERRFLAG_PAGE = 0x8
ERRFLAG_FULL = 0x10

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARG, ERR_CUDA, ERR_SCRATCH = range(7)
STATIC_STAGING_BYTES = 64 << 20  # FP4IDX_STATIC_STAGING_BYTES

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python -m fp4_sparse_attention_fp4idx_gb300.build` (needs nvcc); "
        "there is no CPU fallback")

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_INT = ctypes.c_int

_SIGS = {
    "fp4idx_k_norm_rope_pack_store": (
        _INT, [_P, _I64, _P, _F, _P, _P, _P, _I64, _INT, _P, _P, _I64, _I64, _P, _P]),
    "fp4idx_q_rope_pack_weights": (
        _INT, [_P, _I64, _I64, _P, _I64, _F, _P, _P, _P, _I64, _INT, _P, _P, _P, _I64,
               _I64, _P, _P]),
    "fp4idx_indexer_prepass": (
        _INT, [_P, _I64, _P, _F, _P, _P, _I64,
               _P, _I64, _I64, _P, _I64, _F, _P, _P, _P, _I64,
               _P, _P, _P, _I64, _INT, _I64, _P, _P]),
    "fp4idx_k_norm_rope_pack_store_ex": (
        _INT, [_P, _I64, _P, _F, _P, _P, _P, _I64, _INT, _P, _P, _I64, _I64, _P, _P, _P]),
    "fp4idx_q_rope_pack_weights_ex": (
        _INT, [_P, _I64, _I64, _P, _I64, _F, _P, _P, _P, _I64, _INT, _P, _P, _P, _I64,
               _I64, _P, _P, _P]),
    "fp4idx_indexer_prepass_ex": (
        _INT, [_P, _I64, _P, _F, _P, _P, _I64,
               _P, _I64, _I64, _P, _I64, _F, _P, _P, _P, _I64,
               _P, _P, _P, _I64, _INT, _I64, _P, _P, _P]),
    "fp4idx_rope_fake_quant": (
        _INT, [_P, _I64, _I64, _P, _P, _P, _I64, _INT, _INT, _P, _I64, _P, _P]),
    "fp4idx_paged_mqa_logits": (
        _INT, [_P, _P, _P, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "fp4idx_mqa_logits_prefill": (
        _INT, [_P, _P, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I64, _P, _P]),
    "fp4idx_indexer_prepass_host": (
        _INT, [_P, _P, _P, _F, _P, _I64, _P, _P, _I64, _F, _P, _P, _P, _P, _P, _P, _I64,
               _INT, _I64, _I64, _P, _P, _P]),
    "fp4idx_host_staging_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "fp4idx_indexer_prepass_host_static": (
        _INT, [_P, _P, _P, _F, _P, _I64, _P, _P, _I64, _F, _P, _P, _P, _P, _P, _P, _I64,
               _INT, _I64, _I64, _P, _P]),
    "fp4idx_kv_store_fp8": (
        _INT, [_P, _P, _I64, _I64, _I64, _I64, _INT, _P, _P, _I64, _P, _P]),
    "fp4idx_kv_load_fp8": (_INT, [_P, _P, _P, _P, _INT, _I64, _P, _P]),
    "fp4idx_attention_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64]),
    "fp4idx_paged_attention_fp8": (
        _INT, [_P, _I64, _I64, _INT, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _F, _P, _P,
               _I64, _I64, _I64, _P, ctypes.c_size_t, _P, _P]),
    "fp4idx_sparse_attention_fp8": (
        _INT, [_P, _I64, _I64, _INT, _P, _P, _I64, _I64, _P, _P, _I64, _I64, _F, _P, _P, _I64,
               _I64, _I64, _P, ctypes.c_size_t, _P, _P]),
    "fp4idx_topk_tokens": (_INT, [_P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P]),
    "fp4idx_batch_extend": (
        _INT, [_P, _P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P]),
    "fp4idx_pages_release": (
        _INT, [_P, _P, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _P]),
    "fp4idx_rope_qk": (
        _INT, [_P, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _INT,
               _I64, _P, _I64, _P, _INT, _INT, _P, _P, _I64, _I64, _INT, _I64, _P, _P]),
    "fp4idx_prompt_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64]),
    "fp4idx_prompt_attention": (
        _INT, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _INT, _P, _P, _I64, _I64, _I64,
               _I64, _F, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, ctypes.c_size_t, _P, _P]),
    "fp4idx_default_weight_scale": (_F, [_I64]),
    "fp4idx_test_withhold_next": (_INT, [_INT, _I64]),
    "fp4idx_status_string": (ctypes.c_char_p, [_INT]),
    "fp4idx_version": (ctypes.c_char_p, []),
}

_lib = ctypes.CDLL(LIB_PATH)
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def lib() -> ctypes.CDLL:
    return _lib


OUTPUT_FP4 = 0
OUTPUT_FP8 = 1
FP8_PAGE_BYTES = 8448


class Options(ctypes.Structure):
    """fp4idx_options of include/fp4idx.h."""
    _fields_ = [("compress_ratio", ctypes.c_int32), ("hadamard", ctypes.c_int32),
                ("output_mode", ctypes.c_int32)]


def _options(compress_ratio: int, hadamard: bool, fp8: bool = False):
    """None for the defaults (the plain entry points are called), else a
    pointer to an Options block for the _ex entry points."""
    if compress_ratio == 1 and not hadamard and not fp8:
        return None
    return ctypes.pointer(Options(int(compress_ratio), 1 if hadamard else 0,
                                  OUTPUT_FP8 if fp8 else OUTPUT_FP4))


def declared_symbols(header: str = HEADER_PATH) -> list:
    """Names of the functions include/fp4idx.h declares."""
    with open(header) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(fp4idx_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return _lib.fp4idx_status_string(int(status)).decode()


def version() -> str:
    return _lib.fp4idx_version().decode()


class Fp4idxError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != OK:
        raise Fp4idxError(status, where)


def rope_style_code(style) -> int:
    if style in (ROPE_NEOX, "neox"):
        return ROPE_NEOX
    if style in (ROPE_INTERLEAVED, "interleaved", "gptj"):
        return ROPE_INTERLEAVED
    raise ValueError(f"unknown rope style {style!r}")


TEST_PREPASS = 0
TEST_SCORER = 1
TEST_ATTENTION = 2
TEST_PROMPT = 3


def test_withhold_next(kernel: int, index: int) -> None:
    """Testing hook: the next launch of `kernel` (TEST_PREPASS: the streaming
    pre-pass; TEST_SCORER: the scorers; TEST_ATTENTION: attention over the
    8-bit cache; TEST_PROMPT: attention of prompts) leaves out the copies of
    work item `index` of its first CTA, so its bounded waits run out (TIMEOUT
    flag)."""
    _check(_lib.fp4idx_test_withhold_next(int(kernel), int(index)), "fp4idx_test_withhold_next")


def default_weight_scale(num_heads: int) -> float:
    """The library's head-weight scale, fp32(H^-1/2 * 128^-1/2)."""
    return float(_lib.fp4idx_default_weight_scale(int(num_heads)))


# ------------------------------------------------------------ torch wrappers
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_ptr(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(int(s.cuda_stream))


_HERE = contextlib.nullcontext()


def _on(stream):
    """Where a call makes its own allocations: on the stream that it runs on.
    A fill is then in order with its kernel, and memory given back is used again
    behind it."""
    return _HERE if stream is None else _torch().cuda.stream(stream)


def _need(t, dtype, name, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def k_norm_rope_pack_store(k, gamma, positions, cos_cache, sin_cache, slot_mapping,
                           kv_cache, *, eps: float = 1e-6, rope_style="neox",
                           compress_ratio: int = 1, hadamard: bool = False,
                           err_flags=None, stream=None) -> None:
    """Keys -> paged FP4 index cache, in place.  k bf16 [T,128] (row stride a
    multiple of 8), gamma bf16 [128], positions/slot_mapping int64 [T],
    cos/sin fp32 [max_pos,32], kv_cache uint8 [num_blocks, 4352].
    compress_ratio / hadamard select the stated variants (fp4idx_options)."""
    torch = _torch()
    _need(k, torch.bfloat16, "k", 2)
    _need(gamma, torch.bfloat16, "gamma", 1)
    _need(positions, torch.int64, "positions", 1)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(cos_cache, torch.float32, "cos_cache", 2)
    _need(sin_cache, torch.float32, "sin_cache", 2)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    T = k.shape[0]
    if k.shape[1] != HEAD_DIM or k.stride(1) != 1:
        raise ValueError("k must be [T,128] with unit element stride")
    if gamma.shape[0] != HEAD_DIM or not gamma.is_contiguous():
        raise ValueError("gamma must be contiguous [128]")
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("positions and slot_mapping must have T entries")
    if not (positions.is_contiguous() and slot_mapping.is_contiguous()):
        raise ValueError("positions and slot_mapping must be contiguous")
    if cos_cache.shape != sin_cache.shape or cos_cache.shape[1] != 32:
        raise ValueError("cos/sin caches must both be [max_pos, 32]")
    if not (cos_cache.is_contiguous() and sin_cache.is_contiguous()):
        raise ValueError("cos/sin caches must be contiguous")
    if kv_cache.shape[1] != PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 4352]")
    args = (_ptr(k), k.stride(0), _ptr(gamma), float(eps), _ptr(positions), _ptr(cos_cache),
            _ptr(sin_cache), cos_cache.shape[0], rope_style_code(rope_style),
            _ptr(slot_mapping), _ptr(kv_cache), kv_cache.shape[0], T)
    opts = _options(compress_ratio, hadamard)
    if opts is None:
        st = _lib.fp4idx_k_norm_rope_pack_store(*args, _ptr(err_flags), _stream_ptr(stream))
    else:
        st = _lib.fp4idx_k_norm_rope_pack_store_ex(*args, ctypes.cast(opts, _P),
                                                   _ptr(err_flags), _stream_ptr(stream))
    _check(st, "fp4idx_k_norm_rope_pack_store")


def _q_outputs(q_fp4, q_scale, weights, T, H, device, stream):
    torch = _torch()
    with _on(stream):
        if q_fp4 is None:
            q_fp4 = torch.empty((T, H, 64), dtype=torch.uint8, device=device)
        if q_scale is None:
            q_scale = torch.empty((T, H, 4), dtype=torch.uint8, device=device)
        if weights is None:
            weights = torch.empty((T, H), dtype=torch.float32, device=device)
    for t, shape, dt, name in ((q_fp4, (T, H, 64), torch.uint8, "q_fp4"),
                               (q_scale, (T, H, 4), torch.uint8, "q_scale"),
                               (weights, (T, H), torch.float32, "weights")):
        _need(t, dt, name)
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {shape}")
    return q_fp4, q_scale, weights


def _check_q(q, w, positions, cos_cache, sin_cache):
    torch = _torch()
    _need(q, torch.bfloat16, "q", 3)
    _need(w, torch.bfloat16, "w", 2)
    _need(positions, torch.int64, "positions", 1)
    _need(cos_cache, torch.float32, "cos_cache", 2)
    _need(sin_cache, torch.float32, "sin_cache", 2)
    T, H, D = q.shape
    if D != HEAD_DIM or q.stride(2) != 1:
        raise ValueError("q must be [T,H,128] with unit element stride")
    if tuple(w.shape) != (T, H) or w.stride(1) != 1:
        raise ValueError("w must be [T,H] with unit head stride")
    if positions.shape[0] != T or not positions.is_contiguous():
        raise ValueError("positions must be contiguous [T]")
    if cos_cache.shape != sin_cache.shape or cos_cache.shape[1] != 32:
        raise ValueError("cos/sin caches must both be [max_pos, 32]")
    if not (cos_cache.is_contiguous() and sin_cache.is_contiguous()):
        raise ValueError("cos/sin caches must be contiguous")
    return T, H


def q_rope_pack_weights(q, w, positions, cos_cache, sin_cache, *, rope_style="neox",
                        weight_scale=None, q_fp4=None, q_scale=None, weights=None,
                        hadamard: bool = False, err_flags=None, stream=None):
    """Queries -> (q_fp4 uint8 [T,H,64], q_scale uint8 [T,H,4], weights fp32
    [T,H]).  q bf16 [T,H,128] (strides multiples of 8), w bf16 [T,H]."""
    T, H = _check_q(q, w, positions, cos_cache, sin_cache)
    q_fp4, q_scale, weights = _q_outputs(q_fp4, q_scale, weights, T, H, q.device, stream)
    ws = default_weight_scale(H) if weight_scale is None else float(weight_scale)
    args = (_ptr(q), q.stride(0), q.stride(1), _ptr(w), w.stride(0), ws, _ptr(positions),
            _ptr(cos_cache), _ptr(sin_cache), cos_cache.shape[0], rope_style_code(rope_style),
            _ptr(q_fp4), _ptr(q_scale), _ptr(weights), T, H)
    opts = _options(1, hadamard)
    if opts is None:
        st = _lib.fp4idx_q_rope_pack_weights(*args, _ptr(err_flags), _stream_ptr(stream))
    else:
        st = _lib.fp4idx_q_rope_pack_weights_ex(*args, ctypes.cast(opts, _P), _ptr(err_flags),
                                                _stream_ptr(stream))
    _check(st, "fp4idx_q_rope_pack_weights")
    return q_fp4, q_scale, weights


def indexer_prepass(k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache, sin_cache, *,
                    eps: float = 1e-6, rope_style="neox", weight_scale=None, q_fp4=None,
                    q_scale=None, weights=None, compress_ratio: int = 1,
                    hadamard: bool = False, err_flags=None, stream=None):
    """Both halves in one launch; returns (q_fp4, q_scale, weights) and updates
    kv_cache in place.  Same argument rules as the two separate calls."""
    torch = _torch()
    T, H = _check_q(q, w, positions, cos_cache, sin_cache)
    _need(k, torch.bfloat16, "k", 2)
    _need(gamma, torch.bfloat16, "gamma", 1)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    if k.shape[0] != T or k.shape[1] != HEAD_DIM or k.stride(1) != 1:
        raise ValueError("k must be [T,128] with unit element stride")
    if gamma.shape[0] != HEAD_DIM or not gamma.is_contiguous():
        raise ValueError("gamma must be contiguous [128]")
    if slot_mapping.shape[0] != T or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous [T]")
    if kv_cache.shape[1] != PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 4352]")
    q_fp4, q_scale, weights = _q_outputs(q_fp4, q_scale, weights, T, H, q.device, stream)
    ws = default_weight_scale(H) if weight_scale is None else float(weight_scale)
    args = (_ptr(k), k.stride(0), _ptr(gamma), float(eps), _ptr(slot_mapping), _ptr(kv_cache),
            kv_cache.shape[0], _ptr(q), q.stride(0), q.stride(1), _ptr(w), w.stride(0), ws,
            _ptr(q_fp4), _ptr(q_scale), _ptr(weights), H, _ptr(positions), _ptr(cos_cache),
            _ptr(sin_cache), cos_cache.shape[0], rope_style_code(rope_style), T)
    opts = _options(compress_ratio, hadamard)
    if opts is None:
        st = _lib.fp4idx_indexer_prepass(*args, _ptr(err_flags), _stream_ptr(stream))
    else:
        st = _lib.fp4idx_indexer_prepass_ex(*args, ctypes.cast(opts, _P), _ptr(err_flags),
                                            _stream_ptr(stream))
    _check(st, "fp4idx_indexer_prepass")
    return q_fp4, q_scale, weights


# ------------------------------------------------------- host-buffer pipeline
_STAGING = {}  # (device index, chunk_tokens, H) -> device staging tensor
_STAGING_LOCK = threading.Lock()


def _need_host(t, dtype, name, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")
    return t


def _staging(device, chunk: int, H: int):
    """The device staging buffer of fp4idx_indexer_prepass_host, allocated
    once per (device, chunk, H) and kept (its contents are scratch)."""
    torch = _torch()
    nbytes = int(_lib.fp4idx_host_staging_bytes(chunk, H))
    if nbytes == 0:
        raise ValueError(f"chunk_tokens {chunk} x num_heads {H} is too large")
    key = (device.index, chunk, H)
    with _STAGING_LOCK:
        buf = _STAGING.get(key)
        if buf is None:
            buf = _STAGING[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf


def _host_args(k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache, sin_cache,
               weight_scale, q_fp4, q_scale, weights, chunk_tokens):
    """Checks of the host-buffer calls; returns (T, H, chunk, q_fp4, q_scale,
    weights, weight_scale) with the host outputs allocated pinned when not
    given."""
    torch = _torch()
    _need_host(k, torch.bfloat16, "k", 2)
    _need_host(q, torch.bfloat16, "q", 3)
    _need_host(w, torch.bfloat16, "w", 2)
    _need_host(positions, torch.int64, "positions", 1)
    _need_host(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    _need(gamma, torch.bfloat16, "gamma", 1)
    T, H, D = q.shape
    if D != HEAD_DIM or tuple(k.shape) != (T, HEAD_DIM) or tuple(w.shape) != (T, H):
        raise ValueError("k must be [T,128], q [T,H,128], w [T,H]")
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("positions and slot_mapping must have T entries")
    if gamma.shape[0] != HEAD_DIM or not gamma.is_contiguous():
        raise ValueError("gamma must be contiguous [128]")
    if kv_cache.shape[1] != PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 4352]")
    for t, name in ((cos_cache, "cos_cache"), (sin_cache, "sin_cache")):
        _need(t, torch.float32, name, 2)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if chunk_tokens < 1:
        raise ValueError("chunk_tokens must be >= 1")
    outs = []
    for t, shape, dt, name in ((q_fp4, (T, H, 64), torch.uint8, "q_fp4"),
                               (q_scale, (T, H, 4), torch.uint8, "q_scale"),
                               (weights, (T, H), torch.float32, "weights")):
        if t is None:
            t = torch.empty(shape, dtype=dt).pin_memory()
        _need_host(t, dt, name, len(shape))
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}")
        outs.append(t)
    ws = default_weight_scale(H) if weight_scale is None else float(weight_scale)
    return T, H, min(int(chunk_tokens), max(T, 1)), outs[0], outs[1], outs[2], ws


def indexer_prepass_host(k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache,
                         sin_cache, *, eps: float = 1e-6, rope_style="neox", weight_scale=None,
                         q_fp4=None, q_scale=None, weights=None, chunk_tokens: int = 4096,
                         err_flags=None, stream=None):
    """indexer_prepass for inputs and outputs in host memory, through the
    C-ABI call fp4idx_indexer_prepass_host: k [T,128], q [T,H,128], w [T,H]
    (bf16), positions and slot_mapping [T] (int64) are contiguous host
    tensors, pinned for the copies to overlap; gamma, the cos/sin caches and
    kv_cache are device tensors.  The library pipelines the tokens in chunks
    of chunk_tokens (upload of chunk c+1, fused launch of chunk c, download of
    chunk c-1) on its own streams.  Returns host tensors (q_fp4, q_scale,
    weights), allocated pinned when not given; they are complete once the
    caller's stream (which waits for the pipeline) has reached this point."""
    torch = _torch()
    T, H, chunk, q_fp4, q_scale, weights, ws = _host_args(
        k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache, sin_cache, weight_scale,
        q_fp4, q_scale, weights, chunk_tokens)
    if T == 0:
        return q_fp4, q_scale, weights
    dev = kv_cache.device
    staging = _staging(dev, chunk, H)
    caller = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        st = _lib.fp4idx_indexer_prepass_host(
            _ptr(k), _ptr(slot_mapping), _ptr(gamma), float(eps), _ptr(kv_cache),
            kv_cache.shape[0], _ptr(q), _ptr(w), H, ws, _ptr(q_fp4), _ptr(q_scale),
            _ptr(weights), _ptr(positions), _ptr(cos_cache), _ptr(sin_cache),
            cos_cache.shape[0], rope_style_code(rope_style), T, chunk, _ptr(staging),
            _ptr(err_flags), _stream_ptr(caller))
    _check(st, "fp4idx_indexer_prepass_host")
    return q_fp4, q_scale, weights


def indexer_prepass_host_static(k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache,
                                sin_cache, *, eps: float = 1e-6, rope_style="neox",
                                weight_scale=None, q_fp4=None, q_scale=None, weights=None,
                                chunk_tokens=None, err_flags=None, stream=None):
    """indexer_prepass_host with the staging in the library's static device
    buffer (fp4idx_indexer_prepass_host_static): nothing is allocated on the
    device; chunk_tokens must keep the staging within STATIC_STAGING_BYTES
    (ERR_SCRATCH otherwise).  By default it is the largest power-of-two
    share of 1024 tokens whose staging fits."""
    torch = _torch()
    if chunk_tokens is None:
        H = q.shape[1] if hasattr(q, "shape") and q.dim() == 3 else 1
        chunk_tokens = 1024
        while chunk_tokens > 1 and (
                _lib.fp4idx_host_staging_bytes(chunk_tokens, H) == 0 or
                _lib.fp4idx_host_staging_bytes(chunk_tokens, H) > STATIC_STAGING_BYTES):
            chunk_tokens //= 2
    T, H, chunk, q_fp4, q_scale, weights, ws = _host_args(
        k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache, sin_cache, weight_scale,
        q_fp4, q_scale, weights, chunk_tokens)
    if T == 0:
        return q_fp4, q_scale, weights
    dev = kv_cache.device
    caller = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        st = _lib.fp4idx_indexer_prepass_host_static(
            _ptr(k), _ptr(slot_mapping), _ptr(gamma), float(eps), _ptr(kv_cache),
            kv_cache.shape[0], _ptr(q), _ptr(w), H, ws, _ptr(q_fp4), _ptr(q_scale),
            _ptr(weights), _ptr(positions), _ptr(cos_cache), _ptr(sin_cache),
            cos_cache.shape[0], rope_style_code(rope_style), T, chunk, _ptr(err_flags),
            _stream_ptr(caller))
    _check(st, "fp4idx_indexer_prepass_host_static")
    return q_fp4, q_scale, weights


def paged_mqa_logits(q_fp4, q_scale, weights, kv_cache, block_table, context_lens,
                     max_context: int, *, next_n: int = 1, logits=None, err_flags=None,
                     stream=None):
    """FP4 paged MQA logits -> fp32 [batch*next_n, max_context].  q_fp4 uint8
    [batch*next_n, H, 64], q_scale uint8 [batch*next_n, H, 4], weights fp32
    [batch*next_n, H] (the pre-pass's query outputs), kv_cache uint8
    [num_blocks, 4352], block_table int32 [batch, >= ceil(max_context/64)]
    (unit column stride), context_lens int32 [batch]."""
    torch = _torch()
    _need(q_fp4, torch.uint8, "q_fp4", 3)
    _need(q_scale, torch.uint8, "q_scale", 3)
    _need(weights, torch.float32, "weights", 2)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    _need(block_table, torch.int32, "block_table", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    T, H, nb = q_fp4.shape
    if nb != 64 or not q_fp4.is_contiguous():
        raise ValueError("q_fp4 must be contiguous [batch*next_n, H, 64]")
    if tuple(q_scale.shape) != (T, H, 4) or not q_scale.is_contiguous():
        raise ValueError("q_scale must be contiguous [batch*next_n, H, 4]")
    if tuple(weights.shape) != (T, H) or not weights.is_contiguous():
        raise ValueError("weights must be contiguous [batch*next_n, H]")
    if next_n < 1 or T % next_n:
        raise ValueError("the query rows must be batch*next_n")
    batch = T // next_n
    if block_table.shape[0] != batch or block_table.stride(1) != 1:
        raise ValueError("block_table must be [batch, pages] with unit column stride")
    if context_lens.shape[0] != batch or not context_lens.is_contiguous():
        raise ValueError("context_lens must be contiguous [batch]")
    if kv_cache.shape[1] != PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 4352]")
    if logits is None:
        with _on(stream):
            logits = torch.empty((T, max_context), dtype=torch.float32, device=q_fp4.device)
    _need(logits, torch.float32, "logits", 2)
    if logits.shape[0] != T or logits.shape[1] < max_context or logits.stride(1) != 1:
        raise ValueError("logits must be [batch*next_n, >= max_context] with unit column stride")
    # A size-1 leading dimension may carry any stride (numpy gives 0 to a
    # new axis); the row width is the stride the C ABI's checks expect then.
    bt_stride = block_table.stride(0) if batch > 1 else block_table.shape[1]
    out_stride = logits.stride(0) if T > 1 else logits.shape[1]
    st = _lib.fp4idx_paged_mqa_logits(
        _ptr(q_fp4), _ptr(q_scale), _ptr(weights), _ptr(kv_cache), kv_cache.shape[0],
        _ptr(block_table), bt_stride, _ptr(context_lens), _ptr(logits), out_stride, batch,
        next_n, H, int(max_context), _ptr(err_flags), _stream_ptr(stream))
    _check(st, "fp4idx_paged_mqa_logits")
    return logits


def mqa_logits_prefill(q_fp4, q_scale, weights, kv_cache, ks, ke, num_keys: int, *,
                       logits=None, err_flags=None, stream=None):
    """FP4 prefill MQA logits -> fp32 [T, num_keys]: query token t (q_fp4
    uint8 [T, H, 64], q_scale uint8 [T, H, 4], weights fp32 [T, H]) against
    the consecutive keys 0 .. num_keys-1 of kv_cache uint8 [num_blocks, 4352]
    (key s at page s/64, offset s%64), over the keys in [ks[t], ke[t])
    (int32 [T]); -inf elsewhere."""
    torch = _torch()
    _need(q_fp4, torch.uint8, "q_fp4", 3)
    _need(q_scale, torch.uint8, "q_scale", 3)
    _need(weights, torch.float32, "weights", 2)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    _need(ks, torch.int32, "ks", 1)
    _need(ke, torch.int32, "ke", 1)
    T, H, nb = q_fp4.shape
    if nb != 64 or not q_fp4.is_contiguous():
        raise ValueError("q_fp4 must be contiguous [T, H, 64]")
    if tuple(q_scale.shape) != (T, H, 4) or not q_scale.is_contiguous():
        raise ValueError("q_scale must be contiguous [T, H, 4]")
    if tuple(weights.shape) != (T, H) or not weights.is_contiguous():
        raise ValueError("weights must be contiguous [T, H]")
    if tuple(ks.shape) != (T,) or tuple(ke.shape) != (T,) or not (
            ks.is_contiguous() and ke.is_contiguous()):
        raise ValueError("ks and ke must be contiguous [T]")
    if kv_cache.shape[1] != PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 4352]")
    if logits is None:
        with _on(stream):
            logits = torch.empty((T, num_keys), dtype=torch.float32, device=q_fp4.device)
    _need(logits, torch.float32, "logits", 2)
    if logits.shape[0] != T or logits.shape[1] < num_keys or logits.stride(1) != 1:
        raise ValueError("logits must be [T, >= num_keys] with unit column stride")
    out_stride = logits.stride(0) if T > 1 else logits.shape[1]
    st = _lib.fp4idx_mqa_logits_prefill(
        _ptr(q_fp4), _ptr(q_scale), _ptr(weights), _ptr(kv_cache), kv_cache.shape[0],
        int(num_keys), _ptr(ks), _ptr(ke), _ptr(logits), out_stride, T, H, _ptr(err_flags),
        _stream_ptr(stream))
    _check(st, "fp4idx_mqa_logits_prefill")
    return logits


# ------------------------------------------------------------ FP8 output mode
def k_norm_rope_fp8_store(k, gamma, positions, cos_cache, sin_cache, slot_mapping, kv_cache, *,
                          eps: float = 1e-6, rope_style="neox", compress_ratio: int = 1,
                          hadamard: bool = False, err_flags=None, stream=None) -> None:
    """Keys -> FP8 paged index cache (uint8 [num_blocks, 8448]), in place:
    fp4idx_k_norm_rope_pack_store_ex with output_mode FP8."""
    torch = _torch()
    _need(k, torch.bfloat16, "k", 2)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    if kv_cache.shape[1] != FP8_PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 8448]")
    T = k.shape[0]
    if k.shape[1] != HEAD_DIM or k.stride(1) != 1:
        raise ValueError("k must be [T,128] with unit element stride")
    opts = _options(compress_ratio, hadamard, fp8=True)
    st = _lib.fp4idx_k_norm_rope_pack_store_ex(
        _ptr(k), k.stride(0), _ptr(gamma), float(eps), _ptr(positions), _ptr(cos_cache),
        _ptr(sin_cache), cos_cache.shape[0], rope_style_code(rope_style), _ptr(slot_mapping),
        _ptr(kv_cache), kv_cache.shape[0], T, ctypes.cast(opts, _P), _ptr(err_flags),
        _stream_ptr(stream))
    _check(st, "fp4idx_k_norm_rope_pack_store_ex (FP8)")


def _fp8_q_outputs(q_out, weights, T, H, device, stream):
    torch = _torch()
    with _on(stream):
        if q_out is None:
            q_out = torch.empty((T, H, HEAD_DIM), dtype=torch.uint8, device=device)
        if weights is None:
            weights = torch.empty((T, H), dtype=torch.float32, device=device)
    for t, shape, dt, name in ((q_out, (T, H, HEAD_DIM), torch.uint8, "q_out"),
                               (weights, (T, H), torch.float32, "weights")):
        _need(t, dt, name)
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {shape}")
    return q_out, weights


def q_rope_fp8_weights(q, w, positions, cos_cache, sin_cache, *, rope_style="neox",
                       weight_scale=None, q_out=None, weights=None, hadamard: bool = False,
                       err_flags=None, stream=None):
    """Queries -> (E4M3 codes uint8 [T,H,128], weights fp32 [T,H] with each
    row's power-of-two scale folded in)."""
    T, H = _check_q(q, w, positions, cos_cache, sin_cache)
    q_out, weights = _fp8_q_outputs(q_out, weights, T, H, q.device, stream)
    ws = default_weight_scale(H) if weight_scale is None else float(weight_scale)
    opts = _options(1, hadamard, fp8=True)
    st = _lib.fp4idx_q_rope_pack_weights_ex(
        _ptr(q), q.stride(0), q.stride(1), _ptr(w), w.stride(0), ws, _ptr(positions),
        _ptr(cos_cache), _ptr(sin_cache), cos_cache.shape[0], rope_style_code(rope_style),
        _ptr(q_out), None, _ptr(weights), T, H, ctypes.cast(opts, _P), _ptr(err_flags),
        _stream_ptr(stream))
    _check(st, "fp4idx_q_rope_pack_weights_ex (FP8)")
    return q_out, weights


def indexer_prepass_fp8(k, gamma, slot_mapping, kv_cache, q, w, positions, cos_cache,
                        sin_cache, *, eps: float = 1e-6, rope_style="neox", weight_scale=None,
                        q_out=None, weights=None, compress_ratio: int = 1,
                        hadamard: bool = False, err_flags=None, stream=None):
    """Both halves in the FP8 mode, one launch; returns (q_out, weights) and
    updates kv_cache ([num_blocks, 8448]) in place."""
    torch = _torch()
    T, H = _check_q(q, w, positions, cos_cache, sin_cache)
    _need(k, torch.bfloat16, "k", 2)
    _need(kv_cache, torch.uint8, "kv_cache", 2)
    if kv_cache.shape[1] != FP8_PAGE_BYTES or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous [num_blocks, 8448]")
    if k.shape[0] != T or k.shape[1] != HEAD_DIM or k.stride(1) != 1:
        raise ValueError("k must be [T,128] with unit element stride")
    q_out, weights = _fp8_q_outputs(q_out, weights, T, H, q.device, stream)
    ws = default_weight_scale(H) if weight_scale is None else float(weight_scale)
    opts = _options(compress_ratio, hadamard, fp8=True)
    st = _lib.fp4idx_indexer_prepass_ex(
        _ptr(k), k.stride(0), _ptr(gamma), float(eps), _ptr(slot_mapping), _ptr(kv_cache),
        kv_cache.shape[0], _ptr(q), q.stride(0), q.stride(1), _ptr(w), w.stride(0), ws,
        _ptr(q_out), None, _ptr(weights), H, _ptr(positions), _ptr(cos_cache), _ptr(sin_cache),
        cos_cache.shape[0], rope_style_code(rope_style), T, ctypes.cast(opts, _P),
        _ptr(err_flags), _stream_ptr(stream))
    _check(st, "fp4idx_indexer_prepass_ex (FP8)")
    return q_out, weights


# ------------------------------------------------------ torch-shaped fake quant
FAKE_QUANT_UE8M0_32 = 0
FAKE_QUANT_E4M3_16 = 1


def rope_fake_quant(x, positions, cos_cache, sin_cache, *, rope_style="neox",
                    scale_mode: int = FAKE_QUANT_UE8M0_32, out=None, err_flags=None,
                    stream=None):
    """RoPE + FP4 fake quantisation -> bf16 of x's shape.  x bf16 [T,128]
    (keys, one position per row) or [T,H,128] (queries, one position per
    token), unit element stride, row stride a multiple of 8."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    if x.dim() == 2:
        T, D = x.shape
        rows, per, stride = T, 1, x.stride(0)
    elif x.dim() == 3:
        T, H, D = x.shape
        if x.stride(0) != H * x.stride(1):
            raise ValueError("x [T,H,128] must have token stride H * head stride")
        rows, per, stride = T * H, H, x.stride(1)
    else:
        raise ValueError("x must be [T,128] or [T,H,128]")
    if D != HEAD_DIM or x.stride(-1) != 1:
        raise ValueError("rows must be 128 elements with unit stride")
    _need(positions, torch.int64, "positions", 1)
    if positions.shape[0] != T or not positions.is_contiguous():
        raise ValueError("positions must be contiguous [T]")
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out")
    if tuple(out.shape) != tuple(x.shape) or not out.is_contiguous():
        raise ValueError("out must be contiguous with x's shape")
    st = _lib.fp4idx_rope_fake_quant(
        _ptr(x), stride, per, _ptr(positions), _ptr(cos_cache), _ptr(sin_cache),
        cos_cache.shape[0], rope_style_code(rope_style), int(scale_mode), _ptr(out), rows,
        _ptr(err_flags), _stream_ptr(stream))
    _check(st, "fp4idx_rope_fake_quant")
    return out


# ------------------------------------- 8-bit key/value cache and its attention
# These calls are made once per layer and step, often on a few microseconds of
# GPU work, so their checks are written to be cheap: one test per tensor, and
# plain integers for pointers.
DTYPE_BF16 = 0
DTYPE_FP16 = 1
KV_BLOCK = 64


class KvCache(ctypes.Structure):
    """fp4idx_kv_cache of include/fp4idx_attention.h."""
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scale", _P), ("v_scale", _P),
                ("num_blocks", _I64), ("code_block_stride", _I64), ("scale_block_stride", _I64),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _fits(t, dtype, ndim, dev, name):
    """t is a CUDA tensor of that type and rank on device `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.dim() == ndim and dev >= 0:
            return
    except AttributeError:
        pass
    _need(t, dtype, name, ndim)  # says what is wrong
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _dense(t, shape, name):
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)}")


def _type16(t, name):
    """The fp4idx_dtype code of a tensor of bf16 or fp16."""
    torch = _torch()
    dt = getattr(t, "dtype", None)
    if dt is torch.bfloat16:
        return DTYPE_BF16
    if dt is torch.float16:
        return DTYPE_FP16
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {dt}")


def _block_strides(t, n, inner, name):
    """(block stride, ...) of a [num_blocks, kv_heads, ...] tensor whose heads
    are `inner` elements apart (a size of 1 leaves its stride open)."""
    st = t.stride()
    if n > 1 and st[1] != inner:
        raise ValueError(f"{name}'s heads must be dense")
    return st[0] if t.shape[0] > 1 else n * inner


def _kv_cache(k_cache, v_cache, k_scale, v_scale):
    """(KvCache block, device index) of the four tensors."""
    torch = _torch()
    codes = (torch.uint8, torch.float8_e4m3fn)
    try:  # the usual layouts in one test; what fails it is looked at piece by piece
        shape, st, ss, dev = k_cache.shape, k_cache.stride(), k_scale.stride(), \
            k_cache.get_device()
        B, H, n, D = shape
        if (k_cache.dtype in codes and v_cache.dtype in codes and
                k_scale.dtype is torch.float32 and v_scale.dtype is torch.float32 and
                n == KV_BLOCK and (D == 128 or D == 64) and B > 1 and H > 1 and dev >= 0 and
                v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == dev and
                v_cache.shape == shape and k_scale.shape == v_scale.shape == (B, H) and
                v_cache.stride() == st and v_scale.stride() == ss and ss[1] == 1 and
                st[1:] == (KV_BLOCK * D, D, 1)):
            return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                           v_scale.data_ptr(), B, st[0], ss[0], H, D), dev
    except (AttributeError, ValueError):
        pass
    return _kv_cache_slow(k_cache, v_cache, k_scale, v_scale)


def _kv_cache_slow(k_cache, v_cache, k_scale, v_scale):
    torch = _torch()
    f8, f32 = torch.float8_e4m3fn, torch.float32
    dev = k_cache.get_device() if isinstance(k_cache, torch.Tensor) else -1
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _fits(t, f8 if getattr(t, "dtype", None) == f8 else torch.uint8, 4, dev, name)
    _fits(k_scale, f32, 2, dev, "k_scale")
    _fits(v_scale, f32, 2, dev, "v_scale")
    shape = k_cache.shape
    B, H, n, D = shape
    if n != KV_BLOCK or D not in (64, 128):
        raise ValueError("k_cache must be [num_blocks, kv_heads, 64, 64 or 128]")
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if k_scale.shape != (B, H) or v_scale.shape != (B, H):
        raise ValueError("k_scale and v_scale must be [num_blocks, kv_heads]")
    if k_cache.stride()[2:] != (D, 1) or v_cache.stride()[2:] != (D, 1):
        raise ValueError("the rows of a block must be dense")
    cs = _block_strides(k_cache, H, KV_BLOCK * D, "k_cache")
    ss = _block_strides(k_scale, H, 1, "k_scale")
    if _block_strides(v_cache, H, KV_BLOCK * D, "v_cache") != cs or \
            _block_strides(v_scale, H, 1, "v_scale") != ss:
        raise ValueError("keys and values must have the same block strides")
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                   B, cs, ss, H, D), dev


def _rows16(t, H, D, dev, name):
    """(token stride, head stride) of a 16-bit [T, H, D] tensor."""
    _fits(t, t.dtype, 3, dev, name)
    T, h, d = t.shape
    st = t.stride()
    if h != H or d != D or st[2] != 1:
        raise ValueError(f"{name} must be [T, {H}, {D}] with unit element stride")
    return (st[0] if T > 1 else H * D), (st[1] if H > 1 else D)


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with `dev` the current device; raises on a status."""
    torch = _torch()
    s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != OK:
        raise Fp4idxError(st, fn.__name__)


def _flags(err_flags, dev):
    if err_flags is None:
        return None
    torch = _torch()
    _fits(err_flags, torch.int32, err_flags.dim() if isinstance(err_flags, torch.Tensor) else 1,
          dev, "err_flags")
    if err_flags.numel() < 1:
        raise ValueError("err_flags must hold an element")
    return err_flags.data_ptr()


def kv_store_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, *, err_flags=None,
                 stream=None) -> None:
    """Quantises keys and values into the paged 8-bit cache, in place.  k, v
    bf16 or fp16 [T, kv_heads, D] (strides multiples of 8), slot_mapping int64
    [T] (block*64 + offset; negative: skip), k_cache/v_cache uint8 or
    float8_e4m3fn [num_blocks, kv_heads, 64, D], k_scale/v_scale fp32
    [num_blocks, kv_heads].  A block's scale covers its 64 tokens; storing
    behind kept rows grows it where needed and requantises them."""
    torch = _torch()
    c, dev = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    dt = _type16(k, "k")
    if _type16(v, "v") != dt:
        raise TypeError("k and v must have the same dtype")
    H, D = c.kv_heads, c.head_dim
    kt, kh = _rows16(k, H, D, dev, "k")
    vt, vh = _rows16(v, H, D, dev, "v")
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v must have the same tokens")
    _fits(slot_mapping, torch.int64, 1, dev, "slot_mapping")
    _dense(slot_mapping, (T,), "slot_mapping")
    _call(_lib.fp4idx_kv_store_fp8, dev, stream, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, dt,
          slot_mapping.data_ptr(), ctypes.byref(c), T, _flags(err_flags, dev))


def kv_load_fp8(k_cache, v_cache, k_scale, v_scale, slot_mapping, *, dtype=None, k_out=None,
                v_out=None, err_flags=None, stream=None):
    """Reads cached tokens back -> (k, v) of `dtype` (bf16 by default, or
    fp16), [T, kv_heads, D].  A negative slot leaves its output row as it was
    (zeros where the outputs are allocated here, on `stream`)."""
    torch = _torch()
    c, dev = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    _fits(slot_mapping, torch.int64, 1, dev, "slot_mapping")
    T = slot_mapping.shape[0]
    _dense(slot_mapping, (T,), "slot_mapping")
    shape = (T, c.kv_heads, c.head_dim)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else \
            v_out.dtype if v_out is not None else torch.bfloat16
    with _on(stream):
        if k_out is None:
            k_out = torch.zeros(shape, device=k_cache.device, dtype=dtype)
        if v_out is None:
            v_out = torch.zeros(shape, device=k_cache.device, dtype=dtype)
    dt = _type16(k_out, "k_out")
    _fits(k_out, dtype, 3, dev, "k_out")
    _fits(v_out, dtype, 3, dev, "v_out")
    _dense(k_out, shape, "k_out")
    _dense(v_out, shape, "v_out")
    _call(_lib.fp4idx_kv_load_fp8, dev, stream, ctypes.byref(c), slot_mapping.data_ptr(),
          k_out.data_ptr(), v_out.data_ptr(), dt, T, _flags(err_flags, dev))
    return k_out, v_out


def attention_workspace_bytes(batch: int, max_q: int, num_heads: int, kv_heads: int,
                              head_dim: int) -> int:
    """Workspace of paged_attention_fp8 (for sparse_attention_fp8: batch = T,
    max_q = 1); 0 for arguments out of range."""
    return _lib.fp4idx_attention_workspace_bytes(batch, max_q, num_heads, kv_heads, head_dim)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(batch, max_q, num_heads, kv_heads, head_dim):
    """At least 16, so that an empty call has an address to pass."""
    return attention_workspace_bytes(batch, max_q, num_heads, kv_heads, head_dim) or 16


def _attention_buffers(q, c, dev, block_table, out, lse, workspace, batch, max_q, stream):
    """Checks of q and block_table; (dtype code, strides of q, out, lse,
    workspace), allocated on `stream` where not given."""
    torch = _torch()
    dt = _type16(q, "q")
    H_kv, D = c.kv_heads, c.head_dim
    shape = q.shape
    if len(shape) != 3 or shape[1] % H_kv:
        raise ValueError("q must be [T, H, D], H a multiple of the cache's heads")
    T, H, _ = shape
    qt, qh = _rows16(q, H, D, dev, "q")
    _fits(block_table, torch.int32, 2, dev, "block_table")
    if block_table.stride(1) != 1 and block_table.shape[1] > 1:
        raise ValueError("block_table must have unit column stride")
    device = q.device
    with _on(stream):
        if out is None:
            out = torch.empty_like(q) if q.is_contiguous() else \
                torch.empty((T, H, D), dtype=q.dtype, device=device)
        else:
            _fits(out, q.dtype, 3, dev, "out")
            _dense(out, (T, H, D), "out")
        if lse is None:
            lse = torch.empty((T, H), dtype=torch.float32, device=device)
        else:
            _fits(lse, torch.float32, 2, dev, "lse")
            _dense(lse, (T, H), "lse")
        if workspace is None:
            workspace = torch.empty(_workspace_bytes(batch, max_q, H, H_kv, D), dtype=torch.uint8,
                                    device=device)
        else:
            _fits(workspace, torch.uint8, 1, dev, "workspace")
            _dense(workspace, workspace.shape, "workspace")
    return dt, qt, qh, out, lse, workspace


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens,
                        max_context: int, *, q_starts=None, max_q=None, window: int = 0,
                        sinks: int = 0, softmax_scale=None, out=None, lse=None, workspace=None,
                        err_flags=None, stream=None):
    """Causal attention over the 8-bit cache -> (out [T, H, D] of q's dtype,
    lse fp32 [T, H]).  q bf16 or fp16 [T, H, D]; block_table int32 [batch,
    pages], context_lens int32 [batch] counts the query tokens too (their keys
    and values are in the cache); they are at most max_context, and that at most
    pages * 64.  The query tokens are T / batch per sequence,
    or, with q_starts int32 [batch+1] and max_q (the longest), ragged.
    window > 0: a query sees the last `window` keys and the first `sinks`.
    softmax_scale defaults to D^-1/2."""
    torch = _torch()
    c, dev = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    _type16(q, "q")
    _fits(context_lens, torch.int32, 1, dev, "context_lens")
    T, batch = len(q), len(context_lens)
    _dense(context_lens, (batch,), "context_lens")
    starts = None
    if q_starts is not None:
        _fits(q_starts, torch.int32, 1, dev, "q_starts")
        _dense(q_starts, (batch + 1,), "q_starts")
        if max_q is None:
            raise ValueError("q_starts needs max_q, the longest sequence of query tokens")
        starts = q_starts.data_ptr()
    else:
        if (batch == 0 and T > 0) or (batch > 0 and T % batch):
            raise ValueError("without q_starts, T must be a multiple of the batch")
        max_q = T // batch if batch else 0
    dt, qt, qh, out, lse, workspace = _attention_buffers(q, c, dev, block_table, out, lse,
                                                         workspace, batch, max_q, stream)
    if block_table.shape[0] != batch:
        raise ValueError("block_table must be [batch, pages]")
    if T > 0 and block_table.shape[1] * KV_BLOCK < max_context:
        # a view's rows go on behind its columns, so its stride says nothing
        raise Fp4idxError(ERR_SHAPE, "fp4idx_paged_attention_fp8: max_context beyond block_table")
    _call(_lib.fp4idx_paged_attention_fp8, dev, stream, q.data_ptr(), qt, qh, dt, ctypes.byref(c),
          block_table.data_ptr(), block_table.stride(0) if batch > 1 else block_table.shape[1],
          context_lens.data_ptr(), starts, max_q, max_context, window, sinks,
          c.head_dim ** -0.5 if softmax_scale is None else softmax_scale, out.data_ptr(),
          lse.data_ptr(), batch, T, q.shape[1], workspace.data_ptr(), workspace.numel(),
          _flags(err_flags, dev))
    return out, lse


def sparse_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, indices, *,
                         seq_ids=None, softmax_scale=None, out=None, lse=None, workspace=None,
                         err_flags=None, stream=None):
    """Attention over selected tokens of the 8-bit cache -> (out [T, H, D],
    lse fp32 [T, H]).  indices int32 [T, n]: positions in the token's sequence
    (negative: left out), as topk_tokens returns them; block_table int32
    [batch, pages]; seq_ids int32 [T] names each token's sequence (by default
    T / batch consecutive tokens each)."""
    torch = _torch()
    c, dev = _kv_cache(k_cache, v_cache, k_scale, v_scale)
    _type16(q, "q")
    T = q.shape[0]
    _fits(indices, torch.int32, 2, dev, "indices")
    n = indices.shape[1]
    if indices.shape[0] != T or (n > 1 and indices.stride(1) != 1):
        raise ValueError("indices must be [T, n] with unit column stride")
    dt, qt, qh, out, lse, workspace = _attention_buffers(q, c, dev, block_table, out, lse,
                                                         workspace, T, 1, stream)
    batch, pages = block_table.shape
    seqs = None
    if seq_ids is not None:
        _fits(seq_ids, torch.int32, 1, dev, "seq_ids")
        _dense(seq_ids, (T,), "seq_ids")
        seqs = seq_ids.data_ptr()
    elif (batch == 0 and T > 0) or (batch > 0 and T % batch):
        raise ValueError("without seq_ids, T must be a multiple of the batch")
    _call(_lib.fp4idx_sparse_attention_fp8, dev, stream, q.data_ptr(), qt, qh, dt, ctypes.byref(c),
          block_table.data_ptr(), block_table.stride(0) if batch > 1 else pages, pages, seqs,
          indices.data_ptr(), indices.stride(0) if T > 1 else n, n,
          c.head_dim ** -0.5 if softmax_scale is None else softmax_scale, out.data_ptr(),
          lse.data_ptr(), batch, T, q.shape[1], workspace.data_ptr(), workspace.numel(),
          _flags(err_flags, dev))
    return out, lse


def topk_tokens(logits, k: int, *, row_lens=None, indices=None, counts=None, stream=None):
    """The k largest logits of each row -> (indices int32 [R, k] ascending,
    padded with -1, counts int32 [R]).  logits fp32 [R, N] (unit column
    stride), row_lens int32 [R]: entries behind a row's length are not read;
    -inf and NaN are never selected, equal logits from the lowest index up."""
    torch = _torch()
    dev = logits.get_device() if isinstance(logits, torch.Tensor) else -1
    _fits(logits, torch.float32, 2, dev, "logits")
    R, N = logits.shape
    if N > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    lens = None
    if row_lens is not None:
        _fits(row_lens, torch.int32, 1, dev, "row_lens")
        _dense(row_lens, (R,), "row_lens")
        lens = row_lens.data_ptr()
    with _on(stream):
        if indices is None:
            indices = torch.empty((R, k), dtype=torch.int32, device=logits.device)
        else:
            _fits(indices, torch.int32, 2, dev, "indices")
            if indices.shape != (R, k) or (k > 1 and indices.stride(1) != 1):
                raise ValueError("indices must be [R, k] with unit column stride")
        if counts is None:
            counts = torch.empty((R,), dtype=torch.int32, device=logits.device)
        else:
            _fits(counts, torch.int32, 1, dev, "counts")
            _dense(counts, (R,), "counts")
    _call(_lib.fp4idx_topk_tokens, dev, stream, logits.data_ptr(),
          logits.stride(0) if R > 1 else N, lens, indices.data_ptr(),
          indices.stride(0) if R > 1 else k, counts.data_ptr(), R, N, k)
    return indices, counts


# ------------------------------------ pages and maps, rotary positions, prompts
class BatchMaps(NamedTuple):
    """What batch_extend writes for the step's other calls."""
    q_starts: Any      # int32 [batch+1]
    context_lens: Any  # int32 [batch]
    slot_mapping: Any  # int64 [num_tokens]
    positions: Any     # int64 [num_tokens]
    seq_ids: Any       # int32 [num_tokens]
    row_lens: Any      # int32 [num_tokens]


def _pool(first, second, names, block_table, free_pages, free_count):
    """Checks of two vectors of lengths and the page pool; (device index, batch,
    the pool's C arguments)."""
    i32 = _torch().int32
    try:  # the usual call in one test; what fails it is looked at piece by piece
        batch, pages = block_table.shape
        st, dev = block_table.stride(), block_table.get_device()
        n, = free_pages.shape
        if (block_table.dtype is first.dtype is second.dtype is free_pages.dtype is
                free_count.dtype is i32 and dev >= 0 and
                first.get_device() == second.get_device() == free_pages.get_device() ==
                free_count.get_device() == dev and
                first.shape == second.shape == (batch,) and free_count.shape == (1,) and
                first.is_contiguous() and second.is_contiguous() and
                free_pages.is_contiguous() and batch > 1 and pages > 1 and st[1] == 1 and
                st[0] >= pages):
            return dev, batch, (block_table.data_ptr(), st[0], pages, free_pages.data_ptr(),
                                free_count.data_ptr(), n)
    except (AttributeError, ValueError):
        pass
    return _pool_slow(first, second, names, block_table, free_pages, free_count)


def _pool_slow(first, second, names, block_table, free_pages, free_count):
    torch = _torch()
    i32 = torch.int32
    dev = block_table.get_device() if isinstance(block_table, torch.Tensor) else -1
    _fits(block_table, i32, 2, dev, "block_table")
    _fits(first, i32, 1, dev, names[0])
    _fits(second, i32, 1, dev, names[1])
    _fits(free_pages, i32, 1, dev, "free_pages")
    _fits(free_count, i32, 1, dev, "free_count")
    batch, pages = block_table.shape
    _dense(first, (batch,), names[0])
    _dense(second, (batch,), names[1])
    _dense(free_pages, free_pages.shape, "free_pages")
    if free_count.shape[0] != 1:
        raise ValueError("free_count must be [1]")
    st = block_table.stride()
    if pages > 1 and st[1] != 1:
        raise ValueError("block_table must have unit column stride")
    if batch > 1 and st[0] < pages:
        raise ValueError("block_table's rows must not overlap")
    return dev, batch, (block_table.data_ptr(), st[0] if batch > 1 else pages, pages,
                        free_pages.data_ptr(), free_count.data_ptr(), free_pages.shape[0])


_NO_MAPS = (None,) * 6


def batch_extend(cached_lens, new_lens, block_table, free_pages, free_count, num_tokens: int, *,
                 q_starts=None, context_lens=None, slot_mapping=None, positions=None, seq_ids=None,
                 row_lens=None, err_flags=None, stream=None) -> BatchMaps:
    """The next tokens of a batch: new_lens int32 [batch] tokens behind
    cached_lens int32 [batch] ones.  Takes the pages that they need off the
    stack free_pages int32 [n] / free_count int32 [1] into block_table int32
    [batch, pages], in place, and returns the maps of the step's num_tokens tokens
    (slot -1, position 0, sequence 0, row length 0 behind the last one).  A
    sequence that cannot be served keeps its pages and length, its tokens get slot
    -1, and ERRFLAG_FULL is raised.  context_lens is the next step's cached_lens."""
    torch = _torch()
    dev, batch, pool = _pool(cached_lens, new_lens, ("cached_lens", "new_lens"), block_table,
                             free_pages, free_count)
    if num_tokens < 0:
        raise ValueError("num_tokens must not be negative")
    given = (q_starts, context_lens, slot_mapping, positions, seq_ids, row_lens)
    with _on(stream):
        i32, i64, empty = torch.int32, torch.int64, torch.empty
        if given == _NO_MAPS:  # (six allocations cost less than views of two)
            at = block_table.device
            maps = (empty(batch + 1, dtype=i32, device=at), empty(batch, dtype=i32, device=at),
                    empty(num_tokens, dtype=i64, device=at),
                    empty(num_tokens, dtype=i64, device=at),
                    empty(num_tokens, dtype=i32, device=at),
                    empty(num_tokens, dtype=i32, device=at))
        else:
            maps = []
            for t, n, dt, name in zip(given, (batch + 1, batch, *[num_tokens] * 4),
                                      (i32, i32, i64, i64, i32, i32), BatchMaps._fields):
                if t is None:
                    t = empty(n, dtype=dt, device=block_table.device)
                else:
                    _fits(t, dt, 1, dev, name)
                    _dense(t, (n,), name)
                maps.append(t)
    _call(_lib.fp4idx_batch_extend, dev, stream, cached_lens.data_ptr(), new_lens.data_ptr(),
          *pool, *[t.data_ptr() for t in maps], batch, num_tokens, _flags(err_flags, dev))
    return BatchMaps(*maps)


def pages_release(held_lens, kept_lens, block_table, free_pages, free_count, *, err_flags=None,
                  stream=None) -> None:
    """Gives pages back to the stack, in place: of the pages that held_lens int32
    [batch] tokens fill, those behind the first kept_lens int32 [batch] tokens (0:
    the sequence has ended).  Their entries of block_table become -1.  Undoes a
    batch_extend that went before it."""
    dev, batch, pool = _pool(held_lens, kept_lens, ("held_lens", "kept_lens"), block_table,
                             free_pages, free_count)
    _call(_lib.fp4idx_pages_release, dev, stream, held_lens.data_ptr(), kept_lens.data_ptr(),
          *pool, batch, _flags(err_flags, dev))


AXES_SECTIONS = 0
AXES_INTERLEAVED = 1


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int32 * len(sections))(*sections)


def _heads16(t, like, dev, name):
    """(T, heads, D, token stride, head stride) of a 16-bit tensor on device `dev`
    and of the type of `like`, one test for the usual case."""
    try:
        T, H, D = t.shape
        ts, hs, one = t.stride()
        if one == 1 and t.dtype is like.dtype and t.get_device() == dev and dev >= 0:
            return T, H, D, ts if T > 1 else H * D, hs if H > 1 else D
    except (AttributeError, ValueError):
        pass
    _type16(t, name)
    _fits(t, like.dtype, 3, dev, name)
    raise ValueError(f"{name} must be [T, heads, D] with unit element stride")


def _tables(cos, sin, dev):
    """(max_pos, pairs) of two dense fp32 tables."""
    f32 = _torch().float32
    try:
        shape = cos.shape
        if (cos.dtype is sin.dtype is f32 and cos.get_device() == sin.get_device() == dev and
                sin.shape == shape and cos.is_contiguous() and sin.is_contiguous()):
            max_pos, half = shape
            return max_pos, half
    except (AttributeError, ValueError):
        pass
    _fits(cos, f32, 2, dev, "cos")
    _fits(sin, f32, 2, dev, "sin")
    _dense(cos, cos.shape, "cos")
    _dense(sin, cos.shape, "sin")
    return cos.shape


def rope_qk(q, k, positions, cos, sin, *, rope_style="neox", sections=None,
            interleaved_axes: bool = False, q_out=None, k_out=None, err_flags=None, stream=None):
    """Rotary positions of queries and keys -> (q_out, k_out).  q, k bf16 or fp16
    [T, heads, D] (strides multiples of 8; k may be None), cos, sin fp32 [max_pos,
    R/2]: the first R elements of a row are turned, the others copied.  positions
    int64 [T], or [axes, T] with `sections`, the pairs that each axis turns: ranges
    of pairs, or dealt in turn (interleaved_axes).  q_out may be q and k_out k (in
    place); outputs that are not given are allocated dense."""
    torch = _torch()
    dt = _type16(q, "q")
    dev = q.get_device()
    T, Hq, D, *qs = _heads16(q, q, dev, "q")
    Hk, ks, kp, kop, ko = 0, (0, 0), None, None, (0, 0)
    if k is not None:
        kT, Hk, kD, *ks = _heads16(k, q, dev, "k")
        if kT != T or kD != D:
            raise ValueError("k must be [T, heads, D] with q's tokens and D")
    elif k_out is not None:
        raise ValueError("k_out without k")
    max_pos, half = _tables(cos, sin, dev)
    several = getattr(positions, "ndim", 1) == 2
    _fits(positions, torch.int64, 2 if several else 1, dev, "positions")
    st = positions.stride()
    if positions.shape[-1] != T or (T > 1 and st[-1] != 1):
        raise ValueError("positions must be [T] or [axes, T] with unit token stride")
    axes = len(positions) if several else 1
    if sections is None:
        if axes > 1:
            raise ValueError("positions of several axes need sections")
        sections = (half,)
    elif len(sections) != axes:
        raise ValueError("sections must have an entry for each axis of positions")
    else:
        sections = tuple(map(int, sections))
    if stream is None:
        q_out, k_out, qo, ko = _rope_outputs(torch, q, k, q_out, k_out, T, Hq, Hk, D, dev)
    else:
        with torch.cuda.stream(stream):
            q_out, k_out, qo, ko = _rope_outputs(torch, q, k, q_out, k_out, T, Hq, Hk, D, dev)
    if Hk:
        kp, kop = k.data_ptr(), k_out.data_ptr()
    _call(_lib.fp4idx_rope_qk, dev, stream, q.data_ptr(), *qs, q_out.data_ptr(), *qo, Hq, kp, *ks,
          kop, *ko, Hk, dt, D, positions.data_ptr(), st[0] if axes > 1 else T,
          _sections(sections), axes, AXES_INTERLEAVED if interleaved_axes else AXES_SECTIONS,
          cos.data_ptr(), sin.data_ptr(), max_pos, 2 * half, rope_style_code(rope_style), T,
          None if err_flags is None else _flags(err_flags, dev))
    return q_out, k_out


def _rope_outputs(torch, q, k, q_out, k_out, T, Hq, Hk, D, dev):
    """Outputs, made where not given, and their strides."""
    qo, ko = (Hq * D, D), (Hk * D, D)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    else:
        *shape, a, b = _heads16(q_out, q, dev, "q_out")
        if shape != [T, Hq, D]:
            raise ValueError("q_out must have q's shape")
        qo = a, b
    if k is not None:
        if k_out is None:
            k_out = torch.empty((T, Hk, D), dtype=q.dtype, device=q.device)
        else:
            *shape, a, b = _heads16(k_out, q, dev, "k_out")
            if shape != [T, Hk, D]:
                raise ValueError("k_out must have k's shape")
            ko = a, b
    return q_out, k_out, qo, ko


def prompt_workspace_bytes(batch: int, max_q: int, num_heads: int, kv_heads: int,
                           head_dim: int) -> int:
    """Workspace of prompt_attention; 0 for arguments out of range."""
    return _lib.fp4idx_prompt_workspace_bytes(batch, max_q, num_heads, kv_heads, head_dim)


@functools.lru_cache(maxsize=256)
def _prompt_workspace(batch, max_q, num_heads, kv_heads, head_dim):
    return prompt_workspace_bytes(batch, max_q, num_heads, kv_heads, head_dim) or 16


def prompt_attention(q, k, v, q_starts, max_q: int, *, k_starts=None, max_k=None, window: int = 0,
                     sinks: int = 0, softmax_scale=None, out=None, lse=None, workspace=None,
                     err_flags=None, stream=None):
    """Causal attention of packed sequences over their own keys and values ->
    (out [Tq, H, D] of q's dtype, lse fp32 [Tq, H]).  q bf16 or fp16 [Tq, H, D], k,
    v [Tk, kv_heads, D] (strides multiples of 8); q_starts int32 [batch+1], max_q
    the longest.  Whole prompts, or, with k_starts int32 [batch+1] and max_k,
    queries that end a longer run of keys: chunks and single tokens.  window > 0: a
    query sees the last `window` keys and the first `sinks`.  softmax_scale defaults
    to D^-1/2.  Rows of out and lse in no sequence are left as they were."""
    torch = _torch()
    dt = _type16(q, "q")
    dev = q.get_device()
    Tq, H, D, *qs = _heads16(q, q, dev, "q")
    Tk, Hk, kD, *ks = _heads16(k, q, dev, "k")
    vT, vH, vD, *vs = _heads16(v, q, dev, "v")
    if vT != Tk or vH != Hk or vD != D or kD != D:
        raise ValueError("k and v must have the same tokens and heads, and q's D")
    if Hk == 0 or H % Hk:
        raise ValueError("q's heads must be a multiple of k's")
    _fits(q_starts, torch.int32, 1, dev, "q_starts")
    batch = len(q_starts) - 1
    if batch < 0 or not q_starts.is_contiguous():
        raise ValueError("q_starts must be contiguous [batch+1]")
    kst = None
    if k_starts is not None:
        _fits(k_starts, torch.int32, 1, dev, "k_starts")
        _dense(k_starts, (batch + 1,), "k_starts")
        if max_k is None:
            raise ValueError("k_starts needs max_k, the longest run of keys")
        kst = k_starts.data_ptr()
    elif Tk != Tq:
        raise ValueError("without k_starts, q and k must have the same tokens")
    if max_k is None:
        max_k = max_q
    if out is not None:
        _fits(out, q.dtype, 3, dev, "out")
        _dense(out, (Tq, H, D), "out")
    if lse is not None:
        _fits(lse, torch.float32, 2, dev, "lse")
        _dense(lse, (Tq, H), "lse")
    if workspace is not None:
        _fits(workspace, torch.uint8, 1, dev, "workspace")
        _dense(workspace, workspace.shape, "workspace")
    if out is None or lse is None or workspace is None:
        with _on(stream):
            at = q.device
            if out is None:
                out = torch.empty((Tq, H, D), dtype=q.dtype, device=at)
            if lse is None:
                lse = torch.empty((Tq, H), dtype=torch.float32, device=at)
            if workspace is None:
                workspace = torch.empty(_prompt_workspace(batch, max_q, H, Hk, D),
                                        dtype=torch.uint8, device=at)
    _call(_lib.fp4idx_prompt_attention, dev, stream, q.data_ptr(), *qs, k.data_ptr(), *ks,
          v.data_ptr(), *vs, dt, q_starts.data_ptr(), kst, max_q, max_k, window, sinks,
          D ** -0.5 if softmax_scale is None else softmax_scale, out.data_ptr(), lse.data_ptr(),
          batch, Tq, Tk, H, Hk, D, workspace.data_ptr(), workspace.numel(),
          None if err_flags is None else _flags(err_flags, dev))
    return out, lse
