"""Python binding of the gemm_f16 / attn_f16 C ABI (include/*.h).

Argument marshalling only: every step of an operation runs in the CUDA
kernels of ``csrc/``.  The functions keep the C names; raw pointers are
Python ints.  ``matmul``, ``attention`` and the calls of a serving step over
a paged cache (``paged_maps``, ``rotary``, ``rotary_to_cache``,
``paged_attention``) are conveniences that take torch tensors (PyTorch is
used only for device memory and streams); the latter four marshal in C++
(``csrc/torch_calls.cpp``), because a step makes them for every layer.

The library is built in-tree by ``async_barrier_pipelined_gb300.build.build()``
(``__graft_entry__.build()`` calls it).  If it is missing, loading fails
loudly; there is no fallback implementation.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import importlib.util
import math
import os
import threading

from .build import CALLS_NAME, CALLS_PATH, LIB_PATH

__all__ = [
    "GemmError", "load", "gemm_f16_plan", "gemm_f16_run", "gemm_f16_run_host",
    "gemm_f16_destroy", "gemm_f16_status", "gemm_f16_set_option",
    "gemm_f16_strerror", "gemm_f16_last_cuda_error", "gemm_f16_validate",
    "gemm_f16_tile_order", "gemm_f16_tile_shape", "Plan", "matmul",
    "OK", "ERR_INVALID_ARG", "ERR_MISALIGNED", "ERR_UNSUPPORTED_DEVICE",
    "ERR_OOM", "ERR_CUDA", "ERR_TIMEOUT", "ERR_SCRATCH_TOO_SMALL", "gemm_f16_run_noalloc", "gemm_f16_noalloc_status",
    "OPT_TIMEOUT_NS", "OPT_TILE_ORDER", "OPT_FAULT_UNIT", "OPT_KERNEL", "OPT_TILE_WIDTH", "OPT_SM_LIMIT", "OPT_ATTN_KERNEL", "OPT_ATTN_SPLIT", "OPT_A_REPACK", "OPT_MULTICAST", "OPT_KERNEL_TIMING", "INFO_NUM_SMS", "INFO_MAX_PAIRS", "INFO_MAX_QUADS",
    "gemm_f16_get_option", "gemm_f16_pair_tiles", "EXPORTED_SYMBOLS",
    "gemm_f16_run_ex", "gemm_f16_validate_ex", "attn_f16_fwd", "attn_f16_validate",
    "attn_f16_key_ranges", "gemm_f16_run_info", "gemm_f16_run_choice", "attn_f16_fwd_host", "attention_host",
    "attention", "ATTN_HEAD_DIM", "gemm_f16_kernel_time",
    "LAYOUT_NN", "LAYOUT_TN", "LAYOUT_NT", "LAYOUT_TT",
    "ERR_BAD_INDEX", "attn_f16_paged_maps", "attn_f16_paged_maps_validate",
    "attn_f16_paged_maps_overlap", "attn_f16_rope",
    "attn_f16_rope_validate", "attn_f16_rope_turns", "attn_f16_paged_fwd",
    "attn_f16_paged_validate", "ROPE_HALF", "ROPE_INTERLEAVED", "PagedMaps", "paged_maps",
    "rope_frequencies", "rope_turns", "rotary", "rotary_to_cache", "paged_attention",
    "EXPORTED_SYMBOLS_F8", "GemmF8Operand", "F8_E4M3", "F8_E5M2", "F8_DENSE", "F8_BY_ROWS",
    "F8_BY_INNER", "gemm_f8_quantize", "gemm_f8_quantize_validate", "gemm_f8_run",
    "gemm_f8_workspace", "gemm_f8_run_choice", "gemm_f8_validate", "experts_maps", "experts_maps_validate",
    "experts_max_rows", "experts_gather", "experts_gather_validate", "experts_combine",
    "experts_combine_validate", "experts_combine_gradient",
    "experts_combine_gradient_validate", "Blocks", "quantize", "matmul_f8", "linear_f8",
    "ExpertMaps", "expert_maps", "expert_gather", "expert_combine",
]

OK = 0
ERR_INVALID_ARG = -1
ERR_MISALIGNED = -2
ERR_UNSUPPORTED_DEVICE = -3
ERR_OOM = -4
ERR_CUDA = -5
ERR_TIMEOUT = -6
ERR_SCRATCH_TOO_SMALL = -7
ERR_BAD_INDEX = -8

OPT_TIMEOUT_NS = 1
OPT_TILE_ORDER = 2
OPT_FAULT_UNIT = 3
OPT_KERNEL = 4
OPT_TILE_WIDTH = 5
OPT_SM_LIMIT = 6
OPT_ATTN_KERNEL = 7
OPT_ATTN_SPLIT = 8
OPT_A_REPACK = 9
OPT_KERNEL_TIMING = 10
OPT_MULTICAST = 11
INFO_NUM_SMS = 100
INFO_MAX_PAIRS = 101
INFO_MAX_QUADS = 102

ATTN_HEAD_DIM = 256

LAYOUT_NN = 0
LAYOUT_TN = 1   # A stored K x M
LAYOUT_NT = 2   # B stored N x K
LAYOUT_TT = 3

ROPE_HALF = 0
ROPE_INTERLEAVED = 1

F8_E4M3, F8_E5M2 = 0, 1
F8_F16, F8_BF16, F8_F32 = 0, 1, 2
F8_ROWS, F8_COLUMNS, F8_TILES, F8_BOTH = 0, 1, 2, 3
F8_DENSE, F8_BY_ROWS, F8_BY_INNER = 0, 1, 2

_c_int, _c_i64, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p

_i64p = ctypes.POINTER(_c_i64)
_MAPS_ARGS = [_c_int, _vp, _vp, _vp, _c_i64, _c_int, _vp, _c_int, _vp, _c_int, _c_int,
              _vp, _vp, _vp, _vp, _vp]
_ROPE_TAIL = [_vp, _vp, _vp, _i64p, _vp, _i64p, _vp, _i64p, _vp, _i64p, _vp, _vp, _i64p, _vp,
              _i64p, _c_int, _c_int]
_PAGED_ARGS = [_c_int] * 6 + [_vp, _i64p, _vp, _i64p, _vp, _i64p, _c_int, _c_int, _vp, _c_i64,
                              _c_int, _vp, _vp, _vp, _i64p, ctypes.c_float, _c_int, _c_int]

#: name -> (restype, argtypes) for every entry point of include/*.h
_SIGNATURES = {
    "gemm_f16_plan": (_c_int, [ctypes.POINTER(_vp), _c_int]),
    "gemm_f16_run": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64,
                              _vp, _c_i64, _c_int, _vp]),
    "gemm_f16_run_ex": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _c_i64, _vp,
                                 _c_i64, _vp, _c_i64, _c_int, _vp]),
    "gemm_f16_run_host": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64,
                                   _vp, _c_i64, _c_int, _vp]),
    "gemm_f16_destroy": (_c_int, [_vp]),
    "gemm_f16_status": (_c_int, [_vp]),
    "gemm_f16_set_option": (_c_int, [_vp, _c_int, _c_i64]),
    "gemm_f16_get_option": (_c_int, [_vp, _c_int, ctypes.POINTER(_c_i64)]),
    "gemm_f16_strerror": (ctypes.c_char_p, [_c_int]),
    "gemm_f16_last_cuda_error": (ctypes.c_char_p, []),
    "gemm_f16_validate": (_c_int, [_c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64,
                                   _vp, _c_i64, _c_int]),
    "gemm_f16_validate_ex": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _c_i64, _vp,
                                      _c_i64, _vp, _c_i64, _c_int]),
    "gemm_f16_tile_order": (_c_i64, [_c_int, _c_int, _c_int,
                                     ctypes.POINTER(ctypes.c_uint32), _c_i64]),
    "gemm_f16_tile_shape": (_c_int, [ctypes.POINTER(_c_int)] * 4),
    "gemm_f16_pair_tiles": (_c_i64, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                     ctypes.POINTER(ctypes.c_uint32), _c_i64,
                                     ctypes.POINTER(_c_int)]),
    "gemm_f16_run_noalloc": (_c_int, [_c_int, _c_int, _c_int, _vp, _c_i64, _vp, _c_i64,
                                      _vp, _c_i64, _c_int, _vp, _vp]),
    "gemm_f16_noalloc_status": (_c_int, []),
    "attn_f16_fwd": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                              _vp, ctypes.POINTER(_c_i64), _vp, ctypes.POINTER(_c_i64),
                              _vp, ctypes.POINTER(_c_i64), _vp, ctypes.POINTER(_c_i64),
                              ctypes.c_float, _vp]),
    "attn_f16_validate": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int,
                                   _vp, ctypes.POINTER(_c_i64), _vp, ctypes.POINTER(_c_i64),
                                   _vp, ctypes.POINTER(_c_i64), _vp, ctypes.POINTER(_c_i64),
                                   ctypes.c_float]),
    "attn_f16_key_ranges": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int,
                                     ctypes.POINTER(_c_int)]),
    "gemm_f16_run_info": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int,
                                   ctypes.POINTER(_c_int)]),
    "gemm_f16_run_choice": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int,
                                     _c_int, _c_int, ctypes.POINTER(_c_int)]),
    "attn_f16_fwd_host": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                   _vp, ctypes.c_float, _vp]),
    "attn_f16_paged_maps": (_c_int, [_vp, *_MAPS_ARGS, _vp]),
    "attn_f16_paged_maps_validate": (_c_int, _MAPS_ARGS),
    "attn_f16_paged_maps_overlap": (_c_int, _MAPS_ARGS[:9] + _MAPS_ARGS[10:]),
    "attn_f16_rope": (_c_int, [_vp] + [_c_int] * 7 + [ctypes.c_float, *_ROPE_TAIL, _vp]),
    "attn_f16_rope_validate": (_c_int, [_c_int] * 6 + [ctypes.c_float, *_ROPE_TAIL]),
    "attn_f16_rope_turns": (_c_int, [ctypes.POINTER(ctypes.c_double), _c_int,
                                     ctypes.POINTER(ctypes.c_uint64)]),
    "attn_f16_paged_fwd": (_c_int, [_vp, *_PAGED_ARGS, _vp]),
    "attn_f16_paged_validate": (_c_int, _PAGED_ARGS),
    "gemm_f16_kernel_time": (_c_int, [_vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_c_i64)]),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)


class GemmF8Operand(ctypes.Structure):
    """gemm_f8_operand of gemm_f8.h."""
    _fields_ = [("data", _vp), ("ld", _c_i64), ("batch", _c_i64), ("scales", _vp),
                ("s_outer", _c_i64), ("s_inner", _c_i64), ("s_batch", _c_i64),
                ("format", _c_int), ("transposed", _c_int), ("tiles", _c_int)]


_operandp = ctypes.POINTER(GemmF8Operand)
_F8_QUANTIZE = [_c_int] * 6 + [_vp, _c_i64, _c_i64, _vp, _c_int, _c_int, _vp, _c_i64, _c_i64, _vp,
                               _vp, _vp]
_F8_RUN = [_c_int] * 5 + [_vp, _operandp, _operandp, _vp, _c_i64, _c_i64, _c_int, _c_int]
_EXPERTS_MAPS = [_c_int, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]
_EXPERTS_GATHER = [_c_int] * 3 + [_vp, _c_i64, _c_int, _c_int, _vp, _vp, _c_i64]
_EXPERTS_COMBINE = [_c_int] * 4 + [_vp, _c_i64, _c_int, _vp, _vp, _c_int, _vp, _c_i64]
_EXPERTS_GRADIENT = [_c_int] * 4 + [_vp, _c_i64, _vp, _c_i64, _c_int, _vp, _vp, _vp, _c_int, _vp,
                                    _c_i64, _vp]

#: the same for include/gemm_f8.h
_SIGNATURES_F8 = {
    "gemm_f8_quantize": (_c_int, [_vp, *_F8_QUANTIZE, _vp]),
    "gemm_f8_quantize_validate": (_c_int, _F8_QUANTIZE),
    "gemm_f8_run": (_c_int, [_vp, *_F8_RUN, _vp, ctypes.c_size_t, _vp]),
    "gemm_f8_workspace": (ctypes.c_size_t, [_vp] + [_c_int] * 6),
    "gemm_f8_run_choice": (_c_int, [_c_int] * 9 + [ctypes.POINTER(_c_int)]),
    "gemm_f8_validate": (_c_int, _F8_RUN),
    "experts_maps": (_c_int, [_vp, *_EXPERTS_MAPS, _vp]),
    "experts_maps_validate": (_c_int, _EXPERTS_MAPS),
    "experts_max_rows": (_c_i64, [_c_int] * 3),
    "experts_gather": (_c_int, [_vp, *_EXPERTS_GATHER, _vp]),
    "experts_gather_validate": (_c_int, _EXPERTS_GATHER),
    "experts_combine": (_c_int, [_vp, *_EXPERTS_COMBINE, _vp]),
    "experts_combine_validate": (_c_int, _EXPERTS_COMBINE),
    "experts_combine_gradient": (_c_int, [_vp, *_EXPERTS_GRADIENT, _vp]),
    "experts_combine_gradient_validate": (_c_int, _EXPERTS_GRADIENT),
}
EXPORTED_SYMBOLS_F8 = tuple(_SIGNATURES_F8)

_lock = threading.Lock()
_lib = None


class GemmError(RuntimeError):
    """A negative gemm_f16 return code."""

    def __init__(self, code: int, where: str):
        self.code = code
        msg = gemm_f16_strerror(code)
        if code == ERR_CUDA:
            msg += f" [{gemm_f16_last_cuda_error()}]"
        super().__init__(f"{where}: {msg} (code {code})")


def load() -> ctypes.CDLL:
    """Load the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"gemm_f16 library not built ({LIB_PATH} missing); run "
                    "async_barrier_pipelined_gb300.build.build() first. "
                    "There is no fallback implementation.")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in (*_SIGNATURES.items(), *_SIGNATURES_F8.items()):
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(rc: int, where: str) -> int:
    if rc < 0:
        raise GemmError(rc, where)
    return rc


def gemm_f16_strerror(code: int) -> str:
    return load().gemm_f16_strerror(code).decode()


def gemm_f16_last_cuda_error() -> str:
    return load().gemm_f16_last_cuda_error().decode()


def gemm_f16_plan(device: int = 0) -> int:
    """Create a plan on ``device``; returns the opaque handle as an int."""
    h = _vp()
    _check(load().gemm_f16_plan(ctypes.byref(h), device), "gemm_f16_plan")
    return h.value


def gemm_f16_destroy(plan: int) -> None:
    _check(load().gemm_f16_destroy(plan), "gemm_f16_destroy")


def gemm_f16_status(plan: int) -> int:
    """Device-reported status since the last call (0, ERR_TIMEOUT or
    ERR_BAD_INDEX); clears it."""
    return load().gemm_f16_status(plan)


def gemm_f16_set_option(plan: int, option: int, value: int) -> None:
    _check(load().gemm_f16_set_option(plan, option, value), "gemm_f16_set_option")


def gemm_f16_get_option(plan: int, option: int) -> int:
    v = _c_i64()
    _check(load().gemm_f16_get_option(plan, option, ctypes.byref(v)), "gemm_f16_get_option")
    return v.value


def gemm_f16_run(plan: int, M: int, N: int, K: int, A: int, lda: int, B: int, ldb: int,
                 C: int, ldc: int, split_k: int = 1, stream: int = 0) -> None:
    """Enqueue C = A*B (device pointers) on ``stream`` (a cudaStream_t as int)."""
    _check(load().gemm_f16_run(plan, M, N, K, A, lda, B, ldb, C, ldc, split_k, stream),
           "gemm_f16_run")


def gemm_f16_run_ex(plan: int, layout: int, M: int, N: int, K: int, A: int, lda: int, B: int,
                    ldb: int, C: int, ldc: int, split_k: int = 1, stream: int = 0) -> None:
    """gemm_f16_run with an operand layout (LAYOUT_NN / TN / NT / TT)."""
    _check(load().gemm_f16_run_ex(plan, layout, M, N, K, A, lda, B, ldb, C, ldc, split_k,
                                  stream), "gemm_f16_run_ex")


def gemm_f16_run_host(plan: int, M: int, N: int, K: int, hA: int, lda: int, hB: int,
                      ldb: int, hC: int, ldc: int, split_k: int = 1, stream: int = 0) -> None:
    """Enqueue copy-in, C = A*B and copy-out for HOST pointers on ``stream``."""
    _check(load().gemm_f16_run_host(plan, M, N, K, hA, lda, hB, ldb, hC, ldc, split_k,
                                    stream), "gemm_f16_run_host")


def gemm_f16_run_noalloc(M: int, N: int, K: int, A: int, lda: int, B: int, ldb: int,
                         C: int, ldc: int, split_k: int = 1, status: int = 0,
                         stream: int = 0) -> None:
    """Enqueue C = A*B without a plan and without allocating device memory.

    For callers that may not call cudaMalloc (their device memory belongs to
    another allocator, or they cannot afford its device-wide sync).  Uses the
    library's fixed scratch array; ``status`` is 0 or the address of a
    device-visible int that receives ERR_TIMEOUT if a wait runs out.  Calls
    that overlap on the GPU race on the shared scratch.
    """
    _check(load().gemm_f16_run_noalloc(M, N, K, A, lda, B, ldb, C, ldc, split_k, status,
                                       stream), "gemm_f16_run_noalloc")


def gemm_f16_noalloc_status() -> int:
    """Read and clear the status word of no-alloc calls made with status 0
    on the current device (0, or ERR_TIMEOUT).  Call after their stream has
    been synchronised."""
    rc = int(load().gemm_f16_noalloc_status())
    if rc not in (0, ERR_TIMEOUT):
        _check(rc, "gemm_f16_noalloc_status")
    return rc


def gemm_f16_validate(M, N, K, A, lda, B, ldb, C, ldc, split_k) -> int:
    return load().gemm_f16_validate(M, N, K, A, lda, B, ldb, C, ldc, split_k)


def gemm_f16_validate_ex(layout, M, N, K, A, lda, B, ldb, C, ldc, split_k) -> int:
    return load().gemm_f16_validate_ex(layout, M, N, K, A, lda, B, ldb, C, ldc, split_k)


def _strides3(st):
    if st is None or len(st) != 3:
        raise ValueError("strides are (batch, head, row) in elements")
    return (_c_i64 * 3)(*[int(x) for x in st])


def attn_f16_fwd(plan: int, batch: int, heads: int, seq_q: int, seq_kv: int, head_dim: int,
                 Q: int, q_strides, K: int, k_strides, V: int, v_strides, O: int, o_strides,
                 scale: float, stream: int = 0) -> None:
    """Enqueue attention forward (device pointers; strides (batch, head, row))."""
    _check(load().attn_f16_fwd(plan, batch, heads, seq_q, seq_kv, head_dim,
                               Q, _strides3(q_strides), K, _strides3(k_strides),
                               V, _strides3(v_strides), O, _strides3(o_strides),
                               float(scale), stream), "attn_f16_fwd")


def attn_f16_validate(batch, heads, seq_q, seq_kv, head_dim, Q, q_strides, K, k_strides,
                      V, v_strides, O, o_strides, scale) -> int:
    return load().attn_f16_validate(batch, heads, seq_q, seq_kv, head_dim,
                                    Q, _strides3(q_strides), K, _strides3(k_strides),
                                    V, _strides3(v_strides), O, _strides3(o_strides),
                                    float(scale))


def gemm_f16_run_info(plan: int, layout: int, M: int, N: int, K: int, lda: int,
                      split_k: int = 1) -> dict:
    """What gemm_f16_run_ex would enqueue for these sizes (nothing is run)."""
    info = (_c_int * 4)()
    _check(load().gemm_f16_run_info(plan, layout, M, N, K, lda, split_k, info),
           "gemm_f16_run_info")
    return {"kernel": info[0], "launches": info[1], "repack_a": bool(info[2]),
            "tile_width": info[3]}


def gemm_f16_run_choice(layout: int, M: int, N: int, K: int, lda: int, split_k: int = 1,
                        num_sms: int = 152, max_pairs: int = 76, max_quads: int = 36) -> dict:
    """gemm_f16_run_info for default options on a device with these facts
    (host only; the defaults are a GB300's)."""
    info = (_c_int * 4)()
    _check(load().gemm_f16_run_choice(layout, M, N, K, lda, split_k, num_sms, max_pairs,
                                      max_quads, info), "gemm_f16_run_choice")
    return {"kernel": info[0], "launches": info[1], "repack_a": bool(info[2]),
            "tile_width": info[3]}


def gemm_f16_kernel_time(plan: int) -> tuple:
    """(total milliseconds, launches) of the kernels timed since the last
    read (OPT_KERNEL_TIMING); waits for the recorded events."""
    ms = ctypes.c_double(0.0)
    n = _c_i64(0)
    _check(load().gemm_f16_kernel_time(plan, ctypes.byref(ms), ctypes.byref(n)),
           "gemm_f16_kernel_time")
    return ms.value, n.value


def attn_f16_key_ranges(plan: int, batch: int, heads: int, seq_q: int, seq_kv: int) -> int:
    """Key ranges attn_f16_fwd would use for these sizes (1: no split)."""
    n = _c_int(0)
    _check(load().attn_f16_key_ranges(plan, batch, heads, seq_q, seq_kv, ctypes.byref(n)),
           "attn_f16_key_ranges")
    return n.value


def gemm_f16_tile_order(tiles_m: int, tiles_n: int, order: int = 0) -> list:
    """Tile order as a list of (tile_m, tile_n)."""
    n = _check(load().gemm_f16_tile_order(tiles_m, tiles_n, order, None, 0),
               "gemm_f16_tile_order")
    buf = (ctypes.c_uint32 * n)()
    _check(load().gemm_f16_tile_order(tiles_m, tiles_n, order, buf, n), "gemm_f16_tile_order")
    return [(v & 0xFFFF, v >> 16) for v in buf]


def gemm_f16_pair_tiles(M: int, N: int, pairs: int, split_k: int = 1, order: int = 0,
                        tile_width: int = 256, K: int = 4096, with_parts: bool = False):
    """CTA-pair work list as (row0, col0, width) tuples; with ``with_parts``
    also the K parts of the last (len % pairs) tiles: (tiles, parts)."""
    parts = _c_int(1)
    n = _check(load().gemm_f16_pair_tiles(M, N, K, pairs, split_k, order, tile_width, None, 0,
                                          ctypes.byref(parts)), "gemm_f16_pair_tiles")
    buf = (ctypes.c_uint32 * n)()
    _check(load().gemm_f16_pair_tiles(M, N, K, pairs, split_k, order, tile_width, buf, n, None),
           "gemm_f16_pair_tiles")
    tiles = [((v & 0xFFFF) * 256, ((v >> 16) & 0x3FFF) * 128, 128 << (v >> 30)) for v in buf]
    return (tiles, parts.value) if with_parts else tiles


def gemm_f16_tile_shape() -> tuple:
    """(BM, BN, BK, STAGES) of the compiled kernel."""
    vals = [_c_int() for _ in range(4)]
    load().gemm_f16_tile_shape(*[ctypes.byref(v) for v in vals])
    return tuple(v.value for v in vals)


class Plan:
    """Owning wrapper of a plan handle."""

    def __init__(self, device: int = 0):
        self.device = device
        self.handle = gemm_f16_plan(device)
        if int(os.environ.get("WORLD_SIZE") or 1) > 1:
            # One of several processes, each with its GPU: no multicast copies.
            self.set_option(OPT_MULTICAST, 0)

    def close(self):
        if self.handle:
            gemm_f16_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self) -> int:
        return gemm_f16_status(self.handle)

    def set_option(self, option: int, value: int) -> None:
        gemm_f16_set_option(self.handle, option, value)

    def get_option(self, option: int) -> int:
        return gemm_f16_get_option(self.handle, option)

    def kernel_time(self) -> tuple:
        """(total milliseconds, launches) of the product / attention kernels
        timed since the last read (see OPT_KERNEL_TIMING)."""
        return gemm_f16_kernel_time(self.handle)


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _operand(X, rows: int, cols: int, name: str):
    """(transposed, leading dimension) of a rows x cols view, or raise."""
    if X.stride(1) == 1 and (rows == 1 or X.stride(0) >= cols):
        return False, X.stride(0) if rows > 1 else cols
    if X.stride(0) == 1 and (cols == 1 or X.stride(1) >= rows):
        return True, X.stride(1) if cols > 1 else rows
    raise ValueError(f"{name} must be row-major or a transposed row-major view")


def matmul(plan: Plan, A, B, C=None, split_k: int = 1, stream=None):
    """C = A @ B for float16 CUDA tensors (C allocated if None).

    A and B may each be row-major or the transpose of a row-major tensor
    (``X.t()``); the matching operand layout is passed to the kernel, so no
    copy is made.  C must be row-major.  Forward only: C carries no gradient.
    """
    import torch
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("A and B must be torch.float16")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}")
    M, K = A.shape
    N = B.shape[1]
    at, lda = _operand(A, M, K, "A")
    bt, ldb = _operand(B, K, N, "B")
    if C is None:
        C = torch.empty((M, N), dtype=torch.float16, device=A.device)
    elif C.dtype != torch.float16 or tuple(C.shape) != (M, N) or C.stride(1) != 1:
        raise ValueError("C must be a row-major float16 M x N tensor")
    layout = (LAYOUT_TN if at else 0) | (LAYOUT_NT if bt else 0)
    gemm_f16_run_ex(plan.handle, layout, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                    C.data_ptr(), C.stride(0) if M > 1 else N, split_k, _stream_handle(stream))
    return C


def attention(plan: Plan, Q, K, V, O=None, scale=None, stream=None):
    """softmax(scale * Q K^T) V for float16 CUDA tensors of shape
    [batch, heads, seq, 256] (the last dimension contiguous; other strides
    free, so ``x.transpose(1, 2)`` of a [batch, seq, heads, 256] tensor works).
    ``scale`` defaults to 1/sqrt(256).  O is allocated if None.  Forward only:
    O carries no gradient."""
    import torch
    for name, X in (("Q", Q), ("K", K), ("V", V)):
        if X.dtype != torch.float16 or X.dim() != 4 or X.stride(3) != 1:
            raise ValueError(f"{name} must be a float16 [B, H, S, D] tensor with D contiguous")
    B, H, Sq, D = Q.shape
    Skv = K.shape[2]
    if tuple(K.shape) != (B, H, Skv, D) or tuple(V.shape) != (B, H, Skv, D):
        raise ValueError(f"shape mismatch {tuple(Q.shape)} {tuple(K.shape)} {tuple(V.shape)}")
    if O is None:
        O = torch.empty((B, H, Sq, D), dtype=torch.float16, device=Q.device)
    elif O.dtype != torch.float16 or tuple(O.shape) != (B, H, Sq, D) or O.stride(3) != 1:
        raise ValueError("O must be a float16 [B, H, Sq, D] tensor with D contiguous")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    st = lambda X: (X.stride(0), X.stride(1), X.stride(2))
    attn_f16_fwd(plan.handle, B, H, Sq, Skv, D, Q.data_ptr(), st(Q), K.data_ptr(), st(K),
                 V.data_ptr(), st(V), O.data_ptr(), st(O), scale, _stream_handle(stream))
    return O


def attn_f16_fwd_host(plan: int, batch: int, heads: int, seq_q: int, seq_kv: int, head_dim: int,
                      hQ: int, hK: int, hV: int, hO: int, scale: float, stream: int = 0) -> None:
    """The forward pass on contiguous host buffers (see attn_f16.h)."""
    _check(load().attn_f16_fwd_host(plan, batch, heads, seq_q, seq_kv, head_dim, hQ, hK, hV, hO,
                                    float(scale), stream), "attn_f16_fwd_host")


def attention_host(plan: Plan, hQ, hK, hV, hO, scale=None, stream=None):
    """attention() for contiguous float16 CPU tensors (pinned for asynchronous
    copies): Q, K, V are copied in and O out by the library, overlapping
    consecutive calls.  Synchronise the stream before reading hO."""
    import torch
    for name, X in (("Q", hQ), ("K", hK), ("V", hV), ("O", hO)):
        if X.dtype != torch.float16 or X.dim() != 4 or X.is_cuda or not X.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float16 CPU tensor [B, H, S, D]")
    B, H, Sq, D = hQ.shape
    Skv = hK.shape[2]
    if (tuple(hK.shape) != (B, H, Skv, D) or tuple(hV.shape) != (B, H, Skv, D)
            or tuple(hO.shape) != (B, H, Sq, D)):
        raise ValueError("shape mismatch")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    attn_f16_fwd_host(plan.handle, B, H, Sq, Skv, D, hQ.data_ptr(), hK.data_ptr(), hV.data_ptr(),
                      hO.data_ptr(), scale, _stream_handle(stream))
    return hO


# ---------------------------------------------------------------- paged cache
def attn_f16_paged_maps(plan: int, batch: int, cached: int, added: int, block_table: int,
                        table_stride: int, max_pages: int, free_pages: int, num_free: int,
                        free_head: int, page_size: int, max_tokens: int, starts: int,
                        kv_lens: int, positions: int, slots: int, free_head_out: int,
                        stream: int = 0) -> None:
    """Enqueue the maps of a serving step (device pointers; see attn_f16.h)."""
    _check(load().attn_f16_paged_maps(plan, batch, cached, added, block_table, table_stride,
                                      max_pages, free_pages, num_free, free_head, page_size,
                                      max_tokens, starts, kv_lens, positions, slots,
                                      free_head_out, stream), "attn_f16_paged_maps")


def attn_f16_paged_maps_validate(*args) -> int:
    """The argument check of attn_f16_paged_maps (its arguments without plan and stream)."""
    return load().attn_f16_paged_maps_validate(*args)


def attn_f16_paged_maps_overlap(*args) -> int:
    """Whether buffers of a maps call overlap (attn_f16_paged_maps_validate's
    arguments without page_size)."""
    return load().attn_f16_paged_maps_overlap(*args)


def _i64s(values):
    return None if values is None else (_c_i64 * len(values))(*[int(x) for x in values])


def attn_f16_rope(plan: int, tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                  rot_dim: int, layout: int, inverse: int, factor: float, turns: int,
                  positions: int, Q: int, q_strides, Qo: int, qo_strides, K: int = 0,
                  k_strides=None, V: int = 0, v_strides=None, slots: int = 0, Kc: int = 0,
                  kc_strides=None, Vc: int = 0, vc_strides=None, num_pages: int = 0,
                  page_size: int = 0, stream: int = 0) -> None:
    """Enqueue rotary positions, with the write of K and V into a paged cache
    when kv_heads > 0 (device pointers; see attn_f16.h)."""
    _check(load().attn_f16_rope(plan, tokens, q_heads, kv_heads, head_dim, rot_dim, layout,
                                inverse, factor, turns, positions, Q, _i64s(q_strides), Qo,
                                _i64s(qo_strides), K, _i64s(k_strides), V, _i64s(v_strides),
                                slots, Kc, _i64s(kc_strides), Vc, _i64s(vc_strides), num_pages,
                                page_size, stream), "attn_f16_rope")


def attn_f16_rope_validate(tokens, q_heads, kv_heads, head_dim, rot_dim, layout, factor, turns,
                           positions, Q, q_strides, Qo, qo_strides, K=0, k_strides=None, V=0,
                           v_strides=None, slots=0, Kc=0, kc_strides=None, Vc=0,
                           vc_strides=None, num_pages=0, page_size=0) -> int:
    return load().attn_f16_rope_validate(
        tokens, q_heads, kv_heads, head_dim, rot_dim, layout, factor, turns, positions, Q,
        _i64s(q_strides), Qo, _i64s(qo_strides), K, _i64s(k_strides), V, _i64s(v_strides), slots,
        Kc, _i64s(kc_strides), Vc, _i64s(vc_strides), num_pages, page_size)


def attn_f16_rope_turns(radians) -> list:
    """Frequencies in radians per position -> fixed-point turns (2^64 a turn)."""
    n = len(radians)
    out = (ctypes.c_uint64 * max(n, 1))()
    _check(load().attn_f16_rope_turns((ctypes.c_double * max(n, 1))(*radians), n, out),
           "attn_f16_rope_turns")
    return list(out[:n])


def attn_f16_paged_fwd(plan: int, batch: int, total_q: int, max_q: int, q_heads: int,
                       kv_heads: int, head_dim: int, Q: int, q_strides, Kc: int, kc_strides,
                       Vc: int, vc_strides, num_pages: int, page_size: int, block_table: int,
                       table_stride: int, max_pages: int, starts: int, kv_lens: int, O: int,
                       o_strides, scale: float, window: int = 0, sinks: int = 0,
                       stream: int = 0) -> None:
    """Enqueue attention over a paged cache (device pointers; see attn_f16.h)."""
    _check(load().attn_f16_paged_fwd(plan, batch, total_q, max_q, q_heads, kv_heads, head_dim, Q,
                                     _i64s(q_strides), Kc, _i64s(kc_strides), Vc,
                                     _i64s(vc_strides), num_pages, page_size, block_table,
                                     table_stride, max_pages, starts, kv_lens, O,
                                     _i64s(o_strides), scale, window, sinks, stream),
           "attn_f16_paged_fwd")


def attn_f16_paged_validate(batch, total_q, max_q, q_heads, kv_heads, head_dim, Q, q_strides, Kc,
                            kc_strides, Vc, vc_strides, num_pages, page_size, block_table,
                            table_stride, max_pages, starts, kv_lens, O, o_strides, scale,
                            window=0, sinks=0) -> int:
    return load().attn_f16_paged_validate(
        batch, total_q, max_q, q_heads, kv_heads, head_dim, Q, _i64s(q_strides), Kc,
        _i64s(kc_strides), Vc, _i64s(vc_strides), num_pages, page_size, block_table,
        table_stride, max_pages, starts, kv_lens, O, _i64s(o_strides), scale, window, sinks)


_calls = None


def _torch_calls():
    """The paged-cache calls for torch tensors (raises if they have not been built)."""
    global _calls
    if _calls is None:
        import torch  # noqa: F401  (the module links against it)
        load()
        with _lock:
            if _calls is None:
                if not os.path.exists(CALLS_PATH):
                    raise ImportError(
                        f"paged-cache calls not built ({CALLS_PATH} missing); run "
                        "async_barrier_pipelined_gb300.build.build() first. "
                        "There is no fallback implementation.")
                spec = importlib.util.spec_from_file_location(CALLS_NAME, CALLS_PATH)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                _calls = module
    return _calls


def _result(r, where: str):
    if type(r) is int:
        raise GemmError(r, where)
    return r


PagedMaps = collections.namedtuple("PagedMaps", "starts kv_lens positions slots free_head")
PagedMaps.__doc__ = """The maps of one serving step (see paged_maps)."""


def paged_maps(plan: Plan, cached, added, block_table, free_pages, free_head, page_size: int,
               max_tokens: int, out=None, stream=None) -> PagedMaps:
    """Block tables and slot maps of a serving step, built on the GPU from
    the requests' lengths.

    cached, added: int32 [batch], the tokens of each request that the cache
    holds already and the step's new ones.  block_table: int32 [batch,
    max_pages]; the pages that the new tokens need are taken from free_pages
    (int32 [n]) at free_head (int32 [1]) and written into it.  Returns
    starts [batch + 1], kv_lens [batch], positions and slots [max_tokens]
    (0 and -1 past the last token) and the new free_head [1], written into
    ``out`` (a PagedMaps of an earlier call) if given.  Nothing is advanced
    in place: ``out`` may not hold a tensor that is also an input (its
    kv_lens as ``cached``, its free_head as ``free_head``).
    """
    return PagedMaps._make(_result(
        (_calls or _torch_calls()).paged_maps(
            plan.handle, plan.device, cached, added, block_table, free_pages, free_head, page_size,
            max_tokens, out, stream if stream is None else _stream_handle(stream)),
        "attn_f16_paged_maps"))


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_len: int = 0, slow_turns: float = 1.0,
                     fast_turns: float = 32.0):
    """Frequencies (radians per position, one per pair) of rotary positions.

    scaling "none": base^(-2i/rot_dim).  "linear": divided by ``factor``
    (positions squeezed into the trained range).  "base": the base is raised
    to base * factor^(rot_dim/(rot_dim-2)), so that the slowest pair is
    slowed by ``factor`` and the fastest not at all.  "parts": pairs that make
    at least ``fast_turns`` turns over the trained ``original_len`` positions
    keep their frequency, those with at most ``slow_turns`` are slowed by
    ``factor``, with a ramp linear in the turns between; the values are then
    usually multiplied by 0.1 ln(factor) + 1 (the ``factor`` argument of
    rotary).
    """
    if rot_dim < 2 or rot_dim % 2 or not base > 1.0 or not factor > 0.0:
        raise ValueError("rot_dim must be even, base above 1 and factor above 0")
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("base scaling needs at least two pairs")
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in ("none", "base"):
        return f
    if scaling == "linear":
        return [w / factor for w in f]
    if scaling == "parts":
        if original_len < 1 or not fast_turns > slow_turns:
            raise ValueError("parts scaling needs original_len and fast_turns > slow_turns")
        out = []
        for w in f:
            keep = (original_len * w / (2.0 * math.pi) - slow_turns) / (fast_turns - slow_turns)
            keep = min(1.0, max(0.0, keep))
            out.append(w * keep + w / factor * (1.0 - keep))
        return out
    raise ValueError("scaling is 'none', 'linear', 'base' or 'parts'")


def rope_turns(frequencies):
    """Frequencies (radians per position, a list or a CPU tensor) as the int64
    tensor of fixed-point turns that rotary takes (2^64 a turn, as bits)."""
    import torch
    if isinstance(frequencies, torch.Tensor):
        frequencies = frequencies.tolist()
    bits = attn_f16_rope_turns([float(w) for w in frequencies])
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64)


def _rope_layout(layout: str) -> int:
    if layout == "half":
        return ROPE_HALF
    if layout == "interleaved":
        return ROPE_INTERLEAVED
    raise ValueError("layout is 'half' or 'interleaved'")


_Rotary = None


def _rotary_function():
    """rotary as an autograd function (made on first use: torch is not loaded
    with this module).  Its backward pass is the rotation back, by this
    function again, so that gradients of gradients exist too."""
    global _Rotary
    if _Rotary is None:
        import torch

        class Rotary(torch.autograd.Function):
            @staticmethod
            def forward(ctx, X, positions, turns, plan, layout, factor, inverse):
                ctx.save_for_backward(positions, turns)
                ctx.call = plan, layout, factor, inverse
                return rotary(plan, X, positions, turns, layout=layout, factor=factor,
                              inverse=inverse)

            @staticmethod
            def backward(ctx, dY):
                positions, turns = ctx.saved_tensors
                plan, layout, factor, inverse = ctx.call
                # A gradient may be laid out in ways that X may not (one number for
                # all of it, say).
                dY = dY.contiguous()
                if dY.data_ptr() % 16:
                    dY = dY.clone()
                return (rotary(plan, dY, positions, turns, layout=layout, factor=factor,
                               inverse=not inverse), None, None, None, None, None, None)

        _Rotary = Rotary
    return _Rotary


def rotary(plan: Plan, X, positions, turns, out=None, layout: str = "half", factor: float = 1.0,
           inverse: bool = False, stream=None):
    """Rotary positions of X, float16 [tokens, heads, 256] (tokens and heads
    may be strided): the first 2 * len(turns) numbers of each head are rotated
    by the token's position (int32 [tokens]), in pairs (i, i + half) or, with
    layout "interleaved", (2i, 2i + 1), and multiplied by ``factor``; the rest
    is copied.  turns: int64, from rope_turns, on the device.  ``inverse``
    rotates back: given the gradient of the output it returns the gradient
    of X.  ``out`` may be X.  Where X requires a gradient the result carries
    it (``out`` cannot be given then); ``plan`` must last until the backward
    pass.
    """
    if getattr(X, "requires_grad", False):
        import torch
        if torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out cannot be given where X requires a gradient")
            call = (X, positions, turns, plan, layout, factor, inverse)
            if stream is None:
                return _rotary_function().apply(*call)
            # The backward pass runs on the stream that is current here.
            handle = _stream_handle(stream)
            on = (torch.cuda.ExternalStream(handle, device=plan.device) if handle
                  else torch.cuda.default_stream(plan.device))
            with torch.cuda.stream(on):
                return _rotary_function().apply(*call)
    return _result(
        (_calls or _torch_calls()).rotary(
            plan.handle, plan.device, X, positions, turns, out, _rope_layout(layout), factor,
            inverse, stream if stream is None else _stream_handle(stream)), "attn_f16_rope")


def rotary_to_cache(plan: Plan, Q, K, V, positions, slots, turns, K_cache, V_cache, out=None,
                    layout: str = "half", factor: float = 1.0, stream=None):
    """Rotary positions of a step's new queries and keys, with the rotated
    keys and the values written into their slots of a paged cache.

    Q: float16 [tokens, q_heads, 256]; K, V: [tokens, kv_heads, 256] (all may
    be strided, e.g. views of one projection's output).  K_cache, V_cache:
    [pages, page_size, kv_heads, 256], any strides with the last dimension
    contiguous.  positions, slots: int32 [tokens], from paged_maps (slot -1:
    nothing is written).  Returns the rotated Q (in ``out``, which may be Q).
    Forward only: neither it nor the caches carry a gradient.
    """
    return _result(
        (_calls or _torch_calls()).rotary_to_cache(
            plan.handle, plan.device, Q, K, V, positions, slots, turns, K_cache, V_cache, out,
            _rope_layout(layout), factor, stream if stream is None else _stream_handle(stream)),
        "attn_f16_rope")


def paged_attention(plan: Plan, Q, K_cache, V_cache, block_table, starts, kv_lens, max_q: int,
                    out=None, scale=None, window: int = 0, sinks: int = 0, stream=None):
    """Causal attention of a step's new tokens over their requests' pages.

    Q: float16 [tokens, q_heads, 256], the new tokens of all requests one
    after another (request b's from starts[b] to starts[b + 1] - 1), the last
    of them at position kv_lens[b] - 1.  K_cache, V_cache: [pages, page_size,
    kv_heads, 256] (page_size a multiple of 8), holding the new tokens' keys
    and values too; query head h reads key/value head h * kv_heads // q_heads.
    block_table: int32 [batch, max_pages]; starts [batch + 1], kv_lens
    [batch]: int32.  max_q: the most new tokens a request has (a larger number
    is fine).  A token at position p sees the keys at j <= p; with ``window``
    only j > p - window and the first ``sinks`` of its request.  ``scale``
    defaults to 1/sqrt(256).  Rows that see no key, and rows past the last
    request's, are 0.  Forward only: the result carries no gradient.
    """
    return _result(
        (_calls or _torch_calls()).paged_attention(
            plan.handle, plan.device, Q, K_cache, V_cache, block_table, starts, kv_lens, max_q, out,
            ATTN_HEAD_DIM ** -0.5 if scale is None else scale, window, sinks,
            stream if stream is None else _stream_handle(stream)), "attn_f16_paged_fwd")


# ---------------------------------------------------------------- 8-bit products
def gemm_f8_quantize(plan: int, blocks: int, format: int, type: int, batch: int, rows: int,
                     cols: int, X: int, ldx: int, x_batch: int, source: int, choices: int,
                     x_rows: int, Q: int, ldq: int, q_batch: int, S: int, Q2: int = 0, S2: int = 0,
                     stream: int = 0) -> None:
    """Enqueue a quantisation into blocks of 128 (device pointers; see gemm_f8.h)."""
    _check(load().gemm_f8_quantize(plan, blocks, format, type, batch, rows, cols, X, ldx, x_batch,
                                   source, choices, x_rows, Q, ldq, q_batch, S, Q2, S2, stream),
           "gemm_f8_quantize")


def gemm_f8_quantize_validate(*args) -> int:
    """The argument check of gemm_f8_quantize (its arguments without plan and stream)."""
    return load().gemm_f8_quantize_validate(*args)


def gemm_f8_run(plan: int, form: int, M: int, N: int, K: int, experts: int, starts: int,
                A: GemmF8Operand, B: GemmF8Operand, C: int, ldc: int, c_batch: int, type: int,
                accumulate: int = 0, workspace: int = 0, workspace_bytes: int = 0,
                stream: int = 0) -> None:
    """Enqueue a product of 8-bit operands with block scales (see gemm_f8.h)."""
    _check(load().gemm_f8_run(plan, form, M, N, K, experts, starts, ctypes.byref(A),
                              ctypes.byref(B), C, ldc, c_batch, type, accumulate, workspace,
                              workspace_bytes, stream), "gemm_f8_run")


def gemm_f8_workspace(plan: int, form: int, M: int, N: int, K: int, experts: int = 1,
                      a_transposed: int = 0) -> int:
    """Bytes of workspace that gemm_f8_run needs for these sizes."""
    return load().gemm_f8_workspace(plan, form, M, N, K, experts, a_transposed)


def gemm_f8_run_choice(form: int, M: int, N: int, K: int, experts: int = 1, a_transposed: int = 0,
                       num_sms: int = 152, max_pairs: int = 76, sm_limit: int = 0) -> dict:
    """What a gemm_f8_run of these sizes launches on a device with these facts
    (host only; the defaults are a GB300's; see gemm_f8.h)."""
    info = (_c_int * 4)()
    _check(load().gemm_f8_run_choice(form, M, N, K, experts, a_transposed, num_sms, max_pairs,
                                     sm_limit, info), "gemm_f8_run_choice")
    return {"kernel": info[0], "parts": info[1], "ctas": info[2], "join_ctas": info[3]}


def gemm_f8_validate(form, M, N, K, experts, starts, A, B, C, ldc, c_batch, type,
                     accumulate=0) -> int:
    return load().gemm_f8_validate(form, M, N, K, experts, starts, A and ctypes.byref(A),
                                   B and ctypes.byref(B), C, ldc, c_batch, type, accumulate)


def experts_maps(plan: int, entries: int, experts: int, wide: int, num_experts: int, align: int,
                 max_rows: int, starts: int, rows: int, source: int, stream: int = 0) -> None:
    """Enqueue the sort of entries by expert (device pointers; see gemm_f8.h)."""
    _check(load().experts_maps(plan, entries, experts, wide, num_experts, align, max_rows, starts,
                               rows, source, stream), "experts_maps")


def experts_maps_validate(*args) -> int:
    return load().experts_maps_validate(*args)


def experts_max_rows(entries: int, num_experts: int, align: int = 1) -> int:
    """Rows that hold any choice of experts."""
    return _check(load().experts_max_rows(entries, num_experts, align), "experts_max_rows")


def experts_gather(plan: int, type: int, rows: int, cols: int, X: int, ldx: int, x_rows: int,
                   choices: int, source: int, Y: int, ldy: int, stream: int = 0) -> None:
    """Enqueue the gather of rows in the experts' order (see gemm_f8.h)."""
    _check(load().experts_gather(plan, type, rows, cols, X, ldx, x_rows, choices, source, Y, ldy,
                                 stream), "experts_gather")


def experts_gather_validate(*args) -> int:
    return load().experts_gather_validate(*args)


def experts_combine(plan: int, type: int, tokens: int, choices: int, cols: int, S: int, lds: int,
                    s_rows: int, rows: int, weights: int, weights_type: int, Y: int, ldy: int,
                    stream: int = 0) -> None:
    """Enqueue the weighted sums of the experts' rows (see gemm_f8.h)."""
    _check(load().experts_combine(plan, type, tokens, choices, cols, S, lds, s_rows, rows, weights,
                                  weights_type, Y, ldy, stream), "experts_combine")


def experts_combine_validate(*args) -> int:
    return load().experts_combine_validate(*args)


def experts_combine_gradient(plan: int, type: int, tokens: int, choices: int, cols: int, dY: int,
                             lddy: int, S: int, lds: int, s_rows: int, rows: int, source: int,
                             weights: int, weights_type: int, dS: int, ldds: int, dw: int,
                             stream: int = 0) -> None:
    """Enqueue experts_combine's gradients (see gemm_f8.h)."""
    _check(load().experts_combine_gradient(plan, type, tokens, choices, cols, dY, lddy, S, lds,
                                           s_rows, rows, source, weights, weights_type, dS, ldds,
                                           dw, stream), "experts_combine_gradient")


def experts_combine_gradient_validate(*args) -> int:
    return load().experts_combine_gradient_validate(*args)


class Blocks(collections.namedtuple("Blocks", "data scales")):
    """8-bit codes with a scale for each block of 128: data, float8_e4m3fn or
    float8_e5m2 [.., rows, cols], and scales, float32 with an entry for each
    block (see quantize).  ``t()`` is the transposed matrix, without a copy."""
    __slots__ = ()

    def t(self) -> "Blocks":
        return Blocks(self.data.transpose(-1, -2), self.scales.transpose(-1, -2))


class ExpertMaps(collections.namedtuple("ExpertMaps", "starts rows source")):
    """The order of tokens' choices by expert (see expert_maps).  ``align``: what
    each expert's rows are filled up to a multiple of (None: not known)."""
    align = None


_F8_BLOCKS = {"rows": F8_ROWS, "columns": F8_COLUMNS, "tiles": F8_TILES, "both": F8_BOTH}


def _f8_format(dtype) -> int:
    import torch
    if dtype is None or dtype == torch.float8_e4m3fn:
        return F8_E4M3
    if dtype == torch.float8_e5m2:
        return F8_E5M2
    raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")


def _f8_type(dtype) -> int:
    import torch
    if dtype is None or dtype == torch.float16:
        return F8_F16
    if dtype == torch.bfloat16:
        return F8_BF16
    if dtype == torch.float32:
        return F8_F32
    raise TypeError("dtype must be torch.float16, bfloat16 or float32")


def quantize(plan: Plan, X, blocks: str = "rows", dtype=None, maps=None, stream=None):
    """X (float16, bfloat16 or float32, [rows, cols] or [matrices, rows, cols],
    row-major or a transposed view) as 8-bit codes with a scale for each block
    of 128: ``blocks`` "rows" (128 numbers along a row; scales [rows,
    ceil(cols / 128)]), "columns" (along a column; [ceil(rows / 128), cols]) or
    "tiles" (128 x 128).  "both" returns two Blocks, "rows" and "columns", from
    one reading.  dtype: torch.float8_e4m3fn (if None) or float8_e5m2.

    scale = max(largest finite magnitude, 2^-100) / the format's largest number;
    a code is the nearest to x / scale (computed as x times the rounded
    reciprocal).  Infinities and NaN become NaN.  With ``maps`` (an ExpertMaps)
    X's rows are those of tokens, and the result's are in the experts' order,
    as of expert_gather(X).  The codes carry no gradient.
    """
    if blocks not in _F8_BLOCKS:
        raise ValueError("blocks is 'rows', 'columns', 'tiles' or 'both'")
    source, choices = None, 1
    if maps is not None:
        source, choices = maps.source, maps.rows.shape[1]
        if X.dim() != 2 or X.shape[0] != maps.rows.shape[0]:
            raise ValueError("X must have a row for each token of the maps")
    r = _result((_calls or _torch_calls()).quantize(
        plan.handle, plan.device, X, _F8_BLOCKS[blocks], _f8_format(dtype), source, choices,
        stream if stream is None else _stream_handle(stream)), "gemm_f8_quantize")
    return (Blocks(r[0], r[1]), Blocks(r[2], r[3])) if len(r) == 4 else Blocks(r[0], r[1])


def matmul_f8(plan: Plan, A, B, C=None, dtype=None, starts=None, accumulate: bool = False,
              stream=None):
    """C = A @ B for Blocks A [M, K] and B [K, N] whose blocks lie along K or
    are tiles (both row-major or transposed views; codes on 16-byte boundaries,
    as quantize makes them).  C: float16 (if None), bfloat16 or float32 by
    ``dtype``, or given; FP32 sums, rounded once.  ``accumulate`` adds to a
    given float32 C.

    With ``starts`` (int32 [experts + 1], from expert_maps) the product is by
    expert.  B [experts, K, N]: rows starts[e] to starts[e + 1] - 1 of A times
    B[e], and rows past the last expert's are 0.  B [K, N]: C [experts, M, N],
    each of A's columns and B's rows starts[e] to starts[e + 1] - 1, 0 where
    there are none: the gradient of weights.  Here starts are multiples of 128;
    C is NaN for an expert whose starts are not, and plan.status() tells.
    Forward only: C carries no gradient (linear_f8 does).
    """
    return _result((_calls or _torch_calls()).matmul_f8(
        plan.handle, plan.device, A.data, A.scales, B.data, B.scales, C, _f8_type(dtype), starts,
        accumulate, stream if stream is None else _stream_handle(stream)), "gemm_f8_run")


_no_change = contextlib.nullcontext()


def _on_stream(plan: Plan, stream):
    """A context in which ``stream`` (None: no change) is the current one: an
    autograd function's backward pass runs on its forward pass's stream."""
    if stream is None:
        return _no_change
    import torch
    handle = _stream_handle(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, device=plan.device) if handle
                             else torch.cuda.default_stream(plan.device))


def linear_f8(plan: Plan, X, W, starts=None, dtype=None, grad_dtype=None, stream=None):
    """X @ W^T in 8 bits, with its gradients: X [.., K] and W [N, K], float16,
    bfloat16 or float32, each quantised here (X by rows, W by tiles); or W as
    Blocks of tiles ([N, K], from quantize), which then carries no gradient.
    The result has X's type.  Backward, the gradient of the result is quantised
    by rows for X's gradient and along the rows' dimension, like X, for W's;
    ``dtype`` and ``grad_dtype`` are the formats of X and W and of that
    gradient (float8_e4m3fn if None).  X's gradient has X's type, W's W's.
    Forward-mode derivatives are refused (here, and in expert_gather and
    expert_combine).

    With ``starts`` (an ExpertMaps, or its starts) X is [rows, K], sorted by
    expert, and W [experts, N, K]; for W's gradient the starts are multiples of
    128 (expert_maps with align=128) and rows that no expert has are 0, as
    expert_gather leaves them.  An ExpertMaps of another align is refused where W
    requires a gradient; with starts alone that gradient is NaN for each expert
    whose starts are none (plan.status() tells too).  ``plan`` must last until the backward pass, which runs on the stream of the call.
    To capture a backward pass into a CUDA graph, take it with torch.autograd.grad:
    a leaf whose ``grad`` is accumulated stays tied, by torch, to the stream of an
    earlier graph of it that is still alive.
    """
    W, codes, scales = (None, *W) if isinstance(W, Blocks) else (W, None, None)
    if isinstance(starts, ExpertMaps):
        align, starts = starts.align, starts.starts
        if align is not None and align % 128 and W is not None and W.requires_grad:
            import torch
            if torch.is_grad_enabled():
                raise ValueError(f"W's gradient needs maps with align=128 (these have {align})")
    with _on_stream(plan, stream):
        return _result((_calls or _torch_calls()).linear_f8(
            plan, plan.device, X, W, codes, scales, starts, _f8_format(dtype),
            _f8_format(grad_dtype)), "linear_f8")


# ---------------------------------------------------------------- experts


def expert_maps(plan: Plan, experts, num_experts: int, align: int = 1, stream=None) -> ExpertMaps:
    """The order by expert of the choices of a router: experts, int32 or int64
    [tokens, choices], the expert that each choice goes to (negative: none).

    Returns starts [num_experts + 1], each expert's first row, a multiple of
    ``align``; rows [tokens, choices], the row of each choice (-1: none), by
    expert and then by token; and source [rows], the choice (token * choices +
    choice) at each row, -1 for those that fill an expert's rows up and those
    past the last expert.  There are as many rows as any router can need
    (experts_max_rows), so that a step's shapes do not depend on its tokens.
    """
    maps = ExpertMaps._make(_result((_calls or _torch_calls()).expert_maps(
        plan.handle, plan.device, experts, num_experts, align,
        stream if stream is None else _stream_handle(stream)), "experts_maps"))
    maps.align = align
    return maps


def expert_gather(plan: Plan, X, maps: ExpertMaps, stream=None):
    """The rows of X (float16, bfloat16 or float32 [tokens, cols]) in the
    experts' order: row r is that of the token of maps.source[r], 0 where there
    is none.  Differentiable (the gradient is expert_combine's sum)."""
    with _on_stream(plan, stream):
        return _result((_calls or _torch_calls()).expert_gather(
            plan, plan.device, X, maps.rows, maps.source), "experts_gather")


def expert_combine(plan: Plan, S, maps: ExpertMaps, weights=None, stream=None):
    """Each token's sum over its choices of weights times rows of S (float16,
    bfloat16 or float32 [rows, cols], in the experts' order): FP32 sums in the
    choices' order, rounded once.  weights: [tokens, choices], float32 or of
    S's type (None: all 1); choices without a row are left out.  Differentiable
    in S and weights."""
    with _on_stream(plan, stream):
        return _result((_calls or _torch_calls()).expert_combine(
            plan, plan.device, S, maps.rows, maps.source, weights), "experts_combine")
