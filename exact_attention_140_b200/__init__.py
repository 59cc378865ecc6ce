"""Python binding of libattn, the sm_100a fused exact-attention forward.

Each function here has the name of a C entry point in ``include/attn.h`` and
only marshals arguments (tensor -> device pointer, stream -> handle) before
calling into ``libattn.so``; every step of the computation runs in the CUDA
kernels.  There is no fallback: if the shared library is missing or cannot be
loaded, importing this package raises.

``attention()`` is a convenience wrapper that allocates the outputs with
PyTorch and calls ``attn_fwd``.  The serving operators have such wrappers too:
``Rope`` / ``qk_norm_rope``, ``KVCache`` / ``kv_write`` / ``kv_read``,
``attention_varlen`` and ``attention_paged`` take torch tensors, check them,
and allocate outputs and workspace.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = [
    "ATTN_BF16", "ATTN_FP8_E4M3", "AttnError", "attn_fwd", "attn_fwd_fp8", "attn_hadamard_quant_fp8",
    "attn_hadamard_quant_fp8_workspace_bytes", "attn_get_last_device_error", "attn_status_string",
    "attn_kv_tile_count", "attn_tile_kind", "attn_debug_unsatisfied_wait", "attn_debug_exp2", "attention",
    "attn_fwd_schedule", "attn_hadamard_quant_fp8_noalloc", "attn_fwd_splitkv", "attn_splitkv_workspace_bytes",
    "attn_combine", "attn_kv_tile_count_window", "attn_tile_kind_window", "attn_gemm_add", "lib_path", "EXPORTS",
    "attn_debug_map_cache_stats", "attn_fwd_part", "attn_shard_units", "attention_shard", "attn_fwd_host",
    "attn_rope_freqs", "attn_qk_norm_rope", "attn_kv_write", "attn_kv_read", "attn_fwd_varlen",
    "attn_fwd_varlen_workspace_bytes", "attn_fwd_paged", "attn_fwd_paged_workspace_bytes", "rope_freqs", "Rope",
    "KVCache", "qk_norm_rope", "kv_write", "kv_read", "attention_varlen", "attention_paged",
]

ATTN_BF16 = 0
ATTN_FP8_E4M3 = 1
STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_MISALIGNED",
          4: "ATTN_ERR_CUDA", 5: "ATTN_ERR_DEVICE_TIMEOUT", 6: "ATTN_ERR_DEVICE_INDEX"}

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libattn.so")

# every symbol include/attn.h declares
EXPORTS = (
    "attn_fwd", "attn_fwd_fp8", "attn_hadamard_quant_fp8", "attn_hadamard_quant_fp8_workspace_bytes",
    "attn_get_last_device_error", "attn_status_string", "attn_kv_tile_count", "attn_tile_kind",
    "attn_debug_unsatisfied_wait", "attn_debug_exp2", "attn_hadamard_quant_fp8_noalloc", "attn_fwd_schedule",
    "attn_fwd_splitkv", "attn_splitkv_workspace_bytes", "attn_combine", "attn_kv_tile_count_window",
    "attn_tile_kind_window", "attn_gemm_add", "attn_debug_map_cache_stats", "attn_fwd_part", "attn_shard_units",
    "attn_fwd_host", "attn_rope_freqs", "attn_qk_norm_rope", "attn_kv_write", "attn_kv_read", "attn_fwd_varlen",
    "attn_fwd_varlen_workspace_bytes", "attn_fwd_paged", "attn_fwd_paged_workspace_bytes",
)

if not os.path.exists(lib_path):
    raise ImportError(f"libattn.so is not built ({lib_path}); run `python exact_attention_140_b200/build.py` "
                      "or __graft_entry__.build()")
_lib = ctypes.CDLL(lib_path)

_vp, _I, _LL, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
_lib.attn_fwd.argtypes = [_vp] * 5 + [_I] * 7 + [_F, _I, _vp]
_lib.attn_fwd.restype = _I
_lib.attn_fwd_part.argtypes = [_vp] * 5 + [_I] * 7 + [_F, _I] + [_I] * 4 + [_vp]
_lib.attn_fwd_part.restype = _I
_lib.attn_shard_units.argtypes = [_I] * 4 + [ctypes.POINTER(_I)]
_lib.attn_fwd_host.argtypes = [_vp] * 10 + [_I] * 7 + [_F, _I, _vp]
_lib.attn_fwd_host.restype = _I
_lib.attn_shard_units.restype = _I
_lib.attn_fwd_fp8.argtypes = [_vp] * 5 + [_I] * 7 + [_F, _vp, _vp, _vp, _vp]
_lib.attn_fwd_fp8.restype = _I
_lib.attn_hadamard_quant_fp8.argtypes = [_vp, _vp, _vp, _vp, _LL, _I, _vp, _vp]
_lib.attn_hadamard_quant_fp8.restype = _I
_lib.attn_hadamard_quant_fp8_noalloc.argtypes = [_vp, _vp, _vp, _LL, _I, _vp, _vp]
_lib.attn_hadamard_quant_fp8_noalloc.restype = _I
_lib.attn_hadamard_quant_fp8_workspace_bytes.argtypes = []
_lib.attn_hadamard_quant_fp8_workspace_bytes.restype = _LL
_lib.attn_get_last_device_error.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint)]
_lib.attn_get_last_device_error.restype = _I
_lib.attn_status_string.argtypes = [_I]
_lib.attn_status_string.restype = ctypes.c_char_p
_lib.attn_kv_tile_count.argtypes = [_I] * 6
_lib.attn_kv_tile_count.restype = _I
_lib.attn_tile_kind.argtypes = [_I] * 7
_lib.attn_tile_kind.restype = _I
_lib.attn_fwd_schedule.argtypes = [_I] * 3
_lib.attn_fwd_schedule.restype = _I
_lib.attn_debug_unsatisfied_wait.argtypes = [_LL, _vp]
_lib.attn_debug_unsatisfied_wait.restype = _I
_lib.attn_debug_exp2.argtypes = [_vp, _vp, _LL, _I, _vp]
_lib.attn_debug_exp2.restype = _I
_lib.attn_splitkv_workspace_bytes.argtypes = [_I] * 7
_lib.attn_splitkv_workspace_bytes.restype = _LL
_lib.attn_fwd_splitkv.argtypes = [_vp] * 5 + [_I] * 7 + [_F, _I, _vp, _LL, _vp]
_lib.attn_fwd_splitkv.restype = _I
_lib.attn_combine.argtypes = [_vp, _vp] + [_I] * 5 + [_vp, _vp, _vp]
_lib.attn_combine.restype = _I
_lib.attn_kv_tile_count_window.argtypes = [_I] * 7
_lib.attn_kv_tile_count_window.restype = _I
_lib.attn_tile_kind_window.argtypes = [_I] * 8
_lib.attn_tile_kind_window.restype = _I
_lib.attn_gemm_add.argtypes = [_vp] * 4 + [_I] * 3 + [_vp]
_lib.attn_gemm_add.restype = _I
_lib.attn_debug_map_cache_stats.argtypes = [ctypes.POINTER(ctypes.c_ulonglong)] * 2
_lib.attn_debug_map_cache_stats.restype = _I


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("k_exp", _vp), ("v_exp", _vp), ("n_pages", _I),
                ("page_size", _I), ("Hkv", _I), ("d", _I), ("dtype", _I)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("q_weight", _vp), ("k_weight", _vp), ("freqs", _vp), ("eps", _F), ("amplitude", _F),
                ("rot_dim", _I), ("interleaved", _I)]


_D = ctypes.c_double
_pc, _pr = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_RopeStruct)
_lib.attn_rope_freqs.argtypes = [ctypes.POINTER(_D), _I, _D, _I, _D, _D, _D, _D, ctypes.POINTER(_F)]
_lib.attn_rope_freqs.restype = _I
_lib.attn_qk_norm_rope.argtypes = [_vp] * 4 + [_LL, _I, _I, _I] + [_LL] * 4 + [_vp, _pr, _vp]
_lib.attn_qk_norm_rope.restype = _I
_lib.attn_kv_write.argtypes = [_pc, _vp, _vp, _LL, _LL, _LL, _vp, _pr, _vp, _vp, _vp, _I, _LL, _LL, _vp]
_lib.attn_kv_write.restype = _I
_lib.attn_kv_read.argtypes = [_pc, _vp, _I, _vp, _I, _vp, _vp, _LL, _vp]
_lib.attn_kv_read.restype = _I
_lib.attn_fwd_varlen_workspace_bytes.argtypes = [_I] * 5
_lib.attn_fwd_varlen_workspace_bytes.restype = _LL
_lib.attn_fwd_varlen.argtypes = [_vp] * 5 + [_I] * 3 + [_vp] * 2 + [_I] * 3 + [_LL] * 3 + [_I, _F, _vp, _LL, _vp]
_lib.attn_fwd_varlen.restype = _I
_lib.attn_fwd_paged_workspace_bytes.argtypes = [_pc] + [_I] * 5
_lib.attn_fwd_paged_workspace_bytes.restype = _LL
_lib.attn_fwd_paged.argtypes = [_vp, _pc, _vp, _vp, _I, _I, _I, _vp, _vp, _I, _vp, _I, _I, _LL, _I, _F, _vp, _LL, _vp]
_lib.attn_fwd_paged.restype = _I


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({attn_status_string(status)})")


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str, raise_on_error: bool):
    if rc != 0 and raise_on_error:
        raise AttnError(rc, where)
    return rc


def attn_status_string(status: int) -> str:
    return _lib.attn_status_string(int(status)).decode()


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, dtype=ATTN_BF16, stream=None,
             raise_on_error=True):
    rc = _lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, int(causal),
                       float(scale), int(dtype), _stream(stream))
    return _check(rc, "attn_fwd", raise_on_error)


def attn_fwd_part(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, dtype, b_begin, b_end, kvh_begin,
                  kvh_end, stream=None, raise_on_error=True):
    rc = _lib.attn_fwd_part(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, int(causal),
                            float(scale), int(dtype), int(b_begin), int(b_end), int(kvh_begin), int(kvh_end),
                            _stream(stream))
    return _check(rc, "attn_fwd_part", raise_on_error)


def attn_fwd_host(q_h, k_h, v_h, o_h, lse_h, q_d, k_d, v_d, o_d, lse_d, B, Hq, Hkv, Nq, Nk, d, causal, scale,
                  n_chunks=0, stream=None, raise_on_error=True):
    """attn_fwd with host inputs/outputs (pinned for overlap) and caller-owned
    device buffers; the copies in, kernels and copies out are pipelined over
    n_chunks runs of (batch, key/value head) units (0: the library's default)."""
    rc = _lib.attn_fwd_host(_ptr(q_h), _ptr(k_h), _ptr(v_h), _ptr(o_h), _ptr(lse_h), _ptr(q_d), _ptr(k_d),
                            _ptr(v_d), _ptr(o_d), _ptr(lse_d), B, Hq, Hkv, Nq, Nk, d, int(causal), float(scale),
                            int(n_chunks), _stream(stream))
    return _check(rc, "attn_fwd_host", raise_on_error)


def attn_shard_units(B, Hkv, world, rank):
    """Rank `rank`'s share of the B x Hkv (batch, key/value head) units as a list
    of (b_begin, b_end, kvh_begin, kvh_end) rectangles."""
    buf = (_I * 12)()
    n = _lib.attn_shard_units(int(B), int(Hkv), int(world), int(rank), buf)
    if n < 0:
        raise AttnError(1, "attn_shard_units")
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


def attention_shard(q, k, v, o, lse, rank, world, causal=False, scale=None, stream=None):
    """This rank's share of attention over full bf16 tensors q [B,Nq,Hq,d],
    k/v [B,Nk,Hkv,d] into o/lse (the other ranks' rows are not written);
    returns the rectangles computed."""
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rects = attn_shard_units(B, Hkv, world, rank)
    for (b0, b1, g0, g1) in rects:
        attn_fwd_part(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, ATTN_BF16, b0, b1, g0, g1, stream)
    return rects


def attn_splitkv_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, n_splits=0) -> int:
    return int(_lib.attn_splitkv_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, n_splits))


def attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, n_splits, workspace, workspace_bytes,
                     stream=None, raise_on_error=True):
    rc = _lib.attn_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, int(causal),
                               float(scale), int(n_splits), _ptr(workspace), int(workspace_bytes), _stream(stream))
    return _check(rc, "attn_fwd_splitkv", raise_on_error)


def attn_combine(o_parts, lse_parts, n_splits, B, Hq, Nq, d, o, lse, stream=None, raise_on_error=True):
    rc = _lib.attn_combine(_ptr(o_parts), _ptr(lse_parts), n_splits, B, Hq, Nq, d, _ptr(o), _ptr(lse),
                           _stream(stream))
    return _check(rc, "attn_combine", raise_on_error)


def attn_gemm_add(a, b, c, d, M, N, K, stream=None, raise_on_error=True):
    rc = _lib.attn_gemm_add(_ptr(a), _ptr(b), _ptr(c), _ptr(d), M, N, K, _stream(stream))
    return _check(rc, "attn_gemm_add", raise_on_error)


def attn_fwd_fp8(q8, k8, v8, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, descale_q, descale_k, descale_v,
                 stream=None, raise_on_error=True):
    rc = _lib.attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, int(causal),
                           float(scale), _ptr(descale_q), _ptr(descale_k), _ptr(descale_v), _stream(stream))
    return _check(rc, "attn_fwd_fp8", raise_on_error)


def attn_hadamard_quant_fp8_workspace_bytes() -> int:
    return int(_lib.attn_hadamard_quant_fp8_workspace_bytes())


def attn_hadamard_quant_fp8(x, x8, descale, workspace, rows, d, signs=None, stream=None, raise_on_error=True):
    rc = _lib.attn_hadamard_quant_fp8(_ptr(x), _ptr(x8), _ptr(descale), _ptr(workspace), int(rows), int(d),
                                      _ptr(signs), _stream(stream))
    return _check(rc, "attn_hadamard_quant_fp8", raise_on_error)


def attn_hadamard_quant_fp8_noalloc(x, x8, descale, rows, d, signs=None, stream=None, raise_on_error=True):
    """attn_hadamard_quant_fp8 with the library's own static scratch (no workspace)."""
    rc = _lib.attn_hadamard_quant_fp8_noalloc(_ptr(x), _ptr(x8), _ptr(descale), int(rows), int(d), _ptr(signs),
                                              _stream(stream))
    return _check(rc, "attn_hadamard_quant_fp8_noalloc", raise_on_error)


def attn_get_last_device_error(stream=None):
    """Returns (status, raw error word); synchronises the stream."""
    w = ctypes.c_uint(0)
    rc = _lib.attn_get_last_device_error(_stream(stream), ctypes.byref(w))
    return rc, w.value


def attn_kv_tile_count(row0, row1, Nq, Nk, bn, causal) -> int:
    return int(_lib.attn_kv_tile_count(row0, row1, Nq, Nk, bn, int(causal)))


def attn_tile_kind(row0, row1, kt, Nq, Nk, bn, causal) -> int:
    return int(_lib.attn_tile_kind(row0, row1, kt, Nq, Nk, bn, int(causal)))


def attn_kv_tile_count_window(row0, row1, Nq, Nk, shift, bn, causal) -> int:
    return int(_lib.attn_kv_tile_count_window(row0, row1, Nq, Nk, shift, bn, int(causal)))


def attn_tile_kind_window(row0, row1, kt, Nq, Nk, shift, bn, causal) -> int:
    return int(_lib.attn_tile_kind_window(row0, row1, kt, Nq, Nk, shift, bn, int(causal)))


def attn_fwd_schedule(Nk, d, causal) -> int:
    """1 if attn_fwd runs the persistent kernel for Nk keys at head size d, 0 for one block per item."""
    return int(_lib.attn_fwd_schedule(Nk, d, int(causal)))


def attn_debug_unsatisfied_wait(limit_ns: int, stream=None, raise_on_error=True):
    rc = _lib.attn_debug_unsatisfied_wait(int(limit_ns), _stream(stream))
    return _check(rc, "attn_debug_unsatisfied_wait", raise_on_error)


def attn_debug_map_cache_stats():
    """(hits, encodes) of the library's tensor-map cache."""
    h, e = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
    _check(_lib.attn_debug_map_cache_stats(ctypes.byref(h), ctypes.byref(e)), "attn_debug_map_cache_stats", True)
    return h.value, e.value


def attn_debug_exp2(x, y, n, mode, stream=None, raise_on_error=True):
    rc = _lib.attn_debug_exp2(_ptr(x), _ptr(y), int(n), int(mode), _stream(stream))
    return _check(rc, "attn_debug_exp2", raise_on_error)


def attention(q, k, v, causal: bool = False, scale: float | None = None, return_lse: bool = True, stream=None):
    """O, LSE for torch tensors q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d] (bf16, CUDA, contiguous)."""
    import torch
    B, Nq, Hq, d = q.shape
    _, Nk, Hkv, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("attention() takes bf16 tensors; use attn_fwd_fp8 for e4m3")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if return_lse else None
    attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, ATTN_BF16, stream)
    return (o, lse) if return_lse else o


# ------------------------------------------------------------------ serving
ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3}


def attn_rope_freqs(rot_dim, base, kind=0, factor=1.0, trained_len=0.0, fast_turns=32.0, slow_turns=1.0):
    """(frequencies as a list of rot_dim / 2 floats, amplitude); host only."""
    buf, amp = (_D * max(int(rot_dim) // 2, 1))(), _F(0.0)
    _check(_lib.attn_rope_freqs(buf, int(rot_dim), float(base), int(kind), float(factor), float(trained_len),
                                float(fast_turns), float(slow_turns), ctypes.byref(amp)), "attn_rope_freqs", True)
    return list(buf), amp.value


def attn_qk_norm_rope(q, k, q_out, k_out, T, Hq, Hkv, d, q_stride, k_stride, q_out_stride, k_out_stride, positions,
                      rope, stream=None, raise_on_error=True):
    rc = _lib.attn_qk_norm_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), T, Hq, Hkv, d, q_stride, k_stride,
                                q_out_stride, k_out_stride, _ptr(positions), rope, _stream(stream))
    return _check(rc, "attn_qk_norm_rope", raise_on_error)


def attn_kv_write(cache, k, v, T, k_stride, v_stride, slots, rope=None, positions=None, q=None, q_out=None, Hq=0,
                  q_stride=0, q_out_stride=0, stream=None, raise_on_error=True):
    rc = _lib.attn_kv_write(cache, _ptr(k), _ptr(v), T, k_stride, v_stride, _ptr(slots), rope, _ptr(positions), _ptr(q),
                            _ptr(q_out), Hq, q_stride, q_out_stride, _stream(stream))
    return _check(rc, "attn_kv_write", raise_on_error)


def attn_kv_read(cache, table, table_width, cu, n_seqs, k, v, T, stream=None, raise_on_error=True):
    rc = _lib.attn_kv_read(cache, _ptr(table), table_width, _ptr(cu), n_seqs, _ptr(k), _ptr(v), T, _stream(stream))
    return _check(rc, "attn_kv_read", raise_on_error)


def attn_fwd_varlen_workspace_bytes(Tq, n_seqs, Hq, Hkv, d) -> int:
    return int(_lib.attn_fwd_varlen_workspace_bytes(Tq, n_seqs, Hq, Hkv, d))


def attn_fwd_varlen(q, k, v, o, lse, Tq, Tk, n_seqs, cu_q, cu_k, Hq, Hkv, d, q_stride, k_stride, v_stride, causal,
                    scale, workspace, workspace_bytes, stream=None, raise_on_error=True):
    rc = _lib.attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), Tq, Tk, n_seqs, _ptr(cu_q), _ptr(cu_k),
                              Hq, Hkv, d, q_stride, k_stride, v_stride, int(causal), scale, _ptr(workspace),
                              workspace_bytes, _stream(stream))
    return _check(rc, "attn_fwd_varlen", raise_on_error)


def attn_fwd_paged_workspace_bytes(cache, Tq, n_seqs, max_q, Hq, max_kv) -> int:
    return int(_lib.attn_fwd_paged_workspace_bytes(cache, Tq, n_seqs, max_q, Hq, max_kv))


def attn_fwd_paged(q, cache, o, lse, Tq, n_seqs, max_q, cu_q, table, table_width, kv_lens, max_kv, Hq, q_stride, causal,
                   scale, workspace, workspace_bytes, stream=None, raise_on_error=True):
    rc = _lib.attn_fwd_paged(_ptr(q), cache, _ptr(o), _ptr(lse), Tq, n_seqs, max_q, _ptr(cu_q), _ptr(table),
                             table_width, _ptr(kv_lens), max_kv, Hq, q_stride, int(causal), scale,
                             _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(rc, "attn_fwd_paged", raise_on_error)


torch = None  # the torch module, from the first use of a wrapper below
_bf16 = _f32 = _f64 = _i32 = _i64 = _u8 = None  # its types


def _load_torch():
    global torch, _bf16, _f32, _f64, _i32, _i64, _u8
    if torch is None:
        import torch as t
        _bf16, _f32, _f64, _i32, _i64, _u8 = t.bfloat16, t.float32, t.float64, t.int32, t.int64, t.uint8
        torch = t
    return torch


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _device_of(tensors):
    """The device index that all tensors (None: skipped) are on: -1 for the host, None without a tensor."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            _need(dev is None or d == dev, "the tensors are on different devices")
            dev = d
    return dev


def _on_current_device(*tensors):
    """Every tensor is on the current CUDA device (the library launches there); returns its index."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{cur}")
    return cur


def _rows(x, name):
    """(T, H, d, token stride) of a bf16 [T, H, d] tensor whose heads are contiguous."""
    if torch is None:
        _load_torch()
    if x.dtype is not _bf16 or x.dim() != 3:
        raise TypeError(f"{name} must be a bf16 tensor [T, H, d]")
    T, H, d = x.shape
    st, sh, sd = x.stride()
    if ((sd != 1 and d > 1) or (sh != d and H > 1)) and x.numel() > 0:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return T, H, d, st if T > 1 else H * d


def _index(x, name, dtype, n=None):
    """x is a contiguous 1-D tensor of the type, with n entries; returns their number."""
    if x.dtype is not dtype or x.dim() != 1 or not x.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D {dtype} tensor")
    m = x.shape[0]
    if n is not None and m != n:
        raise ValueError(f"{name} has {m} entries, {n} are needed")
    return m


def _table(x):
    """(sequences, width) of a page table."""
    if torch is None:
        _load_torch()
    if x.dtype is not _i32 or x.dim() != 2 or not x.is_contiguous():
        raise TypeError("table must be a contiguous 2-D int32 tensor")
    return x.shape


def _use_stream(stream, dev, *new):
    """The handle of the stream a call runs on (None: the current one).  Tensors allocated here belong to the
    current stream: the allocator is told of another one that uses them."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    if s != torch.cuda.current_stream():
        s.wait_stream(torch.cuda.current_stream())  # their memory may still be in use there
        for t in new:
            if t is not None:
                t.record_stream(s)
    return s.cuda_stream


def rope_freqs(rot_dim, base, kind="plain", factor=1.0, trained_len=0.0, fast_turns=32.0, slow_turns=1.0,
               device="cuda"):
    """(frequencies as an fp64 tensor on `device`, amplitude) for Rope()."""
    _load_torch()
    f, amp = attn_rope_freqs(rot_dim, base, ROPE_KINDS[kind], factor, trained_len, fast_turns, slow_turns)
    return torch.tensor(f, dtype=torch.float64, device=device), amp


class Rope:
    """Norm weights and rotation of queries and keys (attn_rope_t); keeps its tensors alive."""

    def __init__(self, freqs=None, rot_dim=0, interleaved=False, amplitude=1.0, q_weight=None, k_weight=None,
                 eps=1e-6):
        _load_torch()
        _need(rot_dim == 0 or freqs is not None, "freqs are needed where rot_dim > 0")
        if freqs is not None and rot_dim > 0:
            _index(freqs, "freqs", _f64, rot_dim // 2)
        d = None
        for w in (q_weight, k_weight):
            if w is not None:
                if w.dtype != torch.bfloat16 or w.dim() != 1 or not w.is_contiguous():
                    raise TypeError("norm weights must be contiguous bf16 tensors [d]")
                _need(d is None or w.shape[0] == d, "the norm weights differ in length")
                d = w.shape[0]
        self.d = d  # the head size the weights are for, None without weights
        self.tensors = (freqs, q_weight, k_weight)
        self.device = _device_of(self.tensors)
        self.rot_dim = rot_dim
        self.struct = _RopeStruct(_ptr(q_weight), _ptr(k_weight), _ptr(freqs) if rot_dim > 0 else None, eps, amplitude,
                                  rot_dim, int(interleaved))


class KVCache:
    """A paged key/value cache (attn_kv_cache_t) over torch tensors, which it keeps alive: k_pages and
    v_pages [n_pages, page_size, Hkv, d] in bf16 or float8_e4m3fn (or uint8 codes); for e4m3 the exponent
    bytes k_exp and v_exp [n_pages, page_size, Hkv] in uint8."""

    def __init__(self, k_pages, v_pages, k_exp=None, v_exp=None):
        _load_torch()
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8) or v_pages.dtype != k_pages.dtype:
            raise TypeError("k_pages and v_pages must both be bf16, float8_e4m3fn or uint8")
        _need(k_pages.dim() == 4 and k_pages.shape == v_pages.shape, "k_pages and v_pages must be [n_pages, page_size, Hkv, d]")
        e4m3 = k_pages.dtype != torch.bfloat16
        for e in (k_exp, v_exp):
            _need((e is not None) == e4m3, "an e4m3 cache needs k_exp and v_exp, a bf16 cache has none")
            if e is not None and (e.dtype != torch.uint8 or e.shape != k_pages.shape[:3]):
                raise TypeError("k_exp and v_exp must be uint8 [n_pages, page_size, Hkv]")
        for t in (k_pages, v_pages, k_exp, v_exp):
            _need(t is None or t.is_contiguous(), "the cache's tensors must be contiguous")
        self.tensors = (k_pages, v_pages, k_exp, v_exp)
        self.device = _device_of(self.tensors)
        self.n_pages, self.page_size, self.Hkv, self.d = k_pages.shape
        self.struct = _CacheStruct(_ptr(k_pages), _ptr(v_pages), _ptr(k_exp), _ptr(v_exp), self.n_pages,
                                   self.page_size, self.Hkv, self.d, ATTN_FP8_E4M3 if e4m3 else ATTN_BF16)


def _check_rope_use(rope, d, positions, T, dev):
    _need(rope.d is None or rope.d == d, "the norm weights are for another head size")
    if rope.rot_dim > 0:
        _need(positions is not None, "positions are needed where rot_dim > 0")
        _index(positions, "positions", _i64, T)
    _handle_device(rope, dev)


def _handle_device(handle, dev):
    if handle.device != dev and handle.device is not None:
        raise ValueError(f"the tensors of the {type(handle).__name__} are not on the current device cuda:{dev}")


def _like(x):
    """A new contiguous tensor of x's shape."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _out_rows(out, like, name):
    """Token stride of a given output tensor that must have the shape of `like`."""
    _need(out.shape == like.shape, f"{name} must have its input's shape")
    return _rows(out, name)[3]


def qk_norm_rope(q, k, positions, rope, q_out=None, k_out=None, stream=None):
    """q [T, Hq, d] and k [T, Hkv, d] (bf16, slices of a fused projection allowed) normed and rotated;
    returns (q_out, k_out), new contiguous tensors unless given (q_out=q and k_out=k work in place)."""
    T, Hq, d, qs = _rows(q, "q")
    Tk, Hkv, dk, ks = _rows(k, "k")
    _need(Tk == T and dk == d, "q and k must have the same tokens and head size")
    dev = _on_current_device(q, k, positions, q_out, k_out)
    _check_rope_use(rope, d, positions, T, dev)
    new_q = new_k = None
    if q_out is None:
        q_out = new_q = _like(q)
        qos = Hq * d
    else:
        qos = _out_rows(q_out, q, "q_out")
    if k_out is None:
        k_out = new_k = _like(k)
        kos = Hkv * d
    else:
        kos = _out_rows(k_out, k, "k_out")
    rc = _lib.attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), T, Hq, Hkv, d, qs, ks,
                                qos, kos, _ptr(positions), rope.struct, _use_stream(stream, dev, new_q, new_k))
    if rc:
        raise AttnError(rc, "attn_qk_norm_rope")
    return q_out, k_out


def kv_write(cache, k, v, slots, q=None, positions=None, rope=None, q_out=None, stream=None):
    """Keys and values [T, Hkv, d] (bf16) into the cache's slots (int64 [T], negative: skipped).  With rope the
    keys are normed and rotated on the way, and so are the queries q [T, Hq, d], which are returned."""
    T, Hkv, d, ks = _rows(k, "k")
    Tv, Hv, dv, vs = _rows(v, "v")
    _need(T == Tv and Hkv == Hv == cache.Hkv and d == dv == cache.d, "k and v must be [T, Hkv, d] of the cache")
    _index(slots, "slots", _i64, T)
    _need(rope is not None or q is None, "queries only take part where rope is given")
    dev = _on_current_device(k, v, slots, q, positions, q_out)
    _handle_device(cache, dev)
    rs = None
    if rope is not None:
        _check_rope_use(rope, d, positions, T, dev)
        rs = rope.struct
    Hq = qs = qos = 0
    new = None
    if q is not None:
        Tq, Hq, dq, qs = _rows(q, "q")
        _need(Tq == T and dq == d, "q must have k's tokens and head size")
        if q_out is None:
            q_out = new = _like(q)
            qos = Hq * d
        else:
            qos = _out_rows(q_out, q, "q_out")
    rc = _lib.attn_kv_write(cache.struct, k.data_ptr(), v.data_ptr(), T, ks, vs, slots.data_ptr(), rs, _ptr(positions),
                            _ptr(q), _ptr(q_out), Hq, qs, qos, _use_stream(stream, dev, new))
    if rc:
        raise AttnError(rc, "attn_kv_write")
    return q_out


def kv_read(cache, table, cu, T, k_out=None, v_out=None, stream=None):
    """The cached tokens of each sequence (pages table[s], int32; boundaries cu of the T output rows, int32
    [n_seqs + 1]) as packed bf16 keys and values [T, Hkv, d]."""
    n, width = _table(table)
    _index(cu, "cu", _i32, n + 1)
    dev = _on_current_device(table, cu, k_out, v_out)
    _handle_device(cache, dev)
    shape = (T, cache.Hkv, cache.d)
    new_k = new_v = None
    for t in (k_out, v_out):
        _need(t is None or (t.shape == shape and t.dtype is _bf16 and t.is_contiguous()),
              "k_out and v_out must be contiguous bf16 [T, Hkv, d]")
    if k_out is None:
        k_out = new_k = table.new_empty(shape, dtype=_bf16)
    if v_out is None:
        v_out = new_v = torch.empty_like(k_out)
    rc = _lib.attn_kv_read(cache.struct, table.data_ptr(), width, cu.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(), T,
                           _use_stream(stream, dev, new_k, new_v))
    if rc:
        raise AttnError(rc, "attn_kv_read")
    return k_out, v_out


def _outputs(q, T, H, o, lse, return_lse):
    """(o, lse, the ones that were made here)"""
    new_o = new_lse = None
    if o is None:
        o = new_o = _like(q)
    else:
        _need(o.shape == q.shape and o.dtype is _bf16 and o.is_contiguous(), "o must be contiguous bf16 like q")
    if lse is not None:
        _need(lse.shape == (H, T) and lse.dtype is _f32 and lse.is_contiguous(), "lse must be contiguous fp32 [Hq, T]")
    elif return_lse:
        lse = new_lse = q.new_empty((H, T), dtype=_f32)
    return o, lse, new_o, new_lse


def attention_varlen(q, k, v, cu_q, cu_k, causal: bool = False, scale: float | None = None, return_lse: bool = True,
                     o=None, lse=None, stream=None):
    """O [Tq, Hq, d] (and LSE [Hq, Tq]) of packed sequences: q [Tq, Hq, d], k/v [Tk, Hkv, d] (bf16, slices of a
    fused projection allowed), boundaries cu_q, cu_k int32 [n_seqs + 1].  Rows outside every sequence are
    not written."""
    Tq, Hq, d, qs = _rows(q, "q")
    Tk, Hkv, dk, ks = _rows(k, "k")
    Tv, Hv, dv, vs = _rows(v, "v")
    _need(Tv == Tk and Hv == Hkv and dv == dk == d, "k and v must have the same shape, and q's head size")
    n = _index(cu_q, "cu_q", _i32) - 1
    _index(cu_k, "cu_k", _i32, n + 1)
    dev = _on_current_device(q, k, v, cu_q, cu_k, o, lse)
    o, lse, new_o, new_lse = _outputs(q, Tq, Hq, o, lse, return_lse)
    nbytes = _lib.attn_fwd_varlen_workspace_bytes(Tq, n, Hq, Hkv, d)
    ws = q.new_empty(nbytes // 2) if nbytes > 0 else None  # (bf16 elements; the sizes are multiples of 256)
    rc = _lib.attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), Tq, Tk, n,
                              cu_q.data_ptr(), cu_k.data_ptr(), Hq, Hkv, d, qs, ks, vs, 1 if causal else 0,
                              d ** -0.5 if scale is None else scale, _ptr(ws), nbytes if nbytes > 0 else 0,
                              _use_stream(stream, dev, new_o, new_lse, ws))
    if rc:
        raise AttnError(rc, "attn_fwd_varlen")
    return (o, lse) if return_lse else o


def attention_paged(q, cache, table, kv_lens, cu_q=None, max_q=None, max_kv=None, causal: bool = True,
                    scale: float | None = None, return_lse: bool = True, o=None, lse=None, stream=None):
    """O [Tq, Hq, d] (and LSE [Hq, Tq]) of new tokens q over the cache, which holds them already: table int32
    [n_seqs, width], kv_lens int32 [n_seqs] with the new tokens counted.  cu_q int32 [n_seqs + 1] gives the
    sequences' rows of q and max_q bounds their number; without cu_q every sequence has Tq / n_seqs rows."""
    Tq, Hq, d, qs = _rows(q, "q")
    _need(d == cache.d, "q and the cache differ in head size")
    n, width = _table(table)
    _index(kv_lens, "kv_lens", _i32, n)
    if cu_q is not None:
        _index(cu_q, "cu_q", _i32, n + 1)
        max_q = Tq if max_q is None else min(max_q, Tq)
    else:
        each = Tq // n if n > 0 else 0
        _need(each * n == Tq and max_q in (None, each), "without cu_q every sequence has Tq / n_seqs rows")
        max_q = each
    if max_kv is None:
        max_kv = width * cache.page_size
    dev = _on_current_device(q, table, kv_lens, cu_q, o, lse)
    _handle_device(cache, dev)
    o, lse, new_o, new_lse = _outputs(q, Tq, Hq, o, lse, return_lse)
    nbytes = _lib.attn_fwd_paged_workspace_bytes(cache.struct, Tq, n, max_q, Hq, max_kv)
    ws = q.new_empty(nbytes // 2) if nbytes > 0 else None  # (bf16 elements; the sizes are multiples of 256)
    rc = _lib.attn_fwd_paged(q.data_ptr(), cache.struct, o.data_ptr(), _ptr(lse), Tq, n, max_q, _ptr(cu_q),
                             table.data_ptr(), width, kv_lens.data_ptr(), max_kv, Hq, qs, 1 if causal else 0,
                             d ** -0.5 if scale is None else scale, _ptr(ws), nbytes if nbytes > 0 else 0,
                             _use_stream(stream, dev, new_o, new_lse, ws))
    if rc:
        raise AttnError(rc, "attn_fwd_paged")
    return (o, lse) if return_lse else o
