"""ctypes binding of libmala.so (declared in include/mala.h).

The raw entry points keep the C names (``mala_fwd``, ``mala_bwd``,
``mala_decode`` ...) and only marshal arguments: shapes are read from the
torch tensors, pointers and the current CUDA stream are passed through, and a
non-OK status raises :class:`MalaError`.  Every step of the computation runs
in the library's CUDA kernels; there is no other implementation behind these
names.  ``forward`` / ``backward`` / ``decode`` allocate outputs and
workspace with torch and call the raw entry points.  The serving entry points
(``mala_cache_write``, ``mala_cache_read``, ``mala_decode_quant``,
``mala_decode_shared``) go through the compiled ``_binding.so`` instead, which
calls the same library.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MALA_LIBRARY=debug selects the bounds-checked build (same kernels compiled
# with -DMALA_DEBUG); anything else, or unset, the release build.
LIB_PATH = os.path.join(_HERE, "libmala_debug.so" if os.environ.get("MALA_LIBRARY") == "debug" else "libmala.so")

MALA_BF16, MALA_FP32 = 0, 1
STATUS = {0: "MALA_OK", 1: "MALA_ERR_INVALID_ARG", 2: "MALA_ERR_UNSUPPORTED", 3: "MALA_ERR_WORKSPACE",
          4: "MALA_ERR_CUDA", 5: "MALA_ERR_TIMEOUT"}
EXPORTS = ("mala_status_string", "mala_fwd", "mala_bwd_workspace_size", "mala_bwd",
           "mala_fwd_varlen", "mala_bwd_varlen_workspace_size", "mala_bwd_varlen",
           "mala_decode_workspace_size", "mala_decode", "mala_decode_per_head", "mala_decode_varlen",
           "mala_decode_noalloc", "mala_decode_noalloc_max_floats", "mala_device_status", "mala_launch_count",
           "mala_test_drop_next_load", "mala_last_cuda_error", "mala_cuda_error_string",
           "mala_fwd_forced", "mala_region_mass", "mala_cache_write", "mala_cache_read",
           "mala_decode_quant_workspace_size", "mala_decode_quant",
           "mala_decode_shared_workspace_size", "mala_decode_shared")


class MalaError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str = ""):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}" + (f" ({detail})" if detail else ""))
        self.code = code


_lib = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libmala.so (built by ``build.py``); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{os.path.basename(LIB_PATH)} not built ({LIB_PATH}); run "
                               "`python -m mass_adaptive_sparse_gb300.build` first")
        L = ctypes.CDLL(LIB_PATH)
        L.mala_status_string.restype = ctypes.c_char_p
        L.mala_status_string.argtypes = [_i]
        L.mala_fwd.restype = _i
        L.mala_fwd.argtypes = [_vp] * 5 + [_i] * 6 + [_i, _i, _i, _i, _i, _f, _f, _vp, _vp, _vp]
        L.mala_fwd_forced.restype = _i
        L.mala_fwd_forced.argtypes = [_vp] * 5 + [_i] * 6 + [_i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp]
        L.mala_region_mass.restype = _i
        L.mala_region_mass.argtypes = [_vp] * 4 + [_i] * 6 + [_i, _i, _i, _i, _f, _vp]
        L.mala_bwd_workspace_size.restype = _sz
        L.mala_bwd_workspace_size.argtypes = [_i] * 8
        L.mala_bwd.restype = _i
        L.mala_bwd.argtypes = [_vp] * 9 + [_i] * 6 + [_i, _i, _i, _i, _i, _f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_fwd_varlen.restype = _i
        L.mala_fwd_varlen.argtypes = [_vp] * 6 + [_i] * 6 + [_i, _i, _i, _i, _i, _f, _f, _vp, _vp, _vp]
        L.mala_bwd_varlen_workspace_size.restype = _sz
        L.mala_bwd_varlen_workspace_size.argtypes = [_i] * 6
        L.mala_bwd_varlen.restype = _i
        L.mala_bwd_varlen.argtypes = [_vp] * 10 + [_i] * 6 + [_i, _i, _i, _i, _i, _f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_decode_workspace_size.restype = _sz
        L.mala_decode_workspace_size.argtypes = [_i] * 4
        L.mala_decode.restype = _i
        L.mala_decode.argtypes = [_vp] * 5 + [_i] * 5 + [_i, _i, _i, _i, _f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_decode_per_head.restype = _i
        L.mala_decode_per_head.argtypes = [_vp] * 5 + [_i] * 5 + [_i, _i, _i, _i, _f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_decode_varlen.restype = _i
        L.mala_decode_varlen.argtypes = [_vp] * 6 + [_i] * 9 + [_f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_decode_noalloc.restype = _i
        L.mala_decode_noalloc.argtypes = [_vp] * 5 + [_i] * 5 + [_i, _i, _i, _i, _f, _f, _vp, _vp, _vp]
        L.mala_decode_noalloc_max_floats.restype = _sz
        L.mala_decode_noalloc_max_floats.argtypes = []
        L.mala_cache_write.restype = _i
        L.mala_cache_write.argtypes = [_vp] * 8 + [_i] * 6 + [_vp]
        L.mala_cache_read.restype = _i
        L.mala_cache_read.argtypes = [_vp] * 8 + [_i] * 7 + [_vp]
        L.mala_decode_quant_workspace_size.restype = _sz
        L.mala_decode_quant_workspace_size.argtypes = [_i] * 4
        L.mala_decode_quant.restype = _i
        L.mala_decode_quant.argtypes = [_vp] * 8 + [_i] * 9 + [_f, _f, _vp, _sz, _vp, _vp, _vp]
        L.mala_decode_shared_workspace_size.restype = _sz
        L.mala_decode_shared_workspace_size.argtypes = [_i] * 5
        L.mala_decode_shared.restype = _i
        L.mala_decode_shared.argtypes = [_vp] * 8 + [_i] * 10 + [_f, _vp, _sz, _vp]
        L.mala_device_status.restype = _i
        L.mala_device_status.argtypes = [_vp, ctypes.POINTER(_i)]
        L.mala_launch_count.restype = ctypes.c_uint64
        L.mala_launch_count.argtypes = []
        L.mala_test_drop_next_load.restype = None
        L.mala_test_drop_next_load.argtypes = []
        L.mala_last_cuda_error.restype = _i
        L.mala_last_cuda_error.argtypes = []
        L.mala_cuda_error_string.restype = ctypes.c_char_p
        L.mala_cuda_error_string.argtypes = [_i]
        _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MALA_BF16
    if t.dtype == torch.float32:
        return MALA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, code: int):
    if code != 0:
        detail = ""
        if code == 4:
            err = lib().mala_last_cuda_error()
            detail = f"cuda error {err}: {lib().mala_cuda_error_string(err).decode()}"
        raise MalaError(fn, code, detail)


def _scale(d, softmax_scale):
    return 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)


# ---------------------------------------------------------------------------
# Raw entry points (same names as the C ABI).
# ---------------------------------------------------------------------------

def mala_fwd(q, k, v, o, lse, *, causal=True, block=128, tau=1.0, softmax_scale=None,
             retained_counts=None, tile_mask=None, stream=None):
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    _check("mala_fwd", lib().mala_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Lq, Lk, Hq, Hkv, D, _dt(q), _dt(o),
        int(causal), block, block, float(tau), _scale(D, softmax_scale),
        _ptr(retained_counts), _ptr(tile_mask), _stream(stream)))


def mala_fwd_forced(q, k, v, o, lse, tile_keep, *, causal=True, block=128, softmax_scale=None,
                    retained_counts=None, tile_mask=None, stream=None):
    """Forward over the tiles `tile_keep` (uint8 [B, Hq, Tr, Tc]) marks, no test."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if tile_keep.dtype != torch.uint8 or tile_keep.shape != (B, Hq, -(-Lq // block), -(-Lk // block)):
        raise ValueError("tile_keep must be uint8 [B, Hq, ceil(Lq / block), ceil(Lk / block)]")
    _check("mala_fwd_forced", lib().mala_fwd_forced(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Lq, Lk, Hq, Hkv, D, _dt(q), _dt(o),
        int(causal), block, block, _scale(D, softmax_scale), _ptr(tile_keep),
        _ptr(retained_counts), _ptr(tile_mask), _stream(stream)))


def mala_region_mass(q, k, lse, region_mass, *, causal=True, block=128, softmax_scale=None, stream=None):
    """region_mass (fp32 [B, Hq, Tr, Tc]) = each (query block, key tile) region's
    softmax mass under the row log-normalisers `lse`, summed over the block's rows."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if region_mass.dtype != torch.float32 or region_mass.shape != (B, Hq, -(-Lq // block), -(-Lk // block)):
        raise ValueError("region_mass must be float32 [B, Hq, ceil(Lq / block), ceil(Lk / block)]")
    _check("mala_region_mass", lib().mala_region_mass(
        _ptr(q), _ptr(k), _ptr(lse), _ptr(region_mass), B, Lq, Lk, Hq, Hkv, D, _dt(q), int(causal),
        block, block, _scale(D, softmax_scale), _stream(stream)))


def mala_bwd_workspace_size(q, k, grad_dtype):
    B, Lq, Hq, D = q.shape
    return lib().mala_bwd_workspace_size(B, Lq, k.shape[1], Hq, k.shape[2], D, _dt(q),
                                         MALA_BF16 if grad_dtype == torch.bfloat16 else MALA_FP32)


def mala_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, *, causal=True, block=128, tau=1.0,
             softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    _check("mala_bwd", lib().mala_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
        B, Lq, Lk, Hq, Hkv, D, _dt(q), _dt(dq), int(causal), block, block, float(tau),
        _scale(D, softmax_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(retained_counts), _ptr(tile_mask), _stream(stream)))


def _check_cu(cu_seqlens, batch):
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (batch + 1,) or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor of shape [batch + 1]")


def mala_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen, *, causal=True, block=128, tau=1.0,
                    softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """Packed variable-length forward: q, o [total, Hq, D], k, v [total, Hkv, D],
    lse [Hq, total]; sequence b is rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.shape[0] - 1
    _check_cu(cu_seqlens, B)
    _check("mala_fwd_varlen", lib().mala_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), B, T, int(max_seqlen), Hq, Hkv, D,
        _dt(q), _dt(o), int(causal), block, block, float(tau), _scale(D, softmax_scale),
        _ptr(retained_counts), _ptr(tile_mask), _stream(stream)))


def mala_bwd_varlen_workspace_size(q, k, grad_dtype):
    T, Hq, D = q.shape
    return lib().mala_bwd_varlen_workspace_size(T, Hq, k.shape[1], D, _dt(q),
                                                MALA_BF16 if grad_dtype == torch.bfloat16 else MALA_FP32)


def mala_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, max_seqlen, workspace, *, causal=True,
                    block=128, tau=1.0, softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """Packed variable-length backward (layouts as mala_fwd_varlen)."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.shape[0] - 1
    _check_cu(cu_seqlens, B)
    _check("mala_bwd_varlen", lib().mala_bwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens),
        B, T, int(max_seqlen), Hq, Hkv, D, _dt(q), _dt(dq), int(causal), block, block, float(tau),
        _scale(D, softmax_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(retained_counts), _ptr(tile_mask), _stream(stream)))


def mala_decode_workspace_size(B, Hq, D, num_splits):
    return lib().mala_decode_workspace_size(B, Hq, D, num_splits)


def mala_decode(q, k_cache, v_cache, o, lse, workspace, *, block=128, num_splits=16, tau=1.0,
                softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    B, Hq, D = q.shape
    N, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check("mala_decode", lib().mala_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), B, N, Hq, Hkv, D, _dt(q), _dt(o),
        block, num_splits, float(tau), _scale(D, softmax_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(retained_counts), _ptr(tile_mask),
        _stream(stream)))


def mala_decode_per_head(q, k_cache, v_cache, o, lse, workspace, *, block=128, num_splits=16, tau=1.0,
                         softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """mala_decode with each query head deciding alone; counts / mask per query head."""
    B, Hq, D = q.shape
    N, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check("mala_decode_per_head", lib().mala_decode_per_head(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), B, N, Hq, Hkv, D, _dt(q), _dt(o),
        block, num_splits, float(tau), _scale(D, softmax_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(retained_counts), _ptr(tile_mask),
        _stream(stream)))


def mala_decode_varlen(q, k_cache, v_cache, o, lse, cache_lens, workspace, *, block=128, num_splits=16,
                       tau=1.0, softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """mala_decode with per-sequence cache lengths (int32 CUDA tensor [B]) over
    caches padded to k_cache.shape[1]."""
    B, Hq, D = q.shape
    N, Hkv = k_cache.shape[1], k_cache.shape[2]
    if cache_lens.dtype != torch.int32 or cache_lens.shape != (B,):
        raise ValueError("cache_lens must be an int32 tensor of shape [B]")
    _check("mala_decode_varlen", lib().mala_decode_varlen(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), _ptr(cache_lens), B, N, Hq, Hkv, D,
        _dt(q), _dt(o), block, num_splits, float(tau), _scale(D, softmax_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(retained_counts), _ptr(tile_mask),
        _stream(stream)))


def mala_decode_noalloc(q, k_cache, v_cache, o, lse, *, block=128, num_splits=16, tau=1.0,
                        softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """mala_decode with the split records in the library's fixed device array
    (for callers that cannot allocate; see include/mala.h)."""
    B, Hq, D = q.shape
    N, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check("mala_decode_noalloc", lib().mala_decode_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), B, N, Hq, Hkv, D, _dt(q), _dt(o),
        block, num_splits, float(tau), _scale(D, softmax_scale), _ptr(retained_counts), _ptr(tile_mask),
        _stream(stream)))


# The serving entry points.  Their marshalling is compiled (csrc/binding.cpp: checks
# of shapes, types and devices, a ValueError for each; outputs and workspace where
# None is given), because a decode step's calls are as short as the marshalling.

_binding = None


def _b():
    """The compiled binding, its functions those of the library that lib() loads."""
    global _binding
    if _binding is None:
        L = lib()
        try:
            from mass_adaptive_sparse_gb300 import _binding as m
        except ImportError as e:
            raise RuntimeError(f"_binding.so cannot be loaded ({e}); run "
                               "`python -m mass_adaptive_sparse_gb300.build` first") from e
        m.bind(*(ctypes.cast(f, _vp).value for f in (
            L.mala_cache_write, L.mala_cache_read, L.mala_decode_quant, L.mala_decode_quant_workspace_size,
            L.mala_decode_shared, L.mala_decode_shared_workspace_size)))
        _binding = m
    return _binding


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def mala_cache_write(k, v, k_codes, k_exps, v_codes, v_exps, *, starts=None, new_lens=None, stream=None):
    """Quantise rows of k, v [B, T, Hkv, D] into rows starts[b] .. of an 8-bit
    cache (codes e4m3 [B, N, Hkv, D], exps uint8 [B, Hkv, N]); `starts` and
    `new_lens` are int32 CUDA tensors [B] (default: 0 and T)."""
    code = _b().cache_write(k, v, k_codes, k_exps, v_codes, v_exps, starts, new_lens, _raw(stream))
    if code:
        _check("mala_cache_write", code)


def mala_cache_read(k_codes, k_exps, v_codes, v_exps, k, v, *, starts=None, lens=None, zero_rest=False, stream=None):
    """Write the values of an 8-bit cache's rows starts[b] .. to rows 0 .. of k, v
    [B, T, Hkv, D]; rows behind lens[b] stay as they are, or become zeros."""
    code, _, _ = _b().cache_read(k_codes, k_exps, v_codes, v_exps, k, v, -1, -1, starts, lens, int(zero_rest), _raw(stream))
    if code:
        _check("mala_cache_read", code)


def mala_decode_quant_workspace_size(B, Hq, D, num_splits):
    return lib().mala_decode_quant_workspace_size(B, Hq, D, num_splits)


def mala_decode_quant(q, k_codes, k_exps, v_codes, v_exps, o, lse, workspace, *, cache_lens=None, block=128,
                      num_splits=16, tau=1.0, softmax_scale=None, retained_counts=None, tile_mask=None, stream=None):
    """mala_decode over an 8-bit cache (mala_decode_varlen with cache_lens)."""
    code, _, _ = _b().decode_quant(q, k_codes, k_exps, v_codes, v_exps, o, lse, workspace, cache_lens, retained_counts,
                                   tile_mask, block, num_splits, tau, softmax_scale, -2, _raw(stream))
    if code:
        _check("mala_decode_quant", code)


def mala_decode_shared_workspace_size(B, Hq, D, prefix_splits, suffix_splits):
    return lib().mala_decode_shared_workspace_size(B, Hq, D, prefix_splits, suffix_splits)


def mala_decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, o, lse, workspace, *, suffix_lens=None,
                       prefix_splits=16, suffix_splits=1, softmax_scale=None, stream=None):
    """Exact decode of a batch behind one prefix [P, Hkv, D]; k_cache, v_cache
    [B, N, Hkv, D] hold the sequences' own rows (None: no sequence has any)."""
    code, _, _ = _b().decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, o, lse, workspace, suffix_lens,
                                    prefix_splits, suffix_splits, softmax_scale, -2, _raw(stream))
    if code:
        _check("mala_decode_shared", code)


def mala_device_status(stream=None) -> int:
    code = _i(0)
    rc = lib().mala_device_status(_stream(stream), ctypes.byref(code))
    if rc not in (0, 1, 5):     # OK, a rejected sequence length, an expired wait
        raise MalaError("mala_device_status", rc)
    return code.value


def mala_test_drop_next_load():
    """Failure-detection test hook: the next tensor-core forward call has one
    CTA's bounded waits expire (see include/mala.h)."""
    lib().mala_test_drop_next_load()


def mala_launch_count() -> int:
    return int(lib().mala_launch_count())


# ---------------------------------------------------------------------------
# Allocating conveniences.
# ---------------------------------------------------------------------------

def _ntiles(n, b):
    return -(-n // b)


def forward(q, k, v, tau=1.0, *, causal=True, block=128, softmax_scale=None, out_dtype=None,
            counts=False, mask=False, stream=None):
    """Returns (o, lse, info) with info holding 'counts' / 'mask' when asked."""
    B, Lq, Hq, D = q.shape
    o = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    tr, tc = _ntiles(Lq, block), _ntiles(k.shape[1], block)
    info = {}
    if counts:
        info["counts"] = torch.zeros((B, Hq, tr), dtype=torch.int32, device=q.device)
    if mask:
        info["mask"] = torch.zeros((B, Hq, tr, tc), dtype=torch.uint8, device=q.device)
    mala_fwd(q, k, v, o, lse, causal=causal, block=block, tau=tau, softmax_scale=softmax_scale,
             retained_counts=info.get("counts"), tile_mask=info.get("mask"), stream=stream)
    return o, lse, info


def backward(q, k, v, o, do, lse, tau=1.0, *, causal=True, block=128, softmax_scale=None,
             grad_dtype=torch.float32, counts=False, mask=False, stream=None):
    """Returns (dq, dk, dv, info)."""
    B, Lq, Hq, D = q.shape
    dev = q.device
    dq = torch.empty(q.shape, dtype=grad_dtype, device=dev)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=dev)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=dev)
    ws = torch.empty(max(256, mala_bwd_workspace_size(q, k, grad_dtype)), dtype=torch.uint8, device=dev)
    tr, tc = _ntiles(Lq, block), _ntiles(k.shape[1], block)
    info = {}
    if counts:
        info["counts"] = torch.zeros((B, Hq, tc), dtype=torch.int32, device=dev)
    if mask:
        info["mask"] = torch.zeros((B, Hq, tr, tc), dtype=torch.uint8, device=dev)
    mala_bwd(q, k, v, o, do, lse, dq, dk, dv, ws, causal=causal, block=block, tau=tau,
             softmax_scale=softmax_scale, retained_counts=info.get("counts"),
             tile_mask=info.get("mask"), stream=stream)
    return dq, dk, dv, info


def forward_varlen(q, k, v, cu_seqlens, max_seqlen, tau=1.0, *, causal=True, block=128, softmax_scale=None,
                   out_dtype=None, counts=False, mask=False, stream=None):
    """Packed variable-length forward; returns (o [total, Hq, D], lse [Hq, total], info)."""
    T, Hq, D = q.shape
    B = cu_seqlens.shape[0] - 1
    o = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    t = _ntiles(max_seqlen, block)
    info = {}
    if counts:
        info["counts"] = torch.zeros((B, Hq, t), dtype=torch.int32, device=q.device)
    if mask:
        info["mask"] = torch.zeros((B, Hq, t, t), dtype=torch.uint8, device=q.device)
    mala_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen, causal=causal, block=block, tau=tau,
                    softmax_scale=softmax_scale, retained_counts=info.get("counts"), tile_mask=info.get("mask"),
                    stream=stream)
    return o, lse, info


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen, tau=1.0, *, causal=True, block=128,
                    softmax_scale=None, grad_dtype=torch.float32, counts=False, mask=False, stream=None):
    """Packed variable-length backward; returns (dq, dk, dv, info)."""
    T, Hq, D = q.shape
    B = cu_seqlens.shape[0] - 1
    dev = q.device
    dq = torch.empty(q.shape, dtype=grad_dtype, device=dev)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=dev)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=dev)
    ws = torch.empty(max(256, mala_bwd_varlen_workspace_size(q, k, grad_dtype)), dtype=torch.uint8, device=dev)
    t = _ntiles(max_seqlen, block)
    info = {}
    if counts:
        info["counts"] = torch.zeros((B, Hq, t), dtype=torch.int32, device=dev)
    if mask:
        info["mask"] = torch.zeros((B, Hq, t, t), dtype=torch.uint8, device=dev)
    mala_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, max_seqlen, ws, causal=causal, block=block,
                    tau=tau, softmax_scale=softmax_scale, retained_counts=info.get("counts"),
                    tile_mask=info.get("mask"), stream=stream)
    return dq, dk, dv, info


def decode(q, k_cache, v_cache, tau=1.0, *, block=128, num_splits=16, softmax_scale=None,
           out_dtype=None, counts=False, mask=False, cache_lens=None, per_head=False, stream=None):
    """Returns (o, lse, info).  `cache_lens` (int32 CUDA tensor [B]) selects
    the variable-length decode over caches padded to k_cache.shape[1];
    `per_head` lets each query head decide alone (counts / mask per query head)."""
    B, Hq, D = q.shape
    N, Hkv = k_cache.shape[1], k_cache.shape[2]
    dev = q.device
    o = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    ws = torch.empty(max(256, mala_decode_workspace_size(B, Hq, D, num_splits)), dtype=torch.uint8, device=dev)
    info = {}
    if per_head and cache_lens is not None:
        raise ValueError("per_head and cache_lens are separate entry points")
    rows = Hq if per_head else Hkv
    if counts:
        info["counts"] = torch.zeros((B, rows, num_splits), dtype=torch.int32, device=dev)
    if mask:
        info["mask"] = torch.zeros((B, rows, _ntiles(N, block)), dtype=torch.uint8, device=dev)
    if per_head:
        mala_decode_per_head(q, k_cache, v_cache, o, lse, ws, block=block, num_splits=num_splits, tau=tau,
                             softmax_scale=softmax_scale, retained_counts=info.get("counts"),
                             tile_mask=info.get("mask"), stream=stream)
    elif cache_lens is None:
        mala_decode(q, k_cache, v_cache, o, lse, ws, block=block, num_splits=num_splits, tau=tau,
                    softmax_scale=softmax_scale, retained_counts=info.get("counts"),
                    tile_mask=info.get("mask"), stream=stream)
    else:
        mala_decode_varlen(q, k_cache, v_cache, o, lse, cache_lens, ws, block=block, num_splits=num_splits,
                           tau=tau, softmax_scale=softmax_scale, retained_counts=info.get("counts"),
                           tile_mask=info.get("mask"), stream=stream)
    return o, lse, info


def quant_cache(B, N, Hkv, D, device="cuda"):
    """An empty 8-bit cache for B sequences of up to N rows: (k_codes, k_exps,
    v_codes, v_exps), the tuple that cache_write, cache_read and decode_quant take."""
    codes = [torch.zeros((B, N, Hkv, D), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.ones((B, Hkv, N), dtype=torch.uint8, device=device) for _ in range(2)]
    return codes[0], exps[0], codes[1], exps[1]


def cache_write(k, v, cache, *, starts=None, new_lens=None, stream=None):
    """Quantise k, v [B, T, Hkv, D] into `cache`: row t of sequence b goes to
    cache row starts[b] + t, for t < new_lens[b] (defaults: 0 and T)."""
    mala_cache_write(k, v, *cache, starts=starts, new_lens=new_lens, stream=stream)


def cache_read(cache, T, *, dtype=None, starts=None, lens=None, out=None, stream=None):
    """(k, v) [B, T, Hkv, D] of `dtype` (None: bf16, or that of `out`): the values of cache rows starts[b] + t,
    t < lens[b].  Rows behind lens[b] keep what `out` holds (without `out`: zeros); `out` of another T or dtype than
    these is refused."""
    if stream is not None:
        with torch.cuda.stream(stream):        # its buffers belong to the stream that the call runs on
            return cache_read(cache, T, dtype=dtype, starts=starts, lens=lens, out=out)
    kc, ke, vc, ve = cache
    k, v = (None, None) if out is None else out
    if T < 0:
        raise ValueError(f"T must not be negative, got {T}")
    if out is not None and (k is None or v is None):
        raise ValueError("out must be two tensors")
    code, k, v = _b().cache_read(kc, ke, vc, ve, k, v, T, -1 if dtype is None else _code(dtype), starts, lens, out is None, None)
    if code:
        _check("mala_cache_read", code)
    return k, v


def _code(dtype):
    if dtype is torch.bfloat16:
        return MALA_BF16
    if dtype is torch.float32:
        return MALA_FP32
    raise TypeError(f"unsupported dtype {dtype}")


def decode_quant(q, cache, tau=1.0, *, block=128, num_splits=None, softmax_scale=None, out_dtype=None, counts=False,
                 mask=False, cache_lens=None, stream=None):
    """Decode over an 8-bit cache; returns (o, lse, info) as decode does.
    `num_splits` None: as many as fill the GPU, whether `counts` (which has an entry a split) and `mask` are asked for or
    not.  With tau > 0 each split decides for itself which tiles it keeps: give `num_splits` where the answer must not
    depend on the GPU, the batch, the cache's capacity and q's type."""
    if stream is not None:
        with torch.cuda.stream(stream):        # its buffers belong to the stream that the call runs on
            return decode_quant(q, cache, tau, block=block, num_splits=num_splits, softmax_scale=softmax_scale,
                                out_dtype=out_dtype, counts=counts, mask=mask, cache_lens=cache_lens)
    kc, ke, vc, ve = cache
    info = {}
    if counts:
        num_splits = _b().decode_quant_splits(q, kc, tau) if num_splits is None else num_splits
        if 1 <= num_splits <= 256:             # the library refuses the others
            info["counts"] = torch.zeros((kc.shape[0], kc.shape[2], num_splits), dtype=torch.int32, device=q.device)
    if mask:
        info["mask"] = torch.zeros((kc.shape[0], kc.shape[2], _ntiles(kc.shape[1], block)), dtype=torch.uint8,
                                   device=q.device)
    code, o, lse = _b().decode_quant(q, kc, ke, vc, ve, None, None, None, cache_lens, info.get("counts"),
                                     info.get("mask"), block, num_splits, tau, softmax_scale,
                                     -1 if out_dtype is None else _code(out_dtype), None)
    if code:
        _check("mala_decode_quant", code)
    return o, lse, info


def decode_shared(q, k_prefix, v_prefix, k_cache=None, v_cache=None, *, suffix_lens=None, prefix_splits=None,
                  suffix_splits=None, softmax_scale=None, out_dtype=None, stream=None):
    """Exact decode of a batch behind a shared prefix; returns (o, lse).
    `prefix_splits`, `suffix_splits` None: chosen for the GPU."""
    if stream is not None:
        with torch.cuda.stream(stream):        # its buffers belong to the stream that the call runs on
            return decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, suffix_lens=suffix_lens,
                                 prefix_splits=prefix_splits, suffix_splits=suffix_splits, softmax_scale=softmax_scale,
                                 out_dtype=out_dtype)
    code, o, lse = _b().decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, None, None, None, suffix_lens,
                                      prefix_splits, suffix_splits, softmax_scale, -1 if out_dtype is None else _code(out_dtype), None)
    if code:
        _check("mala_decode_shared", code)
    return o, lse
