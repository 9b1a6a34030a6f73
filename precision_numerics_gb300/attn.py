"""Python binding of libattn.so (ctypes): argument marshalling only.

Every function here checks tensor metadata, allocates outputs with PyTorch
when the caller does not pass them, and calls the C entry point of the same
name; all arithmetic runs in the library's CUDA kernels.  There is no CPU
fallback: if the library is missing or a call fails, an exception is raised.

Tensors are [B, H, N, d], contiguous, on the current CUDA device, either all
torch.bfloat16 (tensor-core path) or all torch.float32 (reference mode).  The
serving calls at the end (packed sequences, paged INT8 cache) state their own
layouts.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import warnings

import torch

from . import build as _build

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT = range(5)
ATTN_DTYPE_BF16, ATTN_DTYPE_FP32 = 0, 1

EXPORTED = ("attn_version", "attn_status_string", "attn_last_error", "attn_fwd",
            "attn_bwd_workspace_bytes", "attn_bwd", "attn_bwd_preprocess", "attn_bwd_main",
            "attn_bwd_dq_convert", "attn_check_status", "attn_selftest_wait_timeout",
            "attn_bwd_noalloc", "attn_fwd_stable", "attn_quantize_int8", "attn_fwd_int8",
            "attn_quantize_int8_as_bf16", "attn_fwd_int8_as_bf16",
            "attn_varlen_plan_bytes", "attn_varlen_plan", "attn_varlen_fwd",
            "attn_cache_append_int8", "attn_cache_read_int8",
            "attn_decode_int8_workspace_bytes", "attn_decode_int8")


class AttnError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{fn} failed: {_status_string(status)}"
                         + (f" -- {detail}" if detail else ""))


_LIB = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong

_SIGNATURES = {
    "attn_version": (_i, []),
    "attn_status_string": (ctypes.c_char_p, [_i]),
    "attn_last_error": (ctypes.c_char_p, []),
    "attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "attn_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_bwd": (_i, [_vp] * 9 + [_i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "attn_bwd_preprocess": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "attn_bwd_main": (_i, [_vp] * 6 + [_i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "attn_bwd_dq_convert": (_i, [_vp, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "attn_check_status": (_i, [_vp]),
    "attn_selftest_wait_timeout": (_i, [ctypes.c_ulonglong, _vp]),
    "attn_bwd_noalloc": (_i, [_vp] * 9 + [_i, _i, _i, _i, _f, _i, _vp]),
    "attn_fwd_stable": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _f, _i, _vp]),
    "attn_quantize_int8": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "attn_fwd_int8": (_i, [_vp] * 7 + [_i, _i, _i, _i, _f, _i, _vp]),
    "attn_quantize_int8_as_bf16": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "attn_fwd_int8_as_bf16": (_i, [_vp] * 7 + [_i, _i, _i, _i, _f, _i, _vp]),
    "attn_varlen_plan_bytes": (_sz, [_i] * 4),
    "attn_varlen_plan": (_i, [_vp] + [_i] * 5 + [_vp, _sz, _vp]),
    "attn_varlen_fwd": (_i, [_vp] * 3 + [_ll] * 6 + [_vp, _sz, _vp, _vp] + [_i] * 5 + [_f, _i, _vp]),
    "attn_cache_append_int8": (_i, [_vp] * 2 + [_ll] * 4 + [_vp] * 7 + [_i] * 7 + [_vp]),
    "attn_cache_read_int8": (_i, [_vp] * 9 + [_i] * 8 + [_vp]),
    "attn_decode_int8_workspace_bytes": (_sz, [_i] * 7),
    "attn_decode_int8": (_i, [_vp] + [_ll] * 3 + [_vp] * 8 + [_i] * 8 + [_f, _vp, _sz, _vp]),
}


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libattn.so (built by precision_numerics_gb300.build.build())."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build the CUDA library first "
                           "(python -m precision_numerics_gb300.build)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == _build.LIB:
        _LIB = lib
    return lib


_BINDING = None


class _NoBinding:
    """Takes no call: every one goes on to the checks and the ctypes call that follow."""

    varlen_fwd = cache_append = cache_read = decode = staticmethod(lambda *args: None)


def _binding():
    """The module _attn_torch (csrc/torch_calls.cpp): the serving calls in C++."""
    global _BINDING
    if _BINDING is None:
        load_library()
        path = _build.binding_path()
        try:
            loader = importlib.machinery.ExtensionFileLoader("_attn_torch", path)
            _BINDING = importlib.util.module_from_spec(importlib.util.spec_from_loader("_attn_torch", loader))
        except ImportError as e:
            warnings.warn(f"{path} cannot be loaded ({e}): serving calls take some 20 us of host time in place of 6 "
                          "(python -m precision_numerics_gb300.build)", RuntimeWarning, stacklevel=3)
            _BINDING = _NoBinding
    return _BINDING


def _status_string(status: int) -> str:
    try:
        return load_library().attn_status_string(status).decode()
    except Exception:  # noqa: BLE001 - only used to format an error
        return f"status {status}"


def _call(name: str, *args) -> int:
    lib = load_library()
    status = getattr(lib, name)(*args)
    if status != ATTN_OK:
        raise AttnError(name, status, lib.attn_last_error().decode())
    return status


def _stream(stream) -> int:
    if stream is None:
        # torch.cuda.current_stream() without the Stream object around the handle.
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return ATTN_DTYPE_BF16
    if t.dtype == torch.float32:
        return ATTN_DTYPE_FP32
    raise TypeError(f"attention tensors must be bfloat16 or float32, got {t.dtype}")


def _check_bhnd(name: str, t: torch.Tensor, shape=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, d], got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _check_lse(lse, B, H, N):
    if tuple(lse.shape) != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")


def _default_scale(d: int, scale):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def attn_version() -> int:
    return int(load_library().attn_version())


def attn_fwd(q, k, v, scale=None, causal=False, o=None, lse=None, stream=None):
    """O, LSE = attention forward.  Returns (o, lse)."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v)):
        _check_bhnd(name, t, q.shape, q.dtype)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_bhnd("o", o, q.shape, q.dtype)
    _check_lse(lse, B, H, N)
    _call("attn_fwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          B, H, N, d, _default_scale(d, scale), int(bool(causal)), _dtype_code(q), _stream(stream))
    return o, lse


def attn_fwd_stable(q, k, v, scale=None, causal=False, beta=2.0, o=None, lse=None, stream=None):
    """Forward with the stabilised normaliser (beta * repeated row max).  Returns (o, lse)."""
    _check_bhnd("q", q, dtype=torch.bfloat16)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v)):
        _check_bhnd(name, t, q.shape, q.dtype)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_bhnd("o", o, q.shape, q.dtype)
    _check_lse(lse, B, H, N)
    _call("attn_fwd_stable", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
          lse.data_ptr(), B, H, N, d, _default_scale(d, scale), int(bool(causal)), float(beta),
          ATTN_DTYPE_BF16, _stream(stream))
    return o, lse


def attn_quantize_int8(x, codes=None, scales=None, stream=None):
    """Per-token symmetric INT8 codes and FP32 scales of a BF16 [B,H,N,d] tensor."""
    _check_bhnd("x", x, dtype=torch.bfloat16)
    B, H, N, d = x.shape
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((B, H, N), dtype=torch.float32, device=x.device)
    _check_bhnd("codes", codes, x.shape, torch.int8)
    _check_lse(scales, B, H, N)
    _call("attn_quantize_int8", x.data_ptr(), codes.data_ptr(), scales.data_ptr(), B, H, N, d,
          _stream(stream))
    return codes, scales


def attn_fwd_int8(q8, q_scale, k8, k_scale, v, scale=None, causal=False, o=None, lse=None,
                  stream=None):
    """Forward on per-token INT8 Q and K (attn_quantize_int8) and BF16 V.  Returns (o, lse)."""
    _check_bhnd("v", v, dtype=torch.bfloat16)
    B, H, N, d = v.shape
    for name, t in (("q8", q8), ("k8", k8)):
        _check_bhnd(name, t, v.shape, torch.int8)
    _check_lse(q_scale, B, H, N)
    _check_lse(k_scale, B, H, N)
    if o is None:
        o = torch.empty_like(v)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=v.device)
    _check_bhnd("o", o, v.shape, v.dtype)
    _check_lse(lse, B, H, N)
    _call("attn_fwd_int8", q8.data_ptr(), q_scale.data_ptr(), k8.data_ptr(), k_scale.data_ptr(),
          v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d, _default_scale(d, scale),
          int(bool(causal)), _stream(stream))
    return o, lse


def int8_scale_rows(N: int) -> int:
    """Rows per head of the padded scale layout of the *_as_bf16 INT8 calls (N rounded up to 128)."""
    return (N + 127) // 128 * 128


def _check_padded_scales(name, t, B, H, N):
    if (tuple(t.shape) != (B, H, int8_scale_rows(N)) or t.dtype != torch.float32
            or not t.is_contiguous() or not t.is_cuda):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor [B, H, {int8_scale_rows(N)}]")


def attn_quantize_int8_as_bf16(x, codes=None, scales=None, stream=None):
    """attn_quantize_int8 with the codes held in BF16 and the scales padded to [B, H, N_pad]."""
    _check_bhnd("x", x, dtype=torch.bfloat16)
    B, H, N, d = x.shape
    if codes is None:
        codes = torch.empty_like(x)
    if scales is None:
        scales = torch.empty((B, H, int8_scale_rows(N)), dtype=torch.float32, device=x.device)
    _check_bhnd("codes", codes, x.shape, torch.bfloat16)
    _check_padded_scales("scales", scales, B, H, N)
    _call("attn_quantize_int8_as_bf16", x.data_ptr(), codes.data_ptr(), scales.data_ptr(), B, H, N,
          d, _stream(stream))
    return codes, scales


def attn_fwd_int8_as_bf16(q_codes, q_scale, k_codes, k_scale, v, scale=None, causal=False, o=None,
                          lse=None, stream=None):
    """attn_fwd_int8 on BF16-held codes (attn_quantize_int8_as_bf16), on the tcgen05 path."""
    _check_bhnd("v", v, dtype=torch.bfloat16)
    B, H, N, d = v.shape
    for name, t in (("q_codes", q_codes), ("k_codes", k_codes)):
        _check_bhnd(name, t, v.shape, torch.bfloat16)
    _check_padded_scales("q_scale", q_scale, B, H, N)
    _check_padded_scales("k_scale", k_scale, B, H, N)
    if o is None:
        o = torch.empty_like(v)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=v.device)
    _check_bhnd("o", o, v.shape, v.dtype)
    _check_lse(lse, B, H, N)
    _call("attn_fwd_int8_as_bf16", q_codes.data_ptr(), q_scale.data_ptr(), k_codes.data_ptr(),
          k_scale.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
          _default_scale(d, scale), int(bool(causal)), _stream(stream))
    return o, lse


def attn_bwd_workspace_bytes(B: int, H: int, N: int, d: int, dtype=torch.bfloat16) -> int:
    code = ATTN_DTYPE_BF16 if dtype == torch.bfloat16 else ATTN_DTYPE_FP32
    return int(load_library().attn_bwd_workspace_bytes(B, H, N, d, code))


def _workspace(q, workspace):
    B, H, N, d = q.shape
    need = attn_bwd_workspace_bytes(B, H, N, d, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if _nbytes(workspace) < need:
        raise ValueError(f"workspace too small: {_nbytes(workspace)} bytes, {need} needed")
    return workspace


def attn_bwd(q, k, v, o, lse, do, scale=None, causal=False, dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """dQ, dK, dV of L = sum(dO o O) from the saved LSE.  Returns (dq, dk, dv)."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do)):
        _check_bhnd(name, t, q.shape, q.dtype)
    _check_lse(lse, B, H, N)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape, q.dtype)
    ws = _workspace(q, workspace)
    _call("attn_bwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
          _default_scale(d, scale), int(bool(causal)), _dtype_code(q), ws.data_ptr(), _nbytes(ws),
          _stream(stream))
    return dq, dk, dv


def attn_bwd_preprocess(o, lse, do, workspace, stream=None):
    """Phase 1 of the BF16 backward (delta, LSE*log2(e), zeroed dQ accumulator)."""
    B, H, N, d = o.shape
    _call("attn_bwd_preprocess", o.data_ptr(), lse.data_ptr(), do.data_ptr(), B, H, N, d,
          _dtype_code(o), workspace.data_ptr(), _nbytes(workspace), _stream(stream))


def attn_bwd_main(q, k, v, do, dk, dv, workspace, scale=None, causal=False, stream=None):
    """Phase 2 of the BF16 backward (dK, dV and the dQ accumulation)."""
    B, H, N, d = q.shape
    _call("attn_bwd_main", q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
          dk.data_ptr(), dv.data_ptr(), B, H, N, d, _default_scale(d, scale), int(bool(causal)),
          _dtype_code(q), workspace.data_ptr(), _nbytes(workspace), _stream(stream))


def attn_bwd_dq_convert(dq, workspace, scale=None, stream=None):
    """Phase 3 of the BF16 backward (dQ = bf16(scale * accumulator))."""
    B, H, N, d = dq.shape
    _call("attn_bwd_dq_convert", dq.data_ptr(), B, H, N, d, _default_scale(d, scale),
          _dtype_code(dq), workspace.data_ptr(), _nbytes(workspace), _stream(stream))


def attn_check_status(stream=None) -> None:
    """Synchronize and raise AttnError if a kernel gave up on a bounded wait."""
    _call("attn_check_status", _stream(stream))


def attn_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test kernel (see include/attn.h)."""
    _call("attn_selftest_wait_timeout", int(limit_ns), _stream(stream))


def attn_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, scale=None, causal=False, stream=None):
    """attn_bwd for callers that must not allocate device memory: BF16 only,
    outputs passed in, scratch taken from the library's fixed 32 MiB array
    (see include/attn.h for the size limit and the sharing rules)."""
    _check_bhnd("q", q, dtype=torch.bfloat16)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape, q.dtype)
    _check_lse(lse, B, H, N)
    _call("attn_bwd_noalloc", q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
          lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
          _default_scale(d, scale), int(bool(causal)), _stream(stream))
    return dq, dk, dv


# ---------------------------------------------------------------------------
# Serving: packed sequences, grouped heads, the paged INT8 cache
# ---------------------------------------------------------------------------
# include/attn.h states the layouts.  A cache is the five tensors (k_cache,
# v_cache, k_scale, v_scale, block_table).  Tensors on another device than the
# current one are refused by the library.
#
# A call on the current stream goes through the C++ binding first, which takes a
# third of the time; it returns None where something is not as it should be, and
# the function's own checks then find out what.  Its new outputs of up to 256 KB
# together share one storage.

# With another stream given, what a call allocates is that stream's memory: the
# current stream's allocator would hand it on while the kernels still use it.

# Each check first asks for everything at once, and looks for what is wrong only
# then: attribute reads are most of what a call costs on the host.

def _check_rows(name, t, shape):
    """A BF16 CUDA tensor of this shape whose rows of d elements are contiguous."""
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is torch.bfloat16 and t.is_cuda and t.stride(-1) == 1:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows (last stride 1)")


def _check_packed_rows(name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a tensor [T, heads, d]")
    _check_rows(name, t, t.shape)


def _check_dense(name, t, shape, dtype):
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {list(shape)}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")


def _check_ints(name, t, n=None):
    if (type(t) is torch.Tensor and t.dtype is torch.int32 and t.is_cuda and t.dim() == 1 and t.is_contiguous()
            and (n is None or t.shape[0] == n)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if (not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous()
            or (n is not None and t.shape[0] != n)):
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor" + (f" [{n}]" if n is not None else ""))


def _check_cache(k_cache, v_cache, k_scale, v_scale, block_table):
    """Shape of the cache: (B, pages, H_kv, page_size, d, max_blocks)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor [pages, H_kv, page_size, d]")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [B, max_blocks]")
    shape = k_cache.shape
    pages, hk, page, d = shape
    _check_dense("k_cache", k_cache, shape, torch.int8)
    _check_dense("v_cache", v_cache, shape, torch.int8)
    _check_dense("k_scale", k_scale, (pages, hk), torch.float32)
    _check_dense("v_scale", v_scale, (pages, hk), torch.float32)
    B, blocks = block_table.shape
    _check_dense("block_table", block_table, (B, blocks), torch.int32)
    return B, pages, hk, page, d, blocks


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def attn_varlen_plan_bytes(B: int, T: int, H: int, H_kv: int) -> int:
    return int(load_library().attn_varlen_plan_bytes(B, T, H, H_kv))


def attn_varlen_plan(cu_seqlens, T, H, H_kv, causal=True, plan=None, stream=None):
    """The work list of attn_varlen_fwd for a packed batch: cu_seqlens int32 [B+1] on
    the device.  Returns a uint8 tensor that serves every call on the same batch.  A plan
    passed in has attn_varlen_plan_bytes(B, T, H, H_kv) bytes: attn_varlen_fwd takes B from
    its size, and in a larger one splits fewer long prompts over an SM's two tiles."""
    _check_ints("cu_seqlens", cu_seqlens)
    B = cu_seqlens.shape[0] - 1
    if plan is None:
        plan = _empty(max(attn_varlen_plan_bytes(B, T, H, H_kv), 1), torch.uint8, cu_seqlens.device, stream)
    _call("attn_varlen_plan", cu_seqlens.data_ptr(), B, T, H, H_kv, int(bool(causal)), plan.data_ptr(),
          _nbytes(plan), _stream(stream))
    return plan


def _plan_batch(plan, T, H, H_kv):
    """Sequences a plan of this size has room for (its buffer grows by 16 bytes each)."""
    if not isinstance(plan, torch.Tensor) or not plan.is_cuda or not plan.is_contiguous():
        raise ValueError("plan must be a tensor made by attn_varlen_plan")
    B = (_nbytes(plan) - 256) // 16 - T // (128 // max(1, min(128, H // H_kv)))
    if B < 1:
        raise ValueError("plan is too small for this T, H and H_kv")
    return B


def attn_varlen_fwd(q, k, v, plan, scale=None, causal=True, o=None, lse=None, stream=None):
    """Attention over packed prompts: q [T,H,d], k, v [T,H_kv,d] BF16 (rows contiguous,
    token and head strides free), plan of attn_varlen_plan.  Returns (o [T,H,d], lse [T,H]);
    rows that belong to no sequence are left as they are."""
    if stream is None:
        done = (_BINDING or _binding()).varlen_fwd(q, k, v, plan, scale, causal, o, lse)
        if done is not None:
            return done
    _check_packed_rows("q", q)
    _check_packed_rows("k", k)
    T, H, d = q.shape
    hk = k.shape[1]
    _check_rows("k", k, (T, hk, d))
    _check_rows("v", v, (T, hk, d))
    if hk < 1 or H < 1 or H % hk:
        raise ValueError(f"H = {H} is not a multiple of H_kv = {hk}")
    if o is None:
        o = _empty((T, H, d), q.dtype, q.device, stream)
    else:
        _check_dense("o", o, (T, H, d), torch.bfloat16)
    if lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    else:
        _check_dense("lse", lse, (T, H), torch.float32)
    B = _plan_batch(plan, T, H, hk)
    _call("attn_varlen_fwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), q.stride(1),
          k.stride(0), k.stride(1), v.stride(0), v.stride(1), plan.data_ptr(), _nbytes(plan),
          o.data_ptr(), lse.data_ptr(), B, T, H, hk, d, _default_scale(d, scale), int(bool(causal)),
          _stream(stream))
    return o, lse


def attn_cache_append_int8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, starts,
                           stream=None):
    """Write the packed rows k, v [T,H_kv,d] BF16 behind the starts[b] positions that every
    sequence holds (see include/attn.h for the scales' rule).  Returns (k_cache, v_cache)."""
    if stream is None:
        done = (_BINDING or _binding()).cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table,
                                                     cu_seqlens, starts)
        if done is not None:
            return done
    B, pages, hk, page, d, blocks = _check_cache(k_cache, v_cache, k_scale, v_scale, block_table)
    _check_packed_rows("k", k)
    T = k.shape[0]
    _check_rows("k", k, (T, hk, d))
    _check_rows("v", v, (T, hk, d))
    _check_ints("cu_seqlens", cu_seqlens, B + 1)
    _check_ints("starts", starts, B)
    _call("attn_cache_append_int8", k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0),
          v.stride(1), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
          block_table.data_ptr(), cu_seqlens.data_ptr(), starts.data_ptr(), B, T, hk, d, pages, page,
          blocks, _stream(stream))
    return k_cache, v_cache


def attn_cache_read_int8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, starts, T,
                         dtype=torch.bfloat16, k=None, v=None, stream=None):
    """Values of positions starts[b] .. of every sequence, packed as cu_seqlens says (T tokens in
    all), in dtype bfloat16 or float32.  Returns (k, v) [T,H_kv,d]."""
    if stream is None:
        done = (_BINDING or _binding()).cache_read(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                                                   starts, T, dtype, k, v)
        if done is not None:
            return done
    B, pages, hk, page, d, blocks = _check_cache(k_cache, v_cache, k_scale, v_scale, block_table)
    _check_ints("cu_seqlens", cu_seqlens, B + 1)
    _check_ints("starts", starts, B)
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    if k is None:
        k = _empty((T, hk, d), dtype, k_cache.device, stream)
    else:
        _check_dense("k", k, (T, hk, d), dtype)
    if v is None:
        v = _empty((T, hk, d), dtype, k_cache.device, stream)
    else:
        _check_dense("v", v, (T, hk, d), dtype)
    _call("attn_cache_read_int8", k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), starts.data_ptr(),
          k.data_ptr(), v.data_ptr(), B, T, hk, d, pages, page, blocks, _dtype_code(k), _stream(stream))
    return k, v


def attn_decode_int8_workspace_bytes(B: int, n_q: int, H: int, H_kv: int, d: int, page_size: int,
                                     max_blocks: int) -> int:
    return int(load_library().attn_decode_int8_workspace_bytes(B, n_q, H, H_kv, d, page_size, max_blocks))


def attn_decode_int8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, scale=None, o=None,
                     lse=None, workspace=None, stream=None):
    """Attention of the newest n_q tokens q [B,n_q,H,d] BF16 over the cache; seqlens int32 [B]
    counts them in.  Returns (o [B,n_q,H,d], lse [B,n_q,H])."""
    if stream is None:
        done = (_BINDING or _binding()).decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, scale, o,
                                               lse, workspace)
        if done is not None:
            return done
    B, pages, hk, page, d, blocks = _check_cache(k_cache, v_cache, k_scale, v_scale, block_table)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor [B, n_q, H, d]")
    n_q, H = q.shape[1], q.shape[2]
    _check_rows("q", q, (B, n_q, H, d))
    _check_ints("seqlens", seqlens, B)
    if o is None:
        o = _empty((B, n_q, H, d), q.dtype, q.device, stream)
    else:
        _check_dense("o", o, (B, n_q, H, d), torch.bfloat16)
    if lse is None:
        lse = _empty((B, n_q, H), torch.float32, q.device, stream)
    else:
        _check_dense("lse", lse, (B, n_q, H), torch.float32)
    if workspace is None:
        need = attn_decode_int8_workspace_bytes(B, n_q, H, hk, d, page, blocks)
        workspace = _empty(max(need, 1), torch.uint8, q.device, stream)
    _call("attn_decode_int8", q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
          seqlens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, n_q, H, hk, d, pages, page, blocks,
          _default_scale(d, scale), workspace.data_ptr(), _nbytes(workspace), _stream(stream))
    return o, lse
