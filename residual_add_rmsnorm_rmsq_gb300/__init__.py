"""Python binding of librmsq (fused residual-add + RMSNorm + FP8 / NVFP4 quantisation).

Argument marshalling only: every step of the op runs in the library's CUDA
kernels.  torch is used for device memory and streams.  The names follow the C
ABI in ``include/rmsq.h``; if the built library is missing this module raises
instead of computing anything another way.

``stream`` (a torch stream or a raw handle; None: the current one) is where a
call launches.  As with any work on a side stream, ordering it after the
producers of its inputs and before the consumers of its outputs is the
caller's.  What a call allocates itself, its missing outputs and its workspace,
comes from the launching stream's memory, and the outputs are kept until the
stream that was current at the call is done with them too: neither can meet
memory that work on the other stream still uses.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "librmsq.so")

# rmsq_status
OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_ALIAS, ERR_UNSUPPORTED_SHAPE, \
    ERR_UNSUPPORTED_DEVICE, ERR_NO_DEVICE, ERR_CUDA = range(8)

# rmsq_quant_mode
MODES = {
    "fp8_static": 0,
    "fp8_per_token": 1,
    "fp8_group128_row": 2,
    "fp8_group128_col": 3,
    "fp8_group64_row": 4,
    "fp8_group64_col": 5,
    "nvfp4": 6,
}
# Scale options (RMSQ_QUANT_E8M0, RMSQ_QUANT_TMA_ALIGNED, RMSQ_QUANT_UE8M0),
# appended to a mode name with "+": e.g. "fp8_group128_col+e8m0+tma",
# "fp8_per_token+ue8m0".
OPTIONS = {"e8m0": 0x10, "tma": 0x20, "ue8m0": 0x40}


@functools.lru_cache(maxsize=None)
def mode_code(mode: str) -> int:
    """The C quant_mode argument for a mode name with optional "+e8m0" / "+tma"."""
    base, *opts = mode.split("+")
    if base not in MODES or any(o not in OPTIONS for o in opts):
        raise ValueError(f"unknown quant mode {mode!r}")
    return MODES[base] | sum(OPTIONS[o] for o in opts)


def _variant(variant: str) -> int:
    if variant not in VARIANTS:
        raise ValueError(f"unknown variant {variant!r} (one of {', '.join(VARIANTS)})")
    return VARIANTS[variant]


# rmsq_dtype
DTYPES = {torch.bfloat16: 0, torch.float16: 1}
MAX_HIDDEN = 16384

VARIANTS = {"auto": 0, "direct": 1, "pipelined": 2}

EXPORTS = ("rmsq_fused_add_rmsnorm_quant", "rmsq_fused_add_rmsnorm_quant_ex",
           "rmsq_fused_add_rmsnorm_nvfp4_dynamic", "rmsq_nvfp4_dynamic_workspace_bytes",
           "rmsq_fused_add_rmsnorm_nvfp4_dynamic_noalloc", "rmsq_silu_mul_quant",
           "rmsq_fused_add_rmsnorm", "rmsq_quant", "rmsq_qk_norm_rope", "rmsq_qk_norm_rope_ex",
           "rmsq_qk_norm_mrope",
           "rmsq_allreduce_add_rmsnorm_quant",
           "rmsq_build_slot_map", "rmsq_kv_cache_store_nvfp4", "rmsq_kv_cache_load_nvfp4",
           "rmsq_paged_attention_nvfp4", "rmsq_paged_attention_nvfp4_ex", "rmsq_paged_attention_workspace_bytes",
           "rmsq_kv_cache_store_fp8", "rmsq_kv_cache_load_fp8", "rmsq_paged_attention_fp8",
           "rmsq_fp8_block_matmul",
           "rmsq_set_pipeline_config", "rmsq_set_programmatic_launch", "rmsq_take_fault_flags",
           "rmsq_query_sizes", "rmsq_query_launch", "rmsq_debug_convert", "rmsq_debug_activation", "rmsq_debug_bounded_wait",
           "rmsq_status_string", "rmsq_last_cuda_error", "rmsq_version")


class RmsqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = status_string(status) if _lib is not None else str(status)
        if status == ERR_CUDA and _lib is not None:
            msg += f" (cudaError {_lib.rmsq_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [status {status}]")


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load librmsq.so (built by ``residual_add_rmsnorm_rmsq_gb300._build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"librmsq.so not built ({p}); run residual_add_rmsnorm_rmsq_gb300._build.build()")
        L = ctypes.CDLL(p)
        vp, i64, f32, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        L.rmsq_fused_add_rmsnorm_quant.argtypes = [vp, vp, vp, f32, ci, vp, vp, vp, vp, i64, i64, ci, vp]
        L.rmsq_fused_add_rmsnorm_quant.restype = ci
        L.rmsq_fused_add_rmsnorm_quant_ex.argtypes = [vp, vp, vp, f32, ci, vp, vp, vp, vp, i64, i64, ci,
                                                      vp, ci]
        L.rmsq_fused_add_rmsnorm_quant_ex.restype = ci
        L.rmsq_fused_add_rmsnorm_nvfp4_dynamic.argtypes = [vp, vp, vp, f32, vp, vp, vp, vp, vp,
                                                           ctypes.c_size_t, i64, i64, ci, vp, ci]
        L.rmsq_fused_add_rmsnorm_nvfp4_dynamic.restype = ci
        L.rmsq_nvfp4_dynamic_workspace_bytes.argtypes = [i64]
        L.rmsq_nvfp4_dynamic_workspace_bytes.restype = ctypes.c_size_t
        L.rmsq_fused_add_rmsnorm.argtypes = [vp, vp, vp, f32, vp, vp, i64, i64, ci, vp]
        L.rmsq_fused_add_rmsnorm.restype = ci
        L.rmsq_qk_norm_rope.argtypes = [vp, vp, vp, i64, vp, vp, f32, i64, ci, ci, ci, ci, ci, vp]
        L.rmsq_qk_norm_rope.restype = ci
        L.rmsq_qk_norm_rope_ex.argtypes = [vp, vp, vp, i64, vp, vp, f32, i64, ci, ci, ci, ci, ci, vp, ci]
        L.rmsq_qk_norm_rope_ex.restype = ci
        L.rmsq_qk_norm_mrope.argtypes = [vp, vp, vp, vp, i64, vp, vp, f32, i64, ci, ci, ci, ci, ci, ci, ci, ci, ci, vp, ci]
        L.rmsq_qk_norm_mrope.restype = ci
        L.rmsq_allreduce_add_rmsnorm_quant.argtypes = [ctypes.POINTER(vp), ci, vp, vp, f32, ci, vp, vp, vp, vp,
                                                       i64, i64, ci, vp]
        L.rmsq_allreduce_add_rmsnorm_quant.restype = ci
        L.rmsq_build_slot_map.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        L.rmsq_build_slot_map.restype = ci
        L.rmsq_kv_cache_store_nvfp4.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, vp]
        L.rmsq_kv_cache_store_nvfp4.restype = ci
        L.rmsq_kv_cache_load_nvfp4.argtypes = [vp, i64, i64, vp, vp, vp, vp, i64, vp, i64, i64, ci, ci, ci, vp]
        L.rmsq_kv_cache_load_nvfp4.restype = ci
        L.rmsq_kv_cache_store_fp8.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, ci, ci, ci, vp]
        L.rmsq_kv_cache_store_fp8.restype = ci
        L.rmsq_kv_cache_load_fp8.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, i64, i64, ci, ci, ci, vp]
        L.rmsq_kv_cache_load_fp8.restype = ci
        L.rmsq_paged_attention_nvfp4.argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, vp, vp, vp, f32, i64, vp, vp, vp,
                                                 ctypes.c_size_t, i64, i64, ci, ci, ci, ci, vp, ci]
        L.rmsq_paged_attention_nvfp4.restype = ci
        L.rmsq_paged_attention_nvfp4_ex.argtypes = L.rmsq_paged_attention_nvfp4.argtypes + [i64]
        L.rmsq_paged_attention_nvfp4_ex.restype = ci
        L.rmsq_paged_attention_fp8.argtypes = [vp, i64, vp, vp, i64, i64, vp, i64, vp, vp, f32, i64, vp, vp, vp,
                                               ctypes.c_size_t, i64, i64, ci, ci, ci, ci, vp, ci, i64]
        L.rmsq_paged_attention_fp8.restype = ci
        L.rmsq_paged_attention_workspace_bytes.argtypes = [i64, i64, ci, ci, ci]
        L.rmsq_paged_attention_workspace_bytes.restype = ctypes.c_size_t
        L.rmsq_fp8_block_matmul.argtypes = [vp, vp, ci, vp, vp, vp, i64, i64, i64, ci, vp]
        L.rmsq_fp8_block_matmul.restype = ci
        L.rmsq_quant.argtypes = [vp, ci, vp, vp, vp, i64, i64, ci, vp]
        L.rmsq_quant.restype = ci
        L.rmsq_silu_mul_quant.argtypes = [vp, ci, vp, vp, vp, i64, i64, ci, vp]
        L.rmsq_silu_mul_quant.restype = ci
        L.rmsq_set_pipeline_config.argtypes = [ci, ci, ci, ci]
        L.rmsq_set_pipeline_config.restype = ci
        L.rmsq_set_programmatic_launch.argtypes = [ci]
        L.rmsq_set_programmatic_launch.restype = ci
        L.rmsq_take_fault_flags.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        L.rmsq_take_fault_flags.restype = ci
        L.rmsq_query_sizes.argtypes = [ci, i64, i64, ctypes.POINTER(ctypes.c_size_t),
                                       ctypes.POINTER(ctypes.c_size_t)]
        L.rmsq_query_sizes.restype = ci
        L.rmsq_query_launch.argtypes = [ci, i64, i64, ci, ci, ci, ctypes.POINTER(ctypes.c_int32)]
        L.rmsq_query_launch.restype = ci
        L.rmsq_debug_convert.argtypes = [ci, vp, vp, i64, vp]
        L.rmsq_debug_convert.restype = ci
        L.rmsq_debug_activation.argtypes = [ci, vp, vp, vp, i64, vp]
        L.rmsq_debug_activation.restype = ci
        L.rmsq_debug_bounded_wait.argtypes = [i64, ctypes.POINTER(ci)]
        L.rmsq_debug_bounded_wait.restype = ci
        L.rmsq_status_string.argtypes = [ci]
        L.rmsq_status_string.restype = ctypes.c_char_p
        L.rmsq_last_cuda_error.argtypes = []
        L.rmsq_last_cuda_error.restype = ci
        L.rmsq_version.argtypes = []
        L.rmsq_version.restype = ci
        _lib = L
        return L


def status_string(status: int) -> str:
    return load().rmsq_status_string(int(status)).decode()


def version() -> int:
    return load().rmsq_version()


def query_sizes(mode: str, n_tokens: int, hidden: int) -> tuple[int, int]:
    q, s = ctypes.c_size_t(), ctypes.c_size_t()
    st = load().rmsq_query_sizes(mode_code(mode), n_tokens, hidden, ctypes.byref(q), ctypes.byref(s))
    if st:
        raise RmsqError(st, "rmsq_query_sizes")
    return q.value, s.value


def _p(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object for it (0.1
# instead of 2.9 us a call on the Grace host); the public way where a torch
# build lacks the function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int = -1) -> int:
    """The handle of `stream`, or of the current one of `device` (of the
    current device if that is not known)."""
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(device if device >= 0 else torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """A context in which `stream` is the current one; None where it is already."""
    if stream is None or not torch.cuda.is_initialized():
        return None
    if not hasattr(stream, "cuda_stream"):      # a handle; 0 and 1 are the default stream
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) > 1 else torch.cuda.default_stream()
    if stream.cuda_stream == torch.cuda.current_stream(stream.device).cuda_stream:
        return None
    return torch.cuda.stream(stream)


def _empty_on(stream, *size, **kwargs) -> torch.Tensor:
    """torch.empty for a launch on `stream`: from that stream's memory.  The
    current stream's may have been let go while work there still uses it (the
    workspace of the call before, say), and nothing orders the launch after
    that work.  The current stream may read the result, so the memory is kept
    until it is done too."""
    on = _on(stream)
    if on is None:
        return torch.empty(*size, **kwargs)
    with on:
        t = torch.empty(*size, **kwargs)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty_for(stream):
    return torch.empty if stream is None else functools.partial(_empty_on, stream)


def scales_like(mode: str, n_tokens: int, hidden: int, device) -> torch.Tensor | None:
    """An output tensor of the right shape and dtype for the scales of ``mode``
    (column-major with "+tma": [hidden/G, n_tokens rounded up to 16 bytes of
    scales]; uint8 with "+ue8m0")."""
    return _scales_like(mode, n_tokens, hidden, device, torch.empty)


def _scales_like(mode, n_tokens, hidden, device, empty):
    base, *opts = mode.split("+")
    if base == "fp8_static":
        return None
    if base == "nvfp4":
        return empty(n_tokens, hidden // 16, dtype=torch.uint8, device=device)
    dt = torch.uint8 if "ue8m0" in opts else torch.float32
    if base == "fp8_per_token":
        return empty(n_tokens, dtype=dt, device=device)
    G = 128 if "128" in base else 64
    per16 = 16 if "ue8m0" in opts else 4
    cols = (n_tokens + per16 - 1) // per16 * per16 if "tma" in opts else n_tokens
    shape = (hidden // G, cols) if base.endswith("_col") else (n_tokens, hidden // G)
    return empty(shape, dtype=dt, device=device)


def fused_add_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor,
                            eps: float, mode: str, scale_in: torch.Tensor | None = None, *,
                            out_q: torch.Tensor | None = None,
                            out_scales: torch.Tensor | None = None,
                            residual_out: torch.Tensor | None = None, stream=None,
                            variant: str = "auto"):
    """rmsq_fused_add_rmsnorm_quant on torch CUDA tensors.

    x, residual, residual_out: [n, H] bf16/fp16, contiguous; weight: [H];
    scale_in: fp32 device tensor with one element (FP8 static scale / NVFP4
    global scale).  Missing outputs are allocated.  Pass
    ``residual_out=residual`` for the in-place update.
    ``variant``: "auto", "direct" or "pipelined" (identical results).
    Returns (q, scales, residual_out).
    """
    vcode = _variant(variant)
    L, empty = load(), _empty_for(stream)
    n, H = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {x.dtype}")
    for t in (x, residual, weight, residual_out, out_q, out_scales, scale_in):
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if out_q is None:
        width = H // 2 if mode == "nvfp4" else H
        out_q = empty(n, width, dtype=torch.uint8, device=x.device)
    if out_scales is None:
        out_scales = _scales_like(mode, n, H, x.device, empty)
    if residual is not None and residual_out is None:
        residual_out = empty(residual.shape, dtype=residual.dtype, device=residual.device)
    st = L.rmsq_fused_add_rmsnorm_quant_ex(_p(x), _p(residual), _p(weight), ctypes.c_float(eps),
                                           mode_code(mode), _p(scale_in), _p(out_q), _p(out_scales),
                                           _p(residual_out), n, H, DTYPES[x.dtype], _stream(stream),
                                           vcode)
    if st:
        raise RmsqError(st, "rmsq_fused_add_rmsnorm_quant")
    return out_q, out_scales, residual_out


MAX_ALLREDUCE_RANKS = 8


def allreduce_add_rmsnorm_quant(partials, residual: torch.Tensor | None, weight: torch.Tensor, eps: float,
                                mode: str, scale_in: torch.Tensor | None = None, *,
                                out_q: torch.Tensor | None = None, out_scales: torch.Tensor | None = None,
                                residual_out: torch.Tensor | None = None, stream=None):
    """rmsq_allreduce_add_rmsnorm_quant: ``partials`` is a sequence of [n, H]
    tensors, one per rank (each readable by the current device), summed in
    rank order; then the fused op on the sum.  Returns (q, scales, residual_out)."""
    L, empty = load(), _empty_for(stream)
    parts = list(partials)
    if not 1 <= len(parts) <= MAX_ALLREDUCE_RANKS:
        raise ValueError(f"1 to {MAX_ALLREDUCE_RANKS} partial tensors")
    x = parts[0]
    n, H = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {x.dtype}")
    for t in parts:
        if t.shape != x.shape or t.dtype != x.dtype:
            raise ValueError("every partial must have the first one's shape and dtype")
    for t in parts + [residual, weight, residual_out, out_q, out_scales, scale_in]:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if out_q is None:
        width = H // 2 if mode == "nvfp4" else H
        out_q = empty(n, width, dtype=torch.uint8, device=x.device)
    if out_scales is None:
        out_scales = _scales_like(mode, n, H, x.device, empty)
    if residual is not None and residual_out is None:
        residual_out = empty(residual.shape, dtype=residual.dtype, device=residual.device)
    arr = (ctypes.c_void_p * len(parts))(*[t.data_ptr() for t in parts])
    st = L.rmsq_allreduce_add_rmsnorm_quant(arr, len(parts), _p(residual), _p(weight), ctypes.c_float(eps),
                                            mode_code(mode), _p(scale_in), _p(out_q), _p(out_scales),
                                            _p(residual_out), n, H, DTYPES[x.dtype], _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_allreduce_add_rmsnorm_quant")
    return out_q, out_scales, residual_out


def row_slice(n_tokens: int, world: int, rank: int) -> tuple[int, int]:
    """Rows [begin, end) of `rank` when `world` ranks split a batch for a
    two-shot all-reduce + norm (each rank reduces and normalises its slice,
    then the slices are gathered): contiguous, as equal as possible, the
    first n % world ranks one row longer."""
    if world < 1 or not 0 <= rank < world or n_tokens < 0:
        raise ValueError("bad world / rank / n_tokens")
    q, r = divmod(n_tokens, world)
    begin = rank * q + min(rank, r)
    return begin, begin + q + (1 if rank < r else 0)


def fused_add_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor, eps: float, *,
                      y_out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None, stream=None):
    """rmsq_fused_add_rmsnorm: the norm alone, y in the activation type.
    Returns (y, residual_out)."""
    L, empty = load(), _empty_for(stream)
    n, H = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {x.dtype}")
    for t in (x, residual, weight, y_out, residual_out):
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if y_out is None:
        y_out = empty(x.shape, dtype=x.dtype, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = empty(residual.shape, dtype=residual.dtype, device=residual.device)
    st = L.rmsq_fused_add_rmsnorm(_p(x), _p(residual), _p(weight), ctypes.c_float(eps), _p(y_out), _p(residual_out),
                                  n, H, DTYPES[x.dtype], _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_fused_add_rmsnorm")
    return y_out, residual_out


def quant(y: torch.Tensor, mode: str, scale_in: torch.Tensor | None = None, *, out_q: torch.Tensor | None = None,
          out_scales: torch.Tensor | None = None, stream=None):
    """rmsq_quant: the quantisation of a [n, H] activation-type tensor.
    Returns (q, scales)."""
    L, empty = load(), _empty_for(stream)
    n, H = y.shape
    if y.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {y.dtype}")
    for t in (y, out_q, out_scales, scale_in):
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if out_q is None:
        width = H // 2 if mode == "nvfp4" else H
        out_q = empty(n, width, dtype=torch.uint8, device=y.device)
    if out_scales is None:
        out_scales = _scales_like(mode, n, H, y.device, empty)
    st = L.rmsq_quant(_p(y), mode_code(mode), _p(scale_in), _p(out_q), _p(out_scales), n, H, DTYPES[y.dtype],
                      _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_quant")
    return out_q, out_scales


def qk_norm_rope(qkv: torch.Tensor, positions: torch.Tensor, cos_sin_cache: torch.Tensor, q_weight: torch.Tensor,
                 k_weight: torch.Tensor, eps: float, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 is_neox: bool = True, stream=None, variant: str = "auto") -> torch.Tensor:
    """rmsq_qk_norm_rope_ex on torch CUDA tensors, in place on qkv (returned);
    variant "auto", "direct" or "pipelined" (bit-identical results)."""
    vcode = _variant(variant)
    L = load()
    if qkv.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {qkv.dtype}")
    for t in (qkv, positions, cos_sin_cache, q_weight, k_weight):
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if positions.dtype != torch.int64 or cos_sin_cache.dtype != torch.float32:
        raise TypeError("positions must be int64 and cos_sin_cache float32")
    n = qkv.shape[0]
    st = L.rmsq_qk_norm_rope_ex(_p(qkv), _p(positions), _p(cos_sin_cache), cos_sin_cache.shape[0],
                                _p(q_weight), _p(k_weight), ctypes.c_float(eps), n, num_q_heads, num_kv_heads,
                                head_dim, 1 if is_neox else 0, DTYPES[qkv.dtype], _stream(stream),
                                vcode)
    if st:
        raise RmsqError(st, "rmsq_qk_norm_rope_ex")
    return qkv


def _check_tensors(named, dtypes) -> None:
    """Every tensor of `named` (name -> tensor) on one device, the current one
    if it is a CUDA device, and of the type `dtypes` says for its name."""
    device = None
    for name, t in named.items():
        if t is None:
            continue
        if t.dtype != dtypes[name]:
            raise TypeError(f"{name} must be {dtypes[name]}, got {t.dtype}")
        if device is None:
            device = t.device
            if device.type == "cuda":
                if device.index != torch.cuda.current_device():
                    raise ValueError(f"{name} is on {device}, not on the current device")
            elif torch.cuda.is_available():
                raise ValueError(f"{name} must be a CUDA tensor")
        elif t.device != device:
            raise ValueError(f"{name} is on {t.device}, the others on {device}")


def _fits(t: torch.Tensor, dtype: torch.dtype, device: int, shape: tuple) -> bool:
    """The checks below in one go, for the path without an error."""
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _is_current(device: int) -> bool:
    return device >= 0 and device == torch.cuda.current_device()


def _want_shape(name: str, t: torch.Tensor, *shape) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _token_rows(name: str, t: torch.Tensor) -> int:
    """The token stride of a [n, heads, D] tensor whose heads are contiguous."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    per_token, per_head, per_element = t.stride()
    if (per_element != 1 and d > 1) or (per_head != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return per_token if n > 1 else h * d


def qk_norm_mrope(qkv: torch.Tensor, positions: torch.Tensor, cos_sin_cache: torch.Tensor,
                  q_weight: torch.Tensor | None, k_weight: torch.Tensor | None, eps: float, num_q_heads: int,
                  num_kv_heads: int, head_dim: int, sections, is_neox: bool = True, *, interleaved: bool = False,
                  out: torch.Tensor | None = None, stream=None, variant: str = "auto") -> torch.Tensor:
    """rmsq_qk_norm_mrope: QK-norm + RoPE with three positions per token.

    qkv [n, (q heads + 2 kv heads) D]; positions int64 [3, n] (time, height,
    width); sections: the number of angles of each axis, together D / 2, one
    after the other or (interleaved) alternating.  q_weight and k_weight None:
    no norm.  In place on qkv, or with `out` [n, (q heads + kv heads) D] there.
    Returns where the heads are.  variant "auto", "direct" or "pipelined"
    (bit-identical results).
    """
    vcode = _variant(variant)
    L = load()
    dt = _act_types(qkv)
    t, h, w = (int(s) for s in sections)
    n = qkv.shape[0]
    width = (num_q_heads + 2 * num_kv_heads) * head_dim
    i = qkv.get_device()
    given = {"qkv": qkv, "positions": positions, "cos_sin_cache": cos_sin_cache, "q_weight": q_weight,
             "k_weight": k_weight, "out": out}
    _check_tensors(given, {"qkv": dt, "positions": _I64, "cos_sin_cache": _F32, "q_weight": dt, "k_weight": dt, "out": dt})
    _want_shape("qkv", qkv, n, width)
    _want_shape("positions", positions, 3, n)
    _want_shape("cos_sin_cache", cos_sin_cache, cos_sin_cache.shape[0], head_dim)
    for name, t_ in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t_ is not None:
            _want_shape(name, t_, head_dim)
    if out is not None:
        _want_shape("out", out, n, width - num_kv_heads * head_dim)
    st = L.rmsq_qk_norm_mrope(qkv.data_ptr(), _p(out), positions.data_ptr(), cos_sin_cache.data_ptr(),
                              cos_sin_cache.shape[0], _p(q_weight), _p(k_weight), eps, n, num_q_heads, num_kv_heads,
                              head_dim, t, h, w, 1 if interleaved else 0, 1 if is_neox else 0, DTYPES[dt],
                              _stream(stream, i), vcode)
    if st:
        raise RmsqError(st, "rmsq_qk_norm_mrope")
    return qkv if out is None else out


_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8
_SLOT_TYPES = {"context_lens": _I32, "query_lens": _I32, "block_table": _I32, "free_pages": _I32, "num_free": _I32,
               "slot_map": _I64, "positions": _I64, "query_start": _I32, "seq_lens": _I32, "num_free_out": _I32,
               "status": _I32}
SLOT_NO_PAGES, SLOT_TABLE_FULL, SLOT_TOO_MANY_TOKENS, SLOT_BAD_LENGTH = 1, 2, 4, 8
MAX_REQUESTS = 8192


def build_slot_map(context_lens: torch.Tensor, query_lens: torch.Tensor, block_table: torch.Tensor,
                   free_pages: torch.Tensor, num_free: torch.Tensor, page_size: int, max_tokens: int, *,
                   slot_map: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                   query_start: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                   num_free_out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """rmsq_build_slot_map: pages, slots and positions of a step's new tokens.

    context_lens, query_lens: int32 [R]; block_table: int32 [R, width], updated
    in place; free_pages: int32 [capacity]; num_free: int32 [1].  Missing
    outputs are allocated.  Returns (slot_map [max_tokens], positions
    [max_tokens], query_start [R + 1], seq_lens [R], num_free_out [1],
    status [1]); status holds SLOT_* bits, 0 when the pages were assigned.
    """
    L, empty = load(), _empty_for(stream)
    R, width = block_table.shape
    dev, i = block_table.device, block_table.get_device()
    if slot_map is None:
        slot_map = empty(max(max_tokens, 0), dtype=_I64, device=dev)
    if positions is None:
        positions = empty(max(max_tokens, 0), dtype=_I64, device=dev)
    if query_start is None:
        query_start = empty(R + 1, dtype=_I32, device=dev)
    if seq_lens is None:
        seq_lens = empty(R, dtype=_I32, device=dev)
    if num_free_out is None:
        num_free_out = empty(1, dtype=_I32, device=dev)
    if status is None:
        status = empty(1, dtype=_I32, device=dev)
    per_r, one, per_t, capacity = (R,), (1,), (max_tokens,), free_pages.shape
    if not (_is_current(i) and _fits(context_lens, _I32, i, per_r) and _fits(query_lens, _I32, i, per_r) and
            _fits(block_table, _I32, i, (R, width)) and _fits(free_pages, _I32, i, capacity) and
            _fits(num_free, _I32, i, one) and _fits(slot_map, _I64, i, per_t) and _fits(positions, _I64, i, per_t) and
            _fits(query_start, _I32, i, (R + 1,)) and _fits(seq_lens, _I32, i, per_r) and
            _fits(num_free_out, _I32, i, one) and _fits(status, _I32, i, one) and len(capacity) == 1):
        given = {"context_lens": context_lens, "query_lens": query_lens, "block_table": block_table,
                 "free_pages": free_pages, "num_free": num_free, "slot_map": slot_map, "positions": positions,
                 "query_start": query_start, "seq_lens": seq_lens, "num_free_out": num_free_out, "status": status}
        _check_tensors(given, _SLOT_TYPES)
        sizes = {"context_lens": per_r, "query_lens": per_r, "block_table": (R, width),
                 "free_pages": (free_pages.numel(),), "num_free": one, "slot_map": per_t, "positions": per_t,
                 "query_start": (R + 1,), "seq_lens": per_r, "num_free_out": one, "status": one}
        for name, t in given.items():
            _want_shape(name, t, *sizes[name])
    st = L.rmsq_build_slot_map(context_lens.data_ptr(), query_lens.data_ptr(), block_table.data_ptr(), width,
                               free_pages.data_ptr(), capacity[0], num_free.data_ptr(), page_size, R, max_tokens,
                               slot_map.data_ptr(), positions.data_ptr(), query_start.data_ptr(), seq_lens.data_ptr(),
                               num_free_out.data_ptr(), status.data_ptr(), _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_build_slot_map")
    return slot_map, positions, query_start, seq_lens, num_free_out, status


def kv_cache_shape(num_pages: int, num_kv_heads: int, head_dim: int, page_size: int) -> tuple[int, int, int, int]:
    """Shape of the uint8 tensor that holds a paged NVFP4 cache."""
    return num_pages, 2, num_kv_heads, page_size * head_dim * 9 // 16


def _check_cache(cache: torch.Tensor, num_kv_heads: int, head_dim: int, page_size: int) -> int:
    _want_shape("cache", cache, *kv_cache_shape(cache.shape[0], num_kv_heads, head_dim, page_size))
    return cache.shape[0]


def _check_global_scales(*scales) -> None:
    for t in scales:
        if t.numel() != 1:
            raise ValueError("a global scale is one element")


def _act_types(t: torch.Tensor) -> torch.dtype:
    if t.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {t.dtype}")
    return t.dtype


def kv_cache_store_nvfp4(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_global_scale: torch.Tensor,
                         v_global_scale: torch.Tensor, cache: torch.Tensor, page_size: int, *, stream=None) -> None:
    """rmsq_kv_cache_store_nvfp4: k, v [n, kv heads, D] (token stride free, so
    slices of a qkv buffer serve) quantised into `cache` (kv_cache_shape) at
    slot_map (int64 [n]); a slot outside the cache skips its token.  The global
    scales are one-element fp32 tensors."""
    L = load()
    dt = _act_types(k)
    ks, vs = _token_rows("k", k), _token_rows("v", v)
    n, h, d = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    i, pages = cache.get_device(), cache.shape[0]
    if not (_is_current(i) and _fits(cache, _U8, i, kv_cache_shape(pages, h, d, page_size)) and
            _fits(slot_map, _I64, i, (n,)) and _fits(k_global_scale, _F32, i, (1,)) and
            _fits(v_global_scale, _F32, i, (1,)) and k.get_device() == i and v.get_device() == i and v.dtype is dt):
        _check_tensors({"k": k, "v": v, "slot_map": slot_map, "k_global_scale": k_global_scale,
                        "v_global_scale": v_global_scale, "cache": cache},
                       {"k": dt, "v": dt, "slot_map": _I64, "k_global_scale": _F32, "v_global_scale": _F32, "cache": _U8})
        _want_shape("slot_map", slot_map, n)
        _check_cache(cache, h, d, page_size)
        _check_global_scales(k_global_scale, v_global_scale)
    st = L.rmsq_kv_cache_store_nvfp4(k.data_ptr(), ks, v.data_ptr(), vs, slot_map.data_ptr(), k_global_scale.data_ptr(),
                                     v_global_scale.data_ptr(), cache.data_ptr(), pages, page_size, n, h, d, DTYPES[dt],
                                     _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_kv_cache_store_nvfp4")


def kv_cache_load_nvfp4(cache: torch.Tensor, slot_map: torch.Tensor, k_global_scale: torch.Tensor,
                        v_global_scale: torch.Tensor, head_dim: int, page_size: int, dtype: torch.dtype = torch.bfloat16, *,
                        k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """rmsq_kv_cache_load_nvfp4: the tokens at slot_map (int64 [n]) as two
    [n, kv heads, D] tensors of `dtype`; zeros for a slot outside the cache.
    Missing outputs are allocated.  Returns (k, v)."""
    L, empty = load(), _empty_for(stream)
    if dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {dtype}")
    if cache.dim() != 4:
        raise ValueError("cache must be [pages, 2, kv heads, bytes of a tile]")
    n, h = slot_map.shape[0], cache.shape[2]
    shape = (n, h, head_dim)
    ks = vs = h * head_dim
    if k_out is None:
        k_out = empty(shape, dtype=dtype, device=cache.device)
    else:
        ks = _token_rows("k_out", k_out)
    if v_out is None:
        v_out = empty(shape, dtype=dtype, device=cache.device)
    else:
        vs = _token_rows("v_out", v_out)
    i, pages = cache.get_device(), cache.shape[0]
    if not (_is_current(i) and _fits(cache, _U8, i, kv_cache_shape(pages, h, head_dim, page_size)) and
            _fits(slot_map, _I64, i, (n,)) and _fits(k_global_scale, _F32, i, (1,)) and
            _fits(v_global_scale, _F32, i, (1,)) and k_out.get_device() == i and v_out.get_device() == i and
            k_out.dtype is dtype and v_out.dtype is dtype):
        _check_tensors({"cache": cache, "slot_map": slot_map, "k_global_scale": k_global_scale,
                        "v_global_scale": v_global_scale, "k_out": k_out, "v_out": v_out},
                       {"cache": _U8, "slot_map": _I64, "k_global_scale": _F32, "v_global_scale": _F32, "k_out": dtype,
                        "v_out": dtype})
        _want_shape("slot_map", slot_map, n)
        _check_cache(cache, h, head_dim, page_size)
        _check_global_scales(k_global_scale, v_global_scale)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"outputs must have shape {shape}")
    st = L.rmsq_kv_cache_load_nvfp4(cache.data_ptr(), pages, page_size, slot_map.data_ptr(), k_global_scale.data_ptr(),
                                    v_global_scale.data_ptr(), k_out.data_ptr(), ks, v_out.data_ptr(), vs, n, h, head_dim,
                                    DTYPES[dtype], _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_kv_cache_load_nvfp4")
    return k_out, v_out


_CODE_TYPES = (torch.uint8, torch.float8_e4m3fn)


def kv_cache_shapes_fp8(num_pages: int, num_kv_heads: int, head_dim: int, page_size: int) -> tuple[tuple, tuple]:
    """Shapes of the two tensors that hold a paged FP8 cache: the codes (uint8 or
    float8_e4m3fn) and the uint8 scales of its blocks of 16 tokens."""
    return (num_pages, 2, num_kv_heads, page_size, head_dim), (num_pages, 2, num_kv_heads, page_size // 16)


def _cache_fp8(cache: torch.Tensor, scales: torch.Tensor) -> tuple[int, int, int, int]:
    """(pages, kv heads, page size, head dim) of a paged FP8 cache, whose two
    tensors have to fit each other."""
    if cache.dtype not in _CODE_TYPES:
        raise TypeError("cache must be uint8 or float8_e4m3fn")
    if cache.dim() != 5 or cache.shape[1] != 2:
        raise ValueError("cache must be [pages, 2, kv heads, page size, head_dim]")
    pages, _, h, page, d = cache.shape
    _want_shape("cache", cache, pages, 2, h, page, d)
    if scales.dtype is not _U8:
        raise TypeError(f"scales must be torch.uint8, got {scales.dtype}")
    _want_shape("scales", scales, pages, 2, h, page // 16)
    return pages, h, page, d


def kv_cache_store_fp8(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, cache: torch.Tensor,
                       scales: torch.Tensor, *, stream=None) -> None:
    """rmsq_kv_cache_store_fp8: k, v [n, kv heads, D] (token stride free, so
    slices of a qkv buffer serve) quantised into `cache` and `scales`
    (kv_cache_shapes_fp8) at slot_map (int64 [n], as build_slot_map writes it:
    the slots of a block of 16 ascend within 16 entries that are no other
    block's); a slot outside the cache skips its token, wherever it stands."""
    L = load()
    dt = _act_types(k)
    ks, vs = _token_rows("k", k), _token_rows("v", v)
    n, h, d = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    pages, heads, page, dim = _cache_fp8(cache, scales)
    if (heads, dim) != (h, d):
        raise ValueError(f"the cache has {heads} heads of {dim}, k has {h} of {d}")
    i = cache.get_device()
    if not (_is_current(i) and scales.get_device() == i and _fits(slot_map, _I64, i, (n,)) and k.get_device() == i and
            v.get_device() == i and v.dtype is dt):
        _check_tensors({"k": k, "v": v, "slot_map": slot_map, "cache": cache, "scales": scales},
                       {"k": dt, "v": dt, "slot_map": _I64, "cache": cache.dtype, "scales": _U8})
        _want_shape("slot_map", slot_map, n)
    st = L.rmsq_kv_cache_store_fp8(k.data_ptr(), ks, v.data_ptr(), vs, slot_map.data_ptr(), cache.data_ptr(),
                                   scales.data_ptr(), pages, page, n, h, d, DTYPES[dt], _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_kv_cache_store_fp8")


def kv_cache_load_fp8(cache: torch.Tensor, scales: torch.Tensor, slot_map: torch.Tensor,
                      dtype: torch.dtype = torch.bfloat16, *, k_out: torch.Tensor | None = None,
                      v_out: torch.Tensor | None = None, stream=None):
    """rmsq_kv_cache_load_fp8: the tokens at slot_map (int64 [n]) as two
    [n, kv heads, D] tensors of `dtype`; zeros for a slot outside the cache.
    Missing outputs are allocated.  Returns (k, v)."""
    L, empty = load(), _empty_for(stream)
    if dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {dtype}")
    pages, h, page, d = _cache_fp8(cache, scales)
    n = slot_map.shape[0]
    shape = (n, h, d)
    ks = vs = h * d
    if k_out is None:
        k_out = empty(shape, dtype=dtype, device=cache.device)
    else:
        ks = _token_rows("k_out", k_out)
    if v_out is None:
        v_out = empty(shape, dtype=dtype, device=cache.device)
    else:
        vs = _token_rows("v_out", v_out)
    i = cache.get_device()
    if not (_is_current(i) and scales.get_device() == i and _fits(slot_map, _I64, i, (n,)) and k_out.get_device() == i and
            v_out.get_device() == i and k_out.dtype is dtype and v_out.dtype is dtype):
        _check_tensors({"cache": cache, "scales": scales, "slot_map": slot_map, "k_out": k_out, "v_out": v_out},
                       {"cache": cache.dtype, "scales": _U8, "slot_map": _I64, "k_out": dtype, "v_out": dtype})
        _want_shape("slot_map", slot_map, n)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"outputs must have shape {shape}")
    st = L.rmsq_kv_cache_load_fp8(cache.data_ptr(), scales.data_ptr(), pages, page, slot_map.data_ptr(), k_out.data_ptr(),
                                  ks, v_out.data_ptr(), vs, n, h, d, DTYPES[dtype], _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_kv_cache_load_fp8")
    return k_out, v_out


def paged_attention_workspace_bytes(n_tokens: int, num_requests: int, num_heads: int, num_kv_heads: int,
                                    head_dim: int) -> int:
    return load().rmsq_paged_attention_workspace_bytes(n_tokens, num_requests, num_heads, num_kv_heads, head_dim)


def paged_attention_nvfp4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, query_start: torch.Tensor,
                          seq_lens: torch.Tensor, k_global_scale: torch.Tensor, v_global_scale: torch.Tensor,
                          page_size: int, softmax_scale: float | None = None, *, window: int = 0,
                          return_lse: bool = False, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None, variant: str = "auto",
                          max_query: int = 0):
    """rmsq_paged_attention_nvfp4_ex: causal attention of q [tokens, heads, D]
    (token stride free) over the paged NVFP4 cache.

    block_table: int32 [R, width]; query_start: int32 [R + 1]; seq_lens: int32
    [R], the lengths with this step's tokens, which are in the cache already.
    softmax_scale: 1 / sqrt(D) by default; window > 0 limits a query to its
    last `window` keys.  Missing outputs and the workspace are allocated (rows
    of q behind query_start[R] are not computed).  variant: "auto", "direct"
    (few queries) or "pipelined" (prompts).  max_query: the most queries any
    request has, if that is known; it lets "auto" choose better.  A launch that
    gives up waiting shows in take_fault_flags.  Returns out [tokens, heads, D], or
    (out, lse [tokens, heads] fp32) with return_lse or a given lse.
    """
    vcode = _variant(variant)
    L, empty = load(), _empty_for(stream)
    dt = _act_types(q)
    qs = _token_rows("q", q)
    n, heads, d = q.shape
    if cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("cache must be [pages, 2, kv heads, bytes of a tile], block_table [requests, width]")
    kv, (R, width) = cache.shape[2], block_table.shape
    if out is None:
        out = empty(q.shape, dtype=dt, device=q.device)
    if lse is None and return_lse:
        lse = empty((n, heads), dtype=_F32, device=q.device)
    if workspace is None:
        size = paged_attention_workspace_bytes(n, R, heads, kv, d)
        workspace = empty(size, dtype=_U8, device=q.device)
    i, pages, size = q.get_device(), cache.shape[0], workspace.numel()
    if not (_is_current(i) and _fits(cache, _U8, i, kv_cache_shape(pages, kv, d, page_size)) and
            _fits(block_table, _I32, i, (R, width)) and _fits(query_start, _I32, i, (R + 1,)) and
            _fits(seq_lens, _I32, i, (R,)) and _fits(k_global_scale, _F32, i, (1,)) and
            _fits(v_global_scale, _F32, i, (1,)) and _fits(out, dt, i, (n, heads, d)) and
            (lse is None or _fits(lse, _F32, i, (n, heads))) and _fits(workspace, _U8, i, (size,))):
        _check_tensors({"q": q, "cache": cache, "block_table": block_table, "query_start": query_start,
                        "seq_lens": seq_lens, "k_global_scale": k_global_scale, "v_global_scale": v_global_scale,
                        "out": out, "lse": lse, "workspace": workspace},
                       {"q": dt, "cache": _U8, "block_table": _I32, "query_start": _I32, "seq_lens": _I32,
                        "k_global_scale": _F32, "v_global_scale": _F32, "out": dt, "lse": _F32, "workspace": _U8})
        _check_cache(cache, kv, d, page_size)
        _want_shape("block_table", block_table, R, width)
        _want_shape("query_start", query_start, R + 1)
        _want_shape("seq_lens", seq_lens, R)
        _want_shape("out", out, n, heads, d)
        if lse is not None:
            _want_shape("lse", lse, n, heads)
        _want_shape("workspace", workspace, size)
        _check_global_scales(k_global_scale, v_global_scale)
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    st = L.rmsq_paged_attention_nvfp4_ex(q.data_ptr(), qs, cache.data_ptr(), pages, page_size, block_table.data_ptr(), width,
                                         query_start.data_ptr(), seq_lens.data_ptr(), k_global_scale.data_ptr(),
                                         v_global_scale.data_ptr(), softmax_scale, window, out.data_ptr(), _p(lse),
                                         workspace.data_ptr(), size, n, R, heads, kv, d, DTYPES[dt], _stream(stream, i),
                                         vcode, max_query)
    if st:
        raise RmsqError(st, "rmsq_paged_attention_nvfp4")
    return out if lse is None else (out, lse)


def paged_attention_fp8(q: torch.Tensor, cache: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                        query_start: torch.Tensor, seq_lens: torch.Tensor, softmax_scale: float | None = None, *,
                        window: int = 0, return_lse: bool = False, out: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                        variant: str = "auto", max_query: int = 0):
    """rmsq_paged_attention_fp8: causal attention of q [tokens, heads, D] (token
    stride free) over the paged FP8 cache (`cache` and `scales` of
    kv_cache_shapes_fp8).  Everything else as in paged_attention_nvfp4: returns
    out [tokens, heads, D], or (out, lse [tokens, heads] fp32) with return_lse or
    a given lse.
    """
    vcode = _variant(variant)
    L, empty = load(), _empty_for(stream)
    dt = _act_types(q)
    qs = _token_rows("q", q)
    n, heads, d = q.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [requests, width]")
    pages, kv, page, dim = _cache_fp8(cache, scales)
    if dim != d:
        raise ValueError(f"q has heads of {d}, the cache of {dim}")
    R, width = block_table.shape
    if out is None:
        out = empty(q.shape, dtype=dt, device=q.device)
    if lse is None and return_lse:
        lse = empty((n, heads), dtype=_F32, device=q.device)
    if workspace is None:
        workspace = empty(paged_attention_workspace_bytes(n, R, heads, kv, d), dtype=_U8, device=q.device)
    i, size = q.get_device(), workspace.numel()
    if not (_is_current(i) and cache.get_device() == i and scales.get_device() == i and
            _fits(block_table, _I32, i, (R, width)) and _fits(query_start, _I32, i, (R + 1,)) and
            _fits(seq_lens, _I32, i, (R,)) and _fits(out, dt, i, (n, heads, d)) and
            (lse is None or _fits(lse, _F32, i, (n, heads))) and _fits(workspace, _U8, i, (size,))):
        _check_tensors({"q": q, "cache": cache, "scales": scales, "block_table": block_table, "query_start": query_start,
                        "seq_lens": seq_lens, "out": out, "lse": lse, "workspace": workspace},
                       {"q": dt, "cache": cache.dtype, "scales": _U8, "block_table": _I32, "query_start": _I32,
                        "seq_lens": _I32, "out": dt, "lse": _F32, "workspace": _U8})
        _want_shape("block_table", block_table, R, width)
        _want_shape("query_start", query_start, R + 1)
        _want_shape("seq_lens", seq_lens, R)
        _want_shape("out", out, n, heads, d)
        if lse is not None:
            _want_shape("lse", lse, n, heads)
        _want_shape("workspace", workspace, size)
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    st = L.rmsq_paged_attention_fp8(q.data_ptr(), qs, cache.data_ptr(), scales.data_ptr(), pages, page,
                                    block_table.data_ptr(), width, query_start.data_ptr(), seq_lens.data_ptr(),
                                    softmax_scale, window, out.data_ptr(), _p(lse), workspace.data_ptr(), size, n, R, heads,
                                    kv, d, DTYPES[dt], _stream(stream, i), vcode, max_query)
    if st:
        raise RmsqError(st, "rmsq_paged_attention_fp8")
    return out if lse is None else (out, lse)


def fp8_block_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, mode: str, b_codes: torch.Tensor,
                     b_scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16, *, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """rmsq_fp8_block_matmul: out [m, n] = a . b^T of E4M3 codes with block scales.

    a_codes [m, k] and a_scales as fused_add_rmsnorm_quant or silu_mul_quant
    return them for `mode` ("fp8_group128_row" / "fp8_group128_col" with their
    options); b_codes [n, k] (uint8 or float8_e4m3fn) with b_scales fp32
    [ceil(n / 128), k / 128].  out is bf16 or fp16, allocated if missing.  A
    launch that gives up waiting shows in take_fault_flags.
    """
    L, empty = load(), _empty_for(stream)
    if dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {dtype}")
    if a_codes.dtype not in _CODE_TYPES or b_codes.dtype not in _CODE_TYPES:
        raise TypeError("codes must be uint8 or float8_e4m3fn")
    code = mode_code(mode)
    if code & 15 not in (MODES["fp8_group128_row"], MODES["fp8_group128_col"]):
        raise ValueError(f"the matrix product takes group-128 scales, not {mode!r}")
    if a_codes.dim() != 2 or b_codes.dim() != 2 or a_codes.shape[1] != b_codes.shape[1]:
        raise ValueError("codes must be [m, k] and [n, k]")
    (m, k), n = a_codes.shape, b_codes.shape[0]
    st_dtype = _U8 if code & OPTIONS["ue8m0"] else _F32
    if out is None:
        out = empty((m, n), dtype=dtype, device=a_codes.device)
    if code & 15 == MODES["fp8_group128_row"]:
        shape = (m, k // 128)
    else:
        per16 = 16 if code & OPTIONS["ue8m0"] else 4
        shape = (k // 128, (m + per16 - 1) // per16 * per16 if code & OPTIONS["tma"] else m)
    i, b_shape = a_codes.get_device(), ((n + 127) // 128, k // 128)
    if not (_is_current(i) and a_codes.is_contiguous() and _fits(a_scales, st_dtype, i, shape) and
            _fits(b_codes, b_codes.dtype, i, (n, k)) and _fits(b_scales, _F32, i, b_shape) and
            _fits(out, dtype, i, (m, n))):
        _check_tensors({"a_codes": a_codes, "a_scales": a_scales, "b_codes": b_codes, "b_scales": b_scales, "out": out},
                       {"a_codes": a_codes.dtype, "a_scales": st_dtype, "b_codes": b_codes.dtype, "b_scales": _F32,
                        "out": dtype})
        _want_shape("a_codes", a_codes, m, k)
        _want_shape("b_codes", b_codes, n, k)
        _want_shape("a_scales", a_scales, *shape)
        _want_shape("b_scales", b_scales, *b_shape)
        _want_shape("out", out, m, n)
    st = L.rmsq_fp8_block_matmul(a_codes.data_ptr(), a_scales.data_ptr(), code, b_codes.data_ptr(), b_scales.data_ptr(),
                                 out.data_ptr(), m, n, k, DTYPES[dtype], _stream(stream, i))
    if st:
        raise RmsqError(st, "rmsq_fp8_block_matmul")
    return out


def silu_mul_quant(gate_up: torch.Tensor, mode: str, scale_in: torch.Tensor | None = None, *,
                   out_q: torch.Tensor | None = None, out_scales: torch.Tensor | None = None, stream=None):
    """rmsq_silu_mul_quant on torch CUDA tensors: gate_up [n, 2d] (gate | up),
    scale_in a one-element fp32 device tensor (FP8 static scale / NVFP4 global
    scale).  Missing outputs are allocated.  Returns (q, scales)."""
    L, empty = load(), _empty_for(stream)
    n, d2 = gate_up.shape
    if gate_up.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {gate_up.dtype}")
    if d2 % 2:
        raise ValueError("gate_up must have an even number of columns (gate | up)")
    d = d2 // 2
    for t in (gate_up, out_q, out_scales, scale_in):
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if out_q is None:
        width = d // 2 if mode == "nvfp4" else d
        out_q = empty(n, width, dtype=torch.uint8, device=gate_up.device)
    if out_scales is None:
        out_scales = _scales_like(mode, n, d, gate_up.device, empty)
    st = L.rmsq_silu_mul_quant(_p(gate_up), mode_code(mode), _p(scale_in), _p(out_q), _p(out_scales), n, d,
                               DTYPES[gate_up.dtype], _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_silu_mul_quant")
    return out_q, out_scales


def nvfp4_dynamic_workspace_bytes(n_tokens: int) -> int:
    return load().rmsq_nvfp4_dynamic_workspace_bytes(n_tokens)


def fused_add_rmsnorm_nvfp4_dynamic(x: torch.Tensor, residual: torch.Tensor | None,
                                    weight: torch.Tensor, eps: float, *,
                                    out_q: torch.Tensor | None = None,
                                    out_scales: torch.Tensor | None = None,
                                    out_global_scale: torch.Tensor | None = None,
                                    residual_out: torch.Tensor | None = None,
                                    workspace: torch.Tensor | None = None, stream=None,
                                    variant: str = "auto"):
    """rmsq_fused_add_rmsnorm_nvfp4_dynamic on torch CUDA tensors: NVFP4 with
    gs = 2688 / amax(all y) computed on the device.  Missing outputs and the
    workspace are allocated.  Returns (q, block_scales, global_scale, residual_out)."""
    vcode = _variant(variant)
    L, empty = load(), _empty_for(stream)
    n, H = x.shape
    if x.dtype not in DTYPES:
        raise TypeError(f"unsupported activation dtype {x.dtype}")
    for t in (x, residual, weight, residual_out, out_q, out_scales, out_global_scale, workspace):
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    dev = x.device
    if out_q is None:
        out_q = empty(n, H // 2, dtype=torch.uint8, device=dev)
    if out_scales is None:
        out_scales = empty(n, H // 16, dtype=torch.uint8, device=dev)
    if out_global_scale is None:
        out_global_scale = empty(1, dtype=torch.float32, device=dev)
    if residual is not None and residual_out is None:
        residual_out = empty(residual.shape, dtype=residual.dtype, device=residual.device)
    ws_bytes = nvfp4_dynamic_workspace_bytes(n)
    if workspace is None:
        workspace = empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    st = L.rmsq_fused_add_rmsnorm_nvfp4_dynamic(
        _p(x), _p(residual), _p(weight), ctypes.c_float(eps), _p(out_q), _p(out_scales),
        _p(out_global_scale), _p(residual_out), _p(workspace),
        workspace.numel() * workspace.element_size(), n, H, DTYPES[x.dtype], _stream(stream),
        vcode)
    if st:
        raise RmsqError(st, "rmsq_fused_add_rmsnorm_nvfp4_dynamic")
    return out_q, out_scales, out_global_scale, residual_out


def query_launch(mode: str, n_tokens: int, hidden: int, residual: bool = True, dtype=torch.bfloat16,
                 variant: str = "auto") -> dict:
    """rmsq_query_launch: the launch the fused op would make on the current
    device for this mode and shape (kernel variant, chunks per thread, ring
    stages, CTAs, threads per CTA); nothing is launched."""
    out = (ctypes.c_int32 * 5)()
    st = load().rmsq_query_launch(mode_code(mode), n_tokens, hidden, 1 if residual else 0, DTYPES[dtype],
                                  _variant(variant), out)
    if st:
        raise RmsqError(st, "rmsq_query_launch")
    return {"pipelined": bool(out[0]), "chunks_per_thread": out[1], "stages": out[2], "ctas": out[3],
            "threads": out[4]}


def set_pipeline_config(chunks_per_thread: int = 0, stages: int = 0, ctas_per_sm: int = 0,
                        rows_per_iter: int = 0) -> None:
    """Tune the pipelined variant's launch shape (0 = automatic); results are unchanged."""
    st = load().rmsq_set_pipeline_config(chunks_per_thread, stages, ctas_per_sm, rows_per_iter)
    if st:
        raise RmsqError(st, "rmsq_set_pipeline_config")


def set_programmatic_launch(enable: bool) -> None:
    """Launch with programmatic dependent launch (default) or plain stream order."""
    st = load().rmsq_set_programmatic_launch(1 if enable else 0)
    if st:
        raise RmsqError(st, "rmsq_set_programmatic_launch")


def take_fault_flags() -> int:
    """Read and clear the flag of launches that gave up waiting (0 = none): the
    pipelined kernels, the FP8 matrix product and the attention of prompts.  The
    outputs of such a launch are incomplete."""
    f = ctypes.c_uint32()
    st = load().rmsq_take_fault_flags(ctypes.byref(f))
    if st:
        raise RmsqError(st, "rmsq_take_fault_flags")
    return f.value


def debug_activation(kind: str, values: torch.Tensor, up: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The library's e^x ("exp"; "exp_mid": the steps used for |x| <= 87),
    silu ("silu") or silu(g) * u ("silu_mul") on fp32 CUDA tensors, elementwise."""
    L, empty = load(), _empty_for(stream)
    with _on(stream) or contextlib.nullcontext():
        v = values.contiguous().float()
        u = None if up is None else up.contiguous().float()
    out = empty(v.shape, dtype=torch.float32, device=v.device)
    st = L.rmsq_debug_activation({"exp": 0, "silu": 1, "silu_mul": 2, "exp_mid": 3}[kind], _p(v), _p(u), _p(out), v.numel(),
                                 _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_debug_activation")
    return out


def debug_bounded_wait(limit_ns: int) -> int:
    """Run the bounded-wait check (rmsq_debug_bounded_wait); returns gave_up."""
    out = ctypes.c_int(-1)
    st = load().rmsq_debug_bounded_wait(int(limit_ns), ctypes.byref(out))
    if st:
        raise RmsqError(st, "rmsq_debug_bounded_wait")
    return out.value


def debug_convert(kind: str, values: torch.Tensor, stream=None) -> torch.Tensor:
    """The library's E4M3 ("e4m3") or E2M1 ("e2m1", low nibble) conversion of a
    fp32 CUDA tensor."""
    L, empty = load(), _empty_for(stream)
    with _on(stream) or contextlib.nullcontext():
        v = values.contiguous().float()
    out = empty(v.shape, dtype=torch.uint8, device=v.device)
    st = L.rmsq_debug_convert({"e4m3": 0, "e2m1": 1}[kind], _p(v), _p(out), v.numel(), _stream(stream))
    if st:
        raise RmsqError(st, "rmsq_debug_convert")
    return out
