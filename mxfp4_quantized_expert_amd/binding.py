"""Binding of libmxfp4moe.so.

Argument marshalling only: dtype/device/shape checks, output allocation with
torch, and the raw C call on torch's current HIP stream, by ctypes or, for plain
calls of the layer's separate operators, in one step of native code.  Every step
of the computation runs in the library's HIP kernels; there is no other code
path.  The C ABI is declared in include/mxfp4moe.h.
"""

from __future__ import annotations

import ctypes
import os
import warnings
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4moe.so")
HOST_PATH = os.path.join(os.path.dirname(LIB_PATH), "_host_calls.so")

STATUS = {
    0: "ok",
    -1: "invalid argument",
    -2: "unsupported shape",
    -3: "workspace too small",
    -4: "pointer not aligned as required",
    -5: "HIP launch error",
    -6: "layer needs more than the no-allocation scratch",
}

STAGES = {"route": 1, "group": 2, "gate_up": 3, "down": 4, "combine": 5, "dequant": 6,
          "gate_up_wide": 7, "gate_up_stream": 8, "down_wide": 9, "down_stream": 10,
          "gate_up_mid": 11, "down_mid": 12, "act_quant": 13, "permute": 14, "unpermute": 15,
          "unpermute_backward": 16, "route_backward": 17, "linear": 18, "linear_backward": 19,
          "rms_norm": 20, "rms_norm_backward": 21, "swiglu": 22, "swiglu_backward": 23, "fp8_quantize": 24,
          "fp8_linear": 25, "fp8_linear_backward": 26, "balance_loss": 27, "balance_loss_backward": 28}

_lib: Optional[ctypes.CDLL] = None
# The module of the short host path (csrc/host_calls.cpp), set with _lib; without it, or with one that
# cannot be loaded, every call goes through ctypes.
_host = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class MXFP4MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the HIP library; raises if it has not been built (no fallback exists)."""
    global _lib, _host
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "or python -m mxfp4_quantized_expert_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    lib.mxfp4_dequantize.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp]
    lib.mxfp4_dequantize.restype = ctypes.c_int
    lib.mxfp4_dequantize_from_host.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, ctypes.POINTER(ctypes.c_size_t), _vp]
    lib.mxfp4_dequantize_from_host.restype = ctypes.c_int
    lib.moe_mxfp4_route.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.moe_mxfp4_route.restype = ctypes.c_int
    lib.moe_mxfp4_forward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i64, _i64, _i64, _i64, _i64, _vp,
                                      ctypes.POINTER(ctypes.c_size_t), _vp]
    lib.moe_mxfp4_forward.restype = ctypes.c_int
    lib.moe_mxfp4_forward_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _i64, _i64, _i64, _i64, _i64, _vp]
    lib.moe_mxfp4_forward_noalloc.restype = ctypes.c_int
    lib.moe_mxfp4_forward_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _i64, _i64, _i64, _i64, _i64, ctypes.c_uint32, _vp,
                                         ctypes.POINTER(ctypes.c_size_t), _vp]
    lib.moe_mxfp4_forward_ex.restype = ctypes.c_int
    lib.moe_nvfp4_forward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i64, _i64, _i64, _i64, _i64, _vp, ctypes.POINTER(ctypes.c_size_t), _vp]
    lib.moe_nvfp4_forward.restype = ctypes.c_int
    lib.moe_mxfp4_router.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
    lib.moe_mxfp4_router.restype = ctypes.c_int
    lib.moe_mxfp4_forward_router.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _i64, _i64, _i64, _i64, _i64, ctypes.c_uint32, _vp,
                                             ctypes.POINTER(ctypes.c_size_t), _vp]
    lib.moe_mxfp4_forward_router.restype = ctypes.c_int
    lib.moe_mxfp8_quantize.argtypes = [_vp, _i64, _i64, ctypes.c_int, _vp, _vp, _vp]
    lib.moe_mxfp8_quantize.restype = ctypes.c_int
    lib.moe_permute.argtypes = [_vp, ctypes.c_int, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp]
    lib.moe_permute.restype = ctypes.c_int
    lib.moe_permute_backward.argtypes = [_vp, ctypes.c_int, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_permute_backward.restype = ctypes.c_int
    lib.moe_unpermute.argtypes = [_vp, ctypes.c_int, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_unpermute.restype = ctypes.c_int
    lib.moe_unpermute_backward.argtypes = [_vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp,
                                           _vp]
    lib.moe_unpermute_backward.restype = ctypes.c_int
    lib.moe_route_backward.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]
    lib.moe_route_backward.restype = ctypes.c_int
    lib.moe_mxfp4_linear.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_mxfp4_linear.restype = ctypes.c_int
    lib.moe_nvfp4_linear.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_nvfp4_linear.restype = ctypes.c_int
    lib.moe_mxfp4_linear_backward.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_mxfp4_linear_backward.restype = ctypes.c_int
    lib.moe_nvfp4_linear_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_nvfp4_linear_backward.restype = ctypes.c_int
    size_p = ctypes.POINTER(ctypes.c_size_t)
    f32, i32 = ctypes.c_float, ctypes.c_int
    lib.moe_rms_norm.argtypes = [_vp, _vp, _vp, i32, i32, f32, _i64, _i64, _vp, _vp, _vp, _vp]
    lib.moe_rms_norm.restype = ctypes.c_int
    lib.moe_rms_norm_fp8.argtypes = [_vp, _vp, _vp, i32, i32, f32, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.moe_rms_norm_fp8.restype = ctypes.c_int
    lib.moe_rms_norm_backward.argtypes = [_vp, _vp, _vp, _vp, i32, i32, _vp, _i64, _i64, _vp, _vp, _vp, size_p, _vp]
    lib.moe_rms_norm_backward.restype = ctypes.c_int
    lib.moe_fp8_quantize.argtypes = [_vp, i32, _i64, _i64, _vp, _vp, _vp]
    lib.moe_fp8_quantize.restype = ctypes.c_int
    lib.moe_fp8_linear.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_fp8_linear.restype = ctypes.c_int
    lib.moe_fp8_linear_backward.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp]
    lib.moe_fp8_linear_backward.restype = ctypes.c_int
    lib.moe_swiglu.argtypes = [_vp, i32, _i64, _i64, f32, f32, f32, i32, _vp, _vp]
    lib.moe_swiglu.restype = ctypes.c_int
    lib.moe_swiglu_fp8.argtypes = [_vp, i32, _i64, _i64, f32, f32, f32, i32, _vp, _vp, _vp]
    lib.moe_swiglu_fp8.restype = ctypes.c_int
    lib.moe_swiglu_backward.argtypes = [_vp, _vp, i32, _i64, _i64, f32, f32, f32, i32, _vp, _vp]
    lib.moe_swiglu_backward.restype = ctypes.c_int
    lib.moe_balance_loss.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, size_p, _vp]
    lib.moe_balance_loss.restype = ctypes.c_int
    lib.moe_balance_loss_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp]
    lib.moe_balance_loss_backward.restype = ctypes.c_int
    lib.mxfp4moe_status_string.argtypes = [ctypes.c_int]
    lib.mxfp4moe_status_string.restype = ctypes.c_char_p
    lib.mxfp4moe_profile_begin.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.mxfp4moe_profile_begin.restype = ctypes.c_int
    lib.mxfp4moe_profile_end.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_int]
    lib.mxfp4moe_profile_end.restype = ctypes.c_int
    if os.path.exists(HOST_PATH):
        try:
            from . import _host_calls
            _host = _host_calls
        except (ImportError, AttributeError) as e:  # built for another Python or torch
            warnings.warn(f"{HOST_PATH} cannot be loaded, calls take the longer way through ctypes: {e}",
                          RuntimeWarning, stacklevel=2)
    _lib = lib
    return lib


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:  # torch.Size is a tuple
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _raise(fn: str, st: int):
    if st != 0:
        raise MXFP4MoEError(fn, st)


def mxfp4_dequantize(blocks: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """blocks [..., N, K/2] uint8 + scales [..., N, K/32] uint8 -> [..., N, K] bfloat16."""
    lib = load()
    half_k = blocks.shape[-1]
    K = 2 * half_k
    lead = tuple(blocks.shape[:-1])
    _check(blocks, "blocks", torch.uint8)
    _check(scales, "scales", torch.uint8, lead + (K // 32,))
    if out is None:
        out = torch.empty(lead + (K,), dtype=torch.bfloat16, device=blocks.device)
    _check(out, "out", torch.bfloat16, lead + (K,))
    N = 1
    for d in lead:
        N *= d
    st = lib.mxfp4_dequantize(blocks.data_ptr(), scales.data_ptr(), out.data_ptr(), N, K, _stream(stream))
    _raise("mxfp4_dequantize", st)
    return out


def offload_staging_bytes(N: int, K: int) -> int:
    """Device staging mxfp4_dequantize_from_host needs for N rows of K elements."""
    n = ctypes.c_size_t(0)
    st = load().mxfp4_dequantize_from_host(None, None, None, N, K, None, ctypes.byref(n), None)
    _raise("mxfp4_dequantize_from_host(staging query)", st)
    return int(n.value)


def mxfp4_dequantize_from_host(blocks: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                               staging: Optional[torch.Tensor] = None, device="cuda",
                               stream=None) -> torch.Tensor:
    """Host blocks [..., N, K/2] + host scales [..., N, K/32] (uint8, CPU; pinned memory copies
    asynchronously) -> device bf16 [..., N, K], copied in chunks and dequantized on arrival."""
    lib = load()
    half_k = blocks.shape[-1]
    K = 2 * half_k
    lead = tuple(blocks.shape[:-1])
    for t, name, shape in ((blocks, "blocks", None), (scales, "scales", lead + (K // 32,))):
        if t.dtype != torch.uint8 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 host tensor")
        if shape is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    N = 1
    for d in lead:
        N *= d
    if out is None:
        out = torch.empty(lead + (K,), dtype=torch.bfloat16, device=device)
    _check(out, "out", torch.bfloat16, lead + (K,))
    need = offload_staging_bytes(N, K)
    if staging is None:
        staging = torch.empty((max(need, 1),), dtype=torch.uint8, device=out.device)
    _check(staging, "staging", torch.uint8)
    n = ctypes.c_size_t(staging.numel())
    st = lib.mxfp4_dequantize_from_host(blocks.data_ptr(), scales.data_ptr(), out.data_ptr(), N, K,
                                        staging.data_ptr(), ctypes.byref(n), _stream(stream))
    _raise("mxfp4_dequantize_from_host", st)
    return out


def moe_mxfp4_route(router_logits: torch.Tensor, top_k: int, stream=None):
    """Returns (topk_ids [T,k] int32, topk_weights [T,k] float32, expert_offsets [E+1] int32,
    sorted_pairs [T*k] int32)."""
    lib = load()
    _check(router_logits, "router_logits", torch.float32)
    T, E = router_logits.shape
    dev = router_logits.device
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    pairs = torch.empty((T * top_k,), dtype=torch.int32, device=dev)
    st = lib.moe_mxfp4_route(router_logits.data_ptr(), T, E, top_k, ids.data_ptr(), w.data_ptr(),
                             offsets.data_ptr(), pairs.data_ptr(), _stream(stream))
    _raise("moe_mxfp4_route", st)
    return ids, w, offsets, pairs


def moe_mxfp8_quantize(src: torch.Tensor, split: bool = True, stream=None):
    """bf16 [rows, K] -> (codes [rows, 128*ceil(K/64)] uint8, scales [rows, 4*ceil(K/64)] uint8)
    in the chunk-interleaved layout of the FP4 scaled-MFMA path."""
    lib = load()
    rows, K = src.shape
    _check(src, "src", torch.bfloat16)
    nc = (K + 63) // 64
    codes = torch.empty((rows, 128 * nc), dtype=torch.uint8, device=src.device)
    scales = torch.empty((rows, 4 * nc), dtype=torch.uint8, device=src.device)
    st = lib.moe_mxfp8_quantize(src.data_ptr(), rows, K, 1 if split else 0, codes.data_ptr(), scales.data_ptr(),
                                _stream(stream))
    _raise("moe_mxfp8_quantize", st)
    return codes, scales


def moe_mxfp4_router(x: torch.Tensor, router_w: torch.Tensor, router_b: torch.Tensor, top_k: int, stream=None):
    """Router projection fused ahead of the top-k.  Returns (logits [T,E] float32,
    topk_ids [T,k] int32, topk_weights [T,k] float32)."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    _check(x, "x", torch.bfloat16, (T, H))
    _check(router_w, "router_w", torch.bfloat16, (E, H))
    _check(router_b, "router_b", torch.bfloat16, (E,))
    dev = x.device
    logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    st = lib.moe_mxfp4_router(x.data_ptr(), router_w.data_ptr(), router_b.data_ptr(), T, H, E, top_k,
                              logits.data_ptr(), ids.data_ptr(), w.data_ptr(), _stream(stream))
    _raise("moe_mxfp4_router", st)
    return logits, ids, w


FLAG_GATE_UP_SPLIT = 1
ACT_FLAGS = {"bf16": 0, "mxfp8": 2, "mxfp8_split": 4}
FLAG_TILES_STREAM = 8


def workspace_bytes(T: int, H: int, I: int, E: int, top_k: int, flags: int = 0) -> int:
    """Device workspace moe_mxfp4_forward needs for these sizes (and layout/activation flags)."""
    lib = load()
    n = ctypes.c_size_t(0)
    st = lib.moe_mxfp4_forward_ex(None, None, None, None, None, None, None, None, None,
                                  T, H, I, E, top_k, flags, None, ctypes.byref(n), None)
    _raise("moe_mxfp4_forward(workspace query)", st)
    return int(n.value)


def moe_mxfp4_forward(x: torch.Tensor, router_logits: torch.Tensor,
                      w13_blocks: torch.Tensor, w13_scales: torch.Tensor, w13_bias: torch.Tensor,
                      w2_blocks: torch.Tensor, w2_scales: torch.Tensor, w2_bias: torch.Tensor,
                      top_k: int, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None,
                      gate_up_split: bool = False, act: str = "bf16",
                      stream_tiles_only: bool = False) -> torch.Tensor:
    """One MXFP4 MoE expert layer; returns y [T, H] bfloat16.  gate_up_split: w13 rows are
    [I gate rows; I up rows] instead of interleaved.  act: "bf16" (exact), or the opt-in
    FP4 scaled-MFMA path for experts with at least 128 pairs over MXFP8 activations,
    "mxfp8_split" (high part + residual) or "mxfp8" (one tensor).  stream_tiles_only:
    every pair through the streaming kernels (MXFP4MOE_TILES_STREAM)."""
    lib = load()
    T, H = x.shape
    E = router_logits.shape[1]
    I = w2_blocks.shape[-1] * 2
    _check(x, "x", torch.bfloat16, (T, H))
    _check(router_logits, "router_logits", torch.float32, (T, E))
    _check(w13_blocks, "w13_blocks", torch.uint8, (E, 2 * I, H // 2))
    _check(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32))
    _check(w13_bias, "w13_bias", torch.bfloat16, (E, 2 * I))
    _check(w2_blocks, "w2_blocks", torch.uint8, (E, H, I // 2))
    _check(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32))
    _check(w2_bias, "w2_bias", torch.bfloat16, (E, H))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (T, H))
    flags = (FLAG_GATE_UP_SPLIT if gate_up_split else 0) | ACT_FLAGS[act] | (FLAG_TILES_STREAM if stream_tiles_only else 0)
    if workspace is None:  # a caller's workspace is size-checked by the library
        workspace = torch.empty((max(workspace_bytes(T, H, I, E, top_k, flags), 1),), dtype=torch.uint8, device=x.device)
    _check(workspace, "workspace", torch.uint8)
    n = ctypes.c_size_t(workspace.numel())
    st = lib.moe_mxfp4_forward_ex(x.data_ptr(), router_logits.data_ptr(),
                                  w13_blocks.data_ptr(), w13_scales.data_ptr(), w13_bias.data_ptr(),
                                  w2_blocks.data_ptr(), w2_scales.data_ptr(), w2_bias.data_ptr(),
                                  out.data_ptr(), T, H, I, E, top_k, flags,
                                  workspace.data_ptr(), ctypes.byref(n), _stream(stream))
    _raise("moe_mxfp4_forward", st)
    return out


NOALLOC_SCRATCH_BYTES = 32 << 20


def moe_mxfp4_forward_noalloc(x: torch.Tensor, router_logits: torch.Tensor,
                              w13_blocks: torch.Tensor, w13_scales: torch.Tensor, w13_bias: torch.Tensor,
                              w2_blocks: torch.Tensor, w2_scales: torch.Tensor, w2_bias: torch.Tensor,
                              top_k: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_mxfp4_forward through the entry point that takes no workspace (its scratch
    is a fixed device array of the library); returns y [T, H] bfloat16."""
    lib = load()
    T, H = x.shape
    E = router_logits.shape[1]
    I = w2_blocks.shape[-1] * 2
    _check(x, "x", torch.bfloat16, (T, H))
    _check(router_logits, "router_logits", torch.float32, (T, E))
    _check(w13_blocks, "w13_blocks", torch.uint8, (E, 2 * I, H // 2))
    _check(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32))
    _check(w13_bias, "w13_bias", torch.bfloat16, (E, 2 * I))
    _check(w2_blocks, "w2_blocks", torch.uint8, (E, H, I // 2))
    _check(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32))
    _check(w2_bias, "w2_bias", torch.bfloat16, (E, H))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (T, H))
    st = lib.moe_mxfp4_forward_noalloc(x.data_ptr(), router_logits.data_ptr(),
                                       w13_blocks.data_ptr(), w13_scales.data_ptr(), w13_bias.data_ptr(),
                                       w2_blocks.data_ptr(), w2_scales.data_ptr(), w2_bias.data_ptr(),
                                       out.data_ptr(), T, H, I, E, top_k, _stream(stream))
    _raise("moe_mxfp4_forward_noalloc", st)
    return out


def moe_mxfp4_forward_router(x: torch.Tensor, router_w: torch.Tensor, router_b: torch.Tensor,
                             w13_blocks: torch.Tensor, w13_scales: torch.Tensor, w13_bias: torch.Tensor,
                             w2_blocks: torch.Tensor, w2_scales: torch.Tensor, w2_bias: torch.Tensor,
                             top_k: int, out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None,
                             gate_up_split: bool = False) -> torch.Tensor:
    """One MXFP4 MoE expert layer whose logits come from the router projection
    x W_r^T + b_r (router_w [E,H], router_b [E] bfloat16); returns y [T, H] bfloat16."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    I = w2_blocks.shape[-1] * 2
    _check(x, "x", torch.bfloat16, (T, H))
    _check(router_w, "router_w", torch.bfloat16, (E, H))
    _check(router_b, "router_b", torch.bfloat16, (E,))
    _check(w13_blocks, "w13_blocks", torch.uint8, (E, 2 * I, H // 2))
    _check(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32))
    _check(w13_bias, "w13_bias", torch.bfloat16, (E, 2 * I))
    _check(w2_blocks, "w2_blocks", torch.uint8, (E, H, I // 2))
    _check(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32))
    _check(w2_bias, "w2_bias", torch.bfloat16, (E, H))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (T, H))
    if workspace is None:  # a caller's workspace is size-checked by the library
        workspace = torch.empty((max(workspace_bytes(T, H, I, E, top_k), 1),), dtype=torch.uint8, device=x.device)
    _check(workspace, "workspace", torch.uint8)
    n = ctypes.c_size_t(workspace.numel())
    st = lib.moe_mxfp4_forward_router(x.data_ptr(), router_w.data_ptr(), router_b.data_ptr(),
                                      w13_blocks.data_ptr(), w13_scales.data_ptr(), w13_bias.data_ptr(),
                                      w2_blocks.data_ptr(), w2_scales.data_ptr(), w2_bias.data_ptr(),
                                      out.data_ptr(), T, H, I, E, top_k, 1 if gate_up_split else 0,
                                      workspace.data_ptr(), ctypes.byref(n), _stream(stream))
    _raise("moe_mxfp4_forward_router", st)
    return out


def moe_nvfp4_forward(x: torch.Tensor, router_logits: torch.Tensor,
                      w13_blocks: torch.Tensor, w13_scales: torch.Tensor, w13_scale2: torch.Tensor,
                      w13_bias: torch.Tensor, w2_blocks: torch.Tensor, w2_scales: torch.Tensor,
                      w2_scale2: torch.Tensor, w2_bias: torch.Tensor, top_k: int,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """One NVFP4 MoE expert layer (E4M3 block scales per 16, float32 second-level
    scales [E]); returns y [T, H] bfloat16."""
    lib = load()
    T, H = x.shape
    E = router_logits.shape[1]
    I = w2_blocks.shape[-1] * 2
    _check(x, "x", torch.bfloat16, (T, H))
    _check(router_logits, "router_logits", torch.float32, (T, E))
    _check(w13_blocks, "w13_blocks", torch.uint8, (E, 2 * I, H // 2))
    _check(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 16))
    _check(w13_scale2, "w13_scale2", torch.float32, (E,))
    _check(w13_bias, "w13_bias", torch.bfloat16, (E, 2 * I))
    _check(w2_blocks, "w2_blocks", torch.uint8, (E, H, I // 2))
    _check(w2_scales, "w2_scales", torch.uint8, (E, H, I // 16))
    _check(w2_scale2, "w2_scale2", torch.float32, (E,))
    _check(w2_bias, "w2_bias", torch.bfloat16, (E, H))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (T, H))
    if workspace is None:  # a caller's workspace is size-checked by the library
        workspace = torch.empty((max(workspace_bytes(T, H, I, E, top_k), 1),), dtype=torch.uint8, device=x.device)
    _check(workspace, "workspace", torch.uint8)
    n = ctypes.c_size_t(workspace.numel())
    st = lib.moe_nvfp4_forward(x.data_ptr(), router_logits.data_ptr(), w13_blocks.data_ptr(),
                               w13_scales.data_ptr(), w13_scale2.data_ptr(), w13_bias.data_ptr(),
                               w2_blocks.data_ptr(), w2_scales.data_ptr(), w2_scale2.data_ptr(),
                               w2_bias.data_ptr(), out.data_ptr(), T, H, I, E, top_k, workspace.data_ptr(),
                               ctypes.byref(n), _stream(stream))
    _raise("moe_nvfp4_forward", st)
    return out


# ---- the layer's steps as operators of their own
#
# They record nothing for autograd: no output requires a gradient, also where an input does.  A caller
# that trains joins a call and its _backward in a torch.autograd.Function.

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


# The current stream's handle without building a torch.cuda.Stream (0.07 against 2.7 us of host
# time a call; a call of a few tokens is bound by its host time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # of an initialised runtime


def _current_stream(t: torch.Tensor) -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream(t.get_device())


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """Whether a call on t has to be moved to another device or stream than the current ones."""
    return stream is not None or (isinstance(t, torch.Tensor) and t.is_cuda
                                  and t.get_device() != _current_device())


def _fits(t: torch.Tensor, dtype: torch.dtype, shape, device: torch.device) -> bool:
    """Whether t passes _check_on, in the few steps that every call of a small batch pays for."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape
            and t.is_contiguous())


def _place(t: torch.Tensor, stream):
    """Context in which t's device and the stream asked for are the current ones, so that the
    outputs and workspaces allocated in it belong to the stream that the kernels run on."""
    if stream is None:
        return torch.cuda.device(t.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                  else torch.cuda.default_stream(t.device))
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _check_on(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: torch.device):
    if _fits(t, dtype, shape, device):
        return
    _check(t, name, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _apart(out: torch.Tensor, name: str, *inputs):
    """Refuses an output that shares memory with an input (None: none): rows are read and written in no order."""
    a, n = out.data_ptr(), out.numel() * out.element_size()
    for t in inputs:
        if t is not None and n and t.numel():
            b = t.data_ptr()
            if a < b + t.numel() * t.element_size() and b < a + n:
                raise ValueError(f"{name} shares memory with an input")


def _element_type(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected 2")
    return code


def _count(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a tensor of one dimension")
    return t.shape[0]


def moe_permute(x: torch.Tensor, sorted_pairs: torch.Tensor, top_k: int, out: Optional[torch.Tensor] = None,
                pair_rows: Optional[torch.Tensor] = None, stream=None):
    """Token rows in expert order: rows[i] = x[sorted_pairs[i] // top_k] for x [T, H] (bfloat16,
    float16 or float32) and sorted_pairs [R] int32, as moe_mxfp4_route gives them; an entry
    outside [0, T * top_k) makes an empty row of zeros.  Returns (rows [R, H], pair_rows
    [T * top_k] int32: every pair's row, -1 for none).  The rows
    never require a gradient: moe_permute_backward computes it."""
    if _host is not None and stream is None and out is None and pair_rows is None:
        got = _host.permute(x, sorted_pairs, top_k)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_permute(x, sorted_pairs, top_k, out, pair_rows)
    code = _element_type(x, "x")
    T, H = x.shape
    R = _count(sorted_pairs, "sorted_pairs")
    if top_k < 1:
        raise ValueError(f"top_k must be at least 1, got {top_k}")
    dev = x.device
    _check(x, "x", x.dtype)
    _check_on(sorted_pairs, "sorted_pairs", torch.int32, (R,), dev)
    if out is None:
        out = x.new_empty((R, H))
    else:
        _check_on(out, "out", x.dtype, (R, H), dev)
        _apart(out, "out", x, sorted_pairs)
    if pair_rows is None:
        pair_rows = sorted_pairs.new_empty((T * top_k,))
    else:
        _check_on(pair_rows, "pair_rows", torch.int32, (T * top_k,), dev)
        _apart(pair_rows, "pair_rows", x, sorted_pairs, out)
    st = load().moe_permute(x.data_ptr(), code, sorted_pairs.data_ptr(), T, H, top_k, R, out.data_ptr(),
                            pair_rows.data_ptr(), _current_stream(x))
    _raise("moe_permute", st)
    return out, pair_rows


def moe_permute_backward(d_rows: torch.Tensor, pair_rows: torch.Tensor, top_k: int,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_permute: dx[t] = sum_j d_rows[pair_rows[t * top_k + j]] over the pairs
    that have a row; d_rows [R, H], pair_rows [T * top_k].  Returns dx [T, H]."""
    if _host is not None and stream is None and out is None:
        got = _host.permute_backward(d_rows, pair_rows, top_k)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(d_rows, stream):
        with _place(d_rows, stream):
            return moe_permute_backward(d_rows, pair_rows, top_k, out)
    code = _element_type(d_rows, "d_rows")
    R, H = d_rows.shape
    P = _count(pair_rows, "pair_rows")
    if top_k < 1 or P % top_k:
        raise ValueError(f"pair_rows has {P} entries, not a multiple of top_k = {top_k}")
    T, dev = P // top_k, d_rows.device
    _check(d_rows, "d_rows", d_rows.dtype)
    _check_on(pair_rows, "pair_rows", torch.int32, (P,), dev)
    if out is None:
        out = d_rows.new_empty((T, H))
    else:
        _check_on(out, "out", d_rows.dtype, (T, H), dev)
        _apart(out, "out", d_rows, pair_rows)
    st = load().moe_permute_backward(d_rows.data_ptr(), code, pair_rows.data_ptr(), T, H, top_k, R, out.data_ptr(),
                                     _current_stream(d_rows))
    _raise("moe_permute_backward", st)
    return out


def moe_unpermute(rows: torch.Tensor, pair_rows: torch.Tensor, topk_weights: torch.Tensor,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' rows summed back: y[t] = sum_j topk_weights[t, j] * rows[pair_rows[t * top_k + j]]
    over the pairs that have a row (fp32, rounded once).  rows [R, H] (bfloat16, float16 or
    float32), pair_rows [T * top_k] int32 of moe_permute, topk_weights [T, top_k] float32.
    Returns y [T, H].  The output
    never requires a gradient: moe_unpermute_backward computes it."""
    if _host is not None and stream is None and out is None:
        got = _host.unpermute(rows, pair_rows, topk_weights)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(rows, stream):
        with _place(rows, stream):
            return moe_unpermute(rows, pair_rows, topk_weights, out)
    code = _element_type(rows, "rows")
    R, H = rows.shape
    T, top_k = topk_weights.shape
    dev = rows.device
    _check(rows, "rows", rows.dtype)
    _check_on(topk_weights, "topk_weights", torch.float32, (T, top_k), dev)
    _check_on(pair_rows, "pair_rows", torch.int32, (T * top_k,), dev)
    if out is None:
        out = rows.new_empty((T, H))
    else:
        _check_on(out, "out", rows.dtype, (T, H), dev)
        _apart(out, "out", rows, pair_rows, topk_weights)
    st = load().moe_unpermute(rows.data_ptr(), code, pair_rows.data_ptr(), topk_weights.data_ptr(), T, H, top_k, R,
                              out.data_ptr(), _current_stream(rows))
    _raise("moe_unpermute", st)
    return out


def moe_unpermute_backward(dy: torch.Tensor, rows: torch.Tensor, sorted_pairs: torch.Tensor,
                           pair_rows: torch.Tensor, topk_weights: torch.Tensor,
                           d_rows: Optional[torch.Tensor] = None, d_weights: Optional[torch.Tensor] = None,
                           stream=None):
    """Gradients of moe_unpermute for dy [T, H]: d_rows [R, H] (the pair's weight times its token's
    dy; zeros for empty rows) and d_weights [T, top_k] float32 (dot products of dy[t] and the pairs'
    rows; 0 for a pair without one).  sorted_pairs and pair_rows as moe_permute read and wrote them."""
    if _host is not None and stream is None and d_rows is None and d_weights is None:
        got = _host.unpermute_backward(dy, rows, sorted_pairs, pair_rows, topk_weights)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(rows, stream):
        with _place(rows, stream):
            return moe_unpermute_backward(dy, rows, sorted_pairs, pair_rows, topk_weights, d_rows, d_weights)
    code = _element_type(rows, "rows")
    R, H = rows.shape
    T, top_k = topk_weights.shape
    dev = rows.device
    _check(rows, "rows", rows.dtype)
    _check_on(dy, "dy", rows.dtype, (T, H), dev)
    _check_on(sorted_pairs, "sorted_pairs", torch.int32, (R,), dev)
    _check_on(pair_rows, "pair_rows", torch.int32, (T * top_k,), dev)
    _check_on(topk_weights, "topk_weights", torch.float32, (T, top_k), dev)
    if d_rows is None:
        d_rows = rows.new_empty((R, H))
    else:
        _check_on(d_rows, "d_rows", rows.dtype, (R, H), dev)
        _apart(d_rows, "d_rows", dy, rows, sorted_pairs, pair_rows, topk_weights)
    if d_weights is None:
        d_weights = topk_weights.new_empty((T, top_k))
    else:
        _check_on(d_weights, "d_weights", torch.float32, (T, top_k), dev)
        _apart(d_weights, "d_weights", dy, rows, sorted_pairs, pair_rows, topk_weights, d_rows)
    st = load().moe_unpermute_backward(dy.data_ptr(), rows.data_ptr(), code, sorted_pairs.data_ptr(),
                                       pair_rows.data_ptr(), topk_weights.data_ptr(), T, H, top_k, R,
                                       d_rows.data_ptr(), d_weights.data_ptr(), _current_stream(rows))
    _raise("moe_unpermute_backward", st)
    return d_rows, d_weights


def moe_route_backward(topk_ids: torch.Tensor, topk_weights: torch.Tensor, d_weights: torch.Tensor,
                       num_experts: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the softmax over a token's picks: topk_ids [T, top_k] int32, topk_weights and
    d_weights [T, top_k] float32 -> d_logits [T, num_experts] float32, zero at experts not picked."""
    if _host is not None and stream is None and out is None:
        got = _host.route_backward(topk_ids, topk_weights, d_weights, num_experts)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(topk_weights, stream):
        with _place(topk_weights, stream):
            return moe_route_backward(topk_ids, topk_weights, d_weights, num_experts, out)
    T, top_k = topk_weights.shape
    dev = topk_weights.device
    _check(topk_weights, "topk_weights", torch.float32)
    _check_on(topk_ids, "topk_ids", torch.int32, (T, top_k), dev)
    _check_on(d_weights, "d_weights", torch.float32, (T, top_k), dev)
    if num_experts < 1:
        raise ValueError(f"num_experts must be at least 1, got {num_experts}")
    if out is None:
        out = topk_weights.new_empty((T, num_experts))
    else:
        _check_on(out, "out", torch.float32, (T, num_experts), dev)
        _apart(out, "out", topk_ids, topk_weights, d_weights)
    st = load().moe_route_backward(topk_ids.data_ptr(), topk_weights.data_ptr(), d_weights.data_ptr(), T,
                                   num_experts, top_k, out.data_ptr(), _current_stream(out))
    _raise("moe_route_backward", st)
    return out


def _linear_sizes(rows, name: str, blocks, scales, group: int, expert_offsets, scale2, bias):
    """(E, N, K) of a linear operator's weights, after the checks of every tensor but the rows' width."""
    if not isinstance(rows, torch.Tensor) or not isinstance(blocks, torch.Tensor):
        raise TypeError(f"{name} and blocks must be torch.Tensors")
    lead = 2 if expert_offsets is None else 3
    shape = blocks.shape
    if rows.dim() != 2:
        raise ValueError(f"{name} has {rows.dim()} dimensions, expected 2")
    if len(shape) != lead:
        raise ValueError(f"blocks has {len(shape)} dimensions, expected {lead} "
                         f"{'without' if lead == 2 else 'with'} expert_offsets")
    E = 1 if lead == 2 else shape[0]
    N, K = shape[-2], 2 * shape[-1]
    dev = rows.device
    if not (rows.dtype is torch.bfloat16 and rows.is_cuda and rows.is_contiguous()):
        _check(rows, name, torch.bfloat16)
    _check_on(blocks, "blocks", torch.uint8, shape, dev)
    _check_on(scales, "scales", torch.uint8, (*shape[:-1], K // group), dev)
    if expert_offsets is not None:
        _check_on(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev)
    if group == 16:
        _check_on(scale2, "scale2", torch.float32, (E,), dev)
    if bias is not None:
        _check_on(bias, "bias", torch.bfloat16, shape[:-1], dev)
    return E, N, K


def _linear(fn: str, forward: bool, group: int, rows, blocks, scales, scale2, bias, expert_offsets, out):
    """A linear operator's call: rows [R, K] -> [R, N], or the gradient's [R, N] -> [R, K]."""
    name = "x" if forward else "dy"
    E, N, K = _linear_sizes(rows, name, blocks, scales, group, expert_offsets, scale2, bias)
    R, width = rows.shape
    have, give = (K, N) if forward else (N, K)
    if width != have:
        raise ValueError(f"{name} has rows of {width}, expected {have}")
    if out is None:
        out = rows.new_empty((R, give))
    else:
        _check_on(out, "out", torch.bfloat16, (R, give), rows.device)
        _apart(out, "out", rows, blocks, scales, scale2, bias, expert_offsets)
    args = [rows.data_ptr(), blocks.data_ptr(), scales.data_ptr()]
    if group == 16:
        args.append(scale2.data_ptr())
    if forward:
        args.append(None if bias is None else bias.data_ptr())
    st = getattr(load(), fn)(*args, None if expert_offsets is None else expert_offsets.data_ptr(), R, K, N, E,
                             out.data_ptr(), _current_stream(rows))
    if st:
        raise MXFP4MoEError(fn, st)
    return out


def moe_mxfp4_linear(x: torch.Tensor, blocks: torch.Tensor, scales: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows times MXFP4 weights: y = x W^T (+ bias) for x [R, K] bfloat16.  Dense: blocks [N, K/2]
    and scales [N, K/32] uint8, bias [N] bfloat16.  Per expert: blocks [E, N, K/2], scales
    [E, N, K/32], bias [E, N] and expert_offsets [E + 1] int32 (expert e has the rows
    [offsets[e], offsets[e + 1]); rows outside them keep what `out` held, and without `out` hold
    anything).  Returns y [R, N].  The output
    never requires a gradient: moe_mxfp4_linear_backward computes it."""
    if _host is not None and stream is None and out is None:
        got = _host.linear(False, 32, x, blocks, scales, None, bias, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_mxfp4_linear(x, blocks, scales, bias, expert_offsets, out)
    return _linear("moe_mxfp4_linear", True, 32, x, blocks, scales, None, bias, expert_offsets, out)


def moe_nvfp4_linear(x: torch.Tensor, blocks: torch.Tensor, scales: torch.Tensor, scale2: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_mxfp4_linear over NVFP4 weights: scales [..., N, K/16] uint8 (E4M3) and scale2 [E]
    float32 ([1] dense), which multiplies the product before the bias.  The output
    never requires a gradient: moe_nvfp4_linear_backward computes it."""
    if _host is not None and stream is None and out is None:
        got = _host.linear(False, 16, x, blocks, scales, scale2, bias, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_nvfp4_linear(x, blocks, scales, scale2, bias, expert_offsets, out)
    return _linear("moe_nvfp4_linear", True, 16, x, blocks, scales, scale2, bias, expert_offsets, out)


def moe_mxfp4_linear_backward(dy: torch.Tensor, blocks: torch.Tensor, scales: torch.Tensor,
                              expert_offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Gradient of moe_mxfp4_linear to its rows: dx = dy W for dy [R, N] bfloat16 (weights and
    offsets as there; the weights are frozen).  Returns dx [R, K]."""
    if _host is not None and stream is None and out is None:
        got = _host.linear(True, 32, dy, blocks, scales, None, None, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(dy, stream):
        with _place(dy, stream):
            return moe_mxfp4_linear_backward(dy, blocks, scales, expert_offsets, out)
    return _linear("moe_mxfp4_linear_backward", False, 32, dy, blocks, scales, None, None, expert_offsets, out)


def moe_nvfp4_linear_backward(dy: torch.Tensor, blocks: torch.Tensor, scales: torch.Tensor, scale2: torch.Tensor,
                              expert_offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Gradient of moe_nvfp4_linear to its rows: dx = scale2 * (dy W).  Returns dx [R, K]."""
    if _host is not None and stream is None and out is None:
        got = _host.linear(True, 16, dy, blocks, scales, scale2, None, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(dy, stream):
        with _place(dy, stream):
            return moe_nvfp4_linear_backward(dy, blocks, scales, scale2, expert_offsets, out)
    return _linear("moe_nvfp4_linear_backward", False, 16, dy, blocks, scales, scale2, None, expert_offsets, out)


# ---- what stands around the expert products: the norm, rows and weights in 8 bits, the activation, the
# balance loss.  As the operators above they record nothing for autograd.

_E4M3 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    """Blocks of 128 elements that share a scale."""
    return (n + 127) // 128


def _workspace(fn, like: torch.Tensor, *args) -> tuple:
    """(workspace tensor, its size as an argument) of a call that answers with its size first."""
    n = ctypes.c_size_t(0)
    _raise(f"{fn.__name__}(workspace query)", fn(*args, None, ctypes.byref(n), None))
    return like.new_empty((max(n.value, 1),), dtype=torch.uint8), n


def _out(out, name: str, dtype: torch.dtype, shape, like: torch.Tensor, *inputs) -> torch.Tensor:
    """The caller's output after its checks, or a new one."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _check_on(out, name, dtype, shape, like.device)
    _apart(out, name, *inputs)
    return out


def _norm_inputs(x, weight, residual):
    """(element type, weight's, T, H) after the checks of the norm's inputs."""
    code = _element_type(x, "x")
    T, H = x.shape
    _check(x, "x", x.dtype)
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    _check_on(weight, "weight", torch.float32 if weight.dtype is torch.float32 else x.dtype, (H,), x.device)
    if residual is not None:
        _check_on(residual, "residual", x.dtype, (T, H), x.device)
    return code, _DTYPES[weight.dtype], T, H


def _ptr(t):
    return None if t is None else t.data_ptr()


def moe_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                 out: Optional[torch.Tensor] = None, summed: Optional[torch.Tensor] = None,
                 rstd: Optional[torch.Tensor] = None, stream=None):
    """The norm ahead of the layer: s = x + residual (rounded to x's type; x without a residual),
    y = s / sqrt(mean(s^2) + eps) * weight over the rows of x [T, H] (bfloat16, float16 or float32;
    weight [H] of x's type or float32).  Returns (y [T, H], s [T, H], rstd [T] float32); without a
    residual s is x itself.  s and rstd are what moe_rms_norm_backward takes; no output but x
    itself ever requires a gradient."""
    if _host is not None and stream is None and out is None and summed is None and rstd is None:
        got = _host.rms_norm(x, weight, residual, eps, False)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_rms_norm(x, weight, residual, eps, out, summed, rstd)
    code, wcode, T, H = _norm_inputs(x, weight, residual)
    out = _out(out, "out", x.dtype, (T, H), x, x, weight, residual)
    if residual is not None:
        summed = _out(summed, "summed", x.dtype, (T, H), x, x, weight, residual, out)
    elif summed is not None:
        raise ValueError("summed is written only with a residual")
    rstd = _out(rstd, "rstd", torch.float32, (T,), x, x, weight, residual, out, summed)
    st = load().moe_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), code, wcode, eps, T, H, _ptr(summed),
                             out.data_ptr(), rstd.data_ptr(), _current_stream(x))
    _raise("moe_rms_norm", st)
    return out, x if residual is None else summed, rstd


def moe_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-5, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                     summed: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None):
    """moe_rms_norm with its rows in 8 bits: returns (codes [T, H] float8_e4m3fn, scales
    [T, ceil(H / 128)] float32, s [T, H], rstd [T]), codes and scales as moe_fp8_quantize makes them
    of the norm's float32 values.  The gradient is moe_rms_norm_backward's: the rounding to 8 bits
    counts as none."""
    plain = codes is None and scales is None and summed is None and rstd is None
    if _host is not None and stream is None and plain:
        got = _host.rms_norm(x, weight, residual, eps, True)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_rms_norm_fp8(x, weight, residual, eps, codes, scales, summed, rstd)
    code, wcode, T, H = _norm_inputs(x, weight, residual)
    codes = _out(codes, "codes", _E4M3, (T, H), x, x, weight, residual)
    scales = _out(scales, "scales", torch.float32, (T, _blocks(H)), x, x, weight, residual, codes)
    if residual is not None:
        summed = _out(summed, "summed", x.dtype, (T, H), x, x, weight, residual, codes, scales)
    elif summed is not None:
        raise ValueError("summed is written only with a residual")
    rstd = _out(rstd, "rstd", torch.float32, (T,), x, x, weight, residual, codes, scales, summed)
    st = load().moe_rms_norm_fp8(x.data_ptr(), _ptr(residual), weight.data_ptr(), code, wcode, eps, T, H,
                                 _ptr(summed), codes.data_ptr(), scales.data_ptr(), rstd.data_ptr(),
                                 _current_stream(x))
    _raise("moe_rms_norm_fp8", st)
    return codes, scales, x if residual is None else summed, rstd


def moe_rms_norm_backward(dy: torch.Tensor, summed: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          d_summed: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                          d_weight: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_rms_norm and moe_rms_norm_fp8 for dy [T, H]: (dx [T, H], d_weight [H] float32).
    dx is the gradient of x and of the residual alike; d_summed [T, H] is what reaches s past the
    norm (the residual stream's gradient) and is added to it."""
    if _host is not None and stream is None and dx is None and d_weight is None:
        got = _host.rms_norm_backward(dy, summed, weight, rstd, d_summed)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(dy, stream):
        with _place(dy, stream):
            return moe_rms_norm_backward(dy, summed, weight, rstd, d_summed, dx, d_weight)
    code = _element_type(dy, "dy")
    T, H = dy.shape
    _check(dy, "dy", dy.dtype)
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    _check_on(summed, "summed", dy.dtype, (T, H), dy.device)
    _check_on(weight, "weight", torch.float32 if weight.dtype is torch.float32 else dy.dtype, (H,), dy.device)
    _check_on(rstd, "rstd", torch.float32, (T,), dy.device)
    if d_summed is not None:
        _check_on(d_summed, "d_summed", dy.dtype, (T, H), dy.device)
    dx = _out(dx, "dx", dy.dtype, (T, H), dy, dy, summed, weight, rstd, d_summed)
    d_weight = _out(d_weight, "d_weight", torch.float32, (H,), dy, dy, summed, weight, rstd, d_summed, dx)
    fn = load().moe_rms_norm_backward
    wcode = _DTYPES[weight.dtype]
    workspace, n = _workspace(fn, dy, None, None, None, None, code, wcode, None, T, H, None, None)
    st = fn(dy.data_ptr(), _ptr(d_summed), summed.data_ptr(), weight.data_ptr(), code, wcode, rstd.data_ptr(), T, H,
            dx.data_ptr(), d_weight.data_ptr(), workspace.data_ptr(), ctypes.byref(n), _current_stream(dy))
    _raise("moe_rms_norm_backward", st)
    return dx, d_weight


def moe_fp8_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                     stream=None):
    """Rows [R, K] (bfloat16, float16 or float32) in 8 bits: (codes [R, K] float8_e4m3fn, scales
    [R, ceil(K / 128)] float32), scale = largest magnitude of 128 elements / 448 and code = element /
    scale to nearest.  (moe_permute moves such rows too, as the two-byte type of half their width:
    codes.view(torch.float16).)"""
    if _host is not None and stream is None and codes is None and scales is None:
        got = _host.fp8_quantize(x)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_fp8_quantize(x, codes, scales)
    code = _element_type(x, "x")
    R, K = x.shape
    _check(x, "x", x.dtype)
    codes = _out(codes, "codes", _E4M3, (R, K), x, x)
    scales = _out(scales, "scales", torch.float32, (R, _blocks(K)), x, x, codes)
    st = load().moe_fp8_quantize(x.data_ptr(), code, R, K, codes.data_ptr(), scales.data_ptr(), _current_stream(x))
    _raise("moe_fp8_quantize", st)
    return codes, scales


def _fp8_weights(rows, name: str, row_type: torch.dtype, weight, weight_scales, bias, expert_offsets):
    """(E, N, K) of an 8-bit linear operator, after the checks of every tensor but the rows' width."""
    if not isinstance(rows, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError(f"{name} and weight must be torch.Tensors")
    lead = 2 if expert_offsets is None else 3
    shape = weight.shape
    if rows.dim() != 2:
        raise ValueError(f"{name} has {rows.dim()} dimensions, expected 2")
    if len(shape) != lead:
        raise ValueError(f"weight has {len(shape)} dimensions, expected {lead} "
                         f"{'without' if lead == 2 else 'with'} expert_offsets")
    E = 1 if lead == 2 else shape[0]
    N, K = shape[-2:]
    dev = rows.device
    _check(rows, name, row_type)
    _check_on(weight, "weight", _E4M3, shape, dev)
    _check_on(weight_scales, "weight_scales", torch.float32, (*shape[:-2], _blocks(N), _blocks(K)), dev)
    if expert_offsets is not None:
        _check_on(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev)
    if bias is not None:
        _check_on(bias, "bias", torch.bfloat16, shape[:-1], dev)
    return E, N, K


def moe_fp8_linear(x: torch.Tensor, x_scales: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows in 8 bits times 8-bit weights with a scale for each block of 128: y = x W^T (+ bias).
    x [R, K] float8_e4m3fn with x_scales [R, ceil(K / 128)] float32, as moe_fp8_quantize and the _fp8
    calls make them.  Dense: weight [N, K] float8_e4m3fn, weight_scales [ceil(N / 128), ceil(K / 128)]
    float32, bias [N] bfloat16.  Per expert: weight [E, N, K], weight_scales [E, ., .], bias [E, N] and
    expert_offsets [E + 1] int32 as in moe_mxfp4_linear (rows of no expert keep what `out` held, and
    without `out` hold anything).  K is a multiple of 16.  Returns y [R, N] bfloat16, which never
    requires a gradient: moe_fp8_linear_backward computes it."""
    if _host is not None and stream is None and out is None:
        got = _host.fp8_linear(x, x_scales, weight, weight_scales, bias, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(x, stream):
        with _place(x, stream):
            return moe_fp8_linear(x, x_scales, weight, weight_scales, bias, expert_offsets, out)
    E, N, K = _fp8_weights(x, "x", _E4M3, weight, weight_scales, bias, expert_offsets)
    R, width = x.shape
    if width != K:
        raise ValueError(f"x has rows of {width}, expected {K}")
    _check_on(x_scales, "x_scales", torch.float32, (R, _blocks(K)), x.device)
    out = _out(out, "out", torch.bfloat16, (R, N), x, x, x_scales, weight, weight_scales, bias, expert_offsets)
    st = load().moe_fp8_linear(x.data_ptr(), x_scales.data_ptr(), weight.data_ptr(), weight_scales.data_ptr(),
                               _ptr(bias), _ptr(expert_offsets), R, K, N, E, out.data_ptr(), _current_stream(x))
    _raise("moe_fp8_linear", st)
    return out


def moe_fp8_linear_backward(dy: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                            expert_offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Gradient of moe_fp8_linear to its rows (as they were before they went to 8 bits): dx = dy W for
    dy [R, N] bfloat16 (weights and offsets as there; the weights are frozen).  Returns dx [R, K]
    bfloat16."""
    if _host is not None and stream is None and out is None:
        got = _host.fp8_linear_backward(dy, weight, weight_scales, expert_offsets)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(dy, stream):
        with _place(dy, stream):
            return moe_fp8_linear_backward(dy, weight, weight_scales, expert_offsets, out)
    E, N, K = _fp8_weights(dy, "dy", torch.bfloat16, weight, weight_scales, None, expert_offsets)
    R, width = dy.shape
    if width != N:
        raise ValueError(f"dy has rows of {width}, expected {N}")
    out = _out(out, "out", torch.bfloat16, (R, K), dy, dy, weight, weight_scales, expert_offsets)
    st = load().moe_fp8_linear_backward(dy.data_ptr(), weight.data_ptr(), weight_scales.data_ptr(),
                                        _ptr(expert_offsets), R, K, N, E, out.data_ptr(), _current_stream(dy))
    _raise("moe_fp8_linear_backward", st)
    return out


def _pairs_of(h):
    """(element type, R, I) of rows of gates and ups."""
    code = _element_type(h, "h")
    R, width = h.shape
    if width % 2:
        raise ValueError(f"h has rows of {width}, not of gates and ups")
    _check(h, "h", h.dtype)
    return code, R, width // 2


def moe_swiglu(h: torch.Tensor, split: bool = False, alpha: float = 1.702, limit: float = 7.0, offset: float = 1.0,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' activation: a = g sigmoid(alpha g) (u + offset) with g = min(gate, limit) and
    u = clamp(up, -limit, limit) for h [R, 2 I] (bfloat16, float16 or float32), gate and up side by
    side or, with split, in two halves of a row.  The defaults are the fused layer's; the plain gated
    SiLU is alpha=1, limit=math.inf, offset=0.  Returns a [R, I], which never requires a gradient:
    moe_swiglu_backward computes it."""
    if _host is not None and stream is None and out is None:
        got = _host.swiglu(h, split, alpha, limit, offset, False)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(h, stream):
        with _place(h, stream):
            return moe_swiglu(h, split, alpha, limit, offset, out)
    code, R, I = _pairs_of(h)
    out = _out(out, "out", h.dtype, (R, I), h, h)
    st = load().moe_swiglu(h.data_ptr(), code, R, I, alpha, limit, offset, 1 if split else 0, out.data_ptr(),
                           _current_stream(h))
    _raise("moe_swiglu", st)
    return out


def moe_swiglu_fp8(h: torch.Tensor, split: bool = False, alpha: float = 1.702, limit: float = 7.0,
                   offset: float = 1.0, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                   stream=None):
    """moe_swiglu with its rows in 8 bits: returns (codes [R, I] float8_e4m3fn, scales [R, ceil(I / 128)]
    float32) as moe_fp8_quantize makes them of the activation's float32 values.  The gradient is
    moe_swiglu_backward's: the rounding to 8 bits counts as none."""
    if _host is not None and stream is None and codes is None and scales is None:
        got = _host.swiglu(h, split, alpha, limit, offset, True)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(h, stream):
        with _place(h, stream):
            return moe_swiglu_fp8(h, split, alpha, limit, offset, codes, scales)
    code, R, I = _pairs_of(h)
    codes = _out(codes, "codes", _E4M3, (R, I), h, h)
    scales = _out(scales, "scales", torch.float32, (R, _blocks(I)), h, h, codes)
    st = load().moe_swiglu_fp8(h.data_ptr(), code, R, I, alpha, limit, offset, 1 if split else 0, codes.data_ptr(),
                               scales.data_ptr(), _current_stream(h))
    _raise("moe_swiglu_fp8", st)
    return codes, scales


def moe_swiglu_backward(da: torch.Tensor, h: torch.Tensor, split: bool = False, alpha: float = 1.702,
                        limit: float = 7.0, offset: float = 1.0, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Gradient of moe_swiglu and moe_swiglu_fp8 for da [R, I] (h's type): dh [R, 2 I] in h's layout, 0
    for gates past the limit and ups past the limits."""
    if _host is not None and stream is None and out is None:
        got = _host.swiglu_backward(da, h, split, alpha, limit, offset)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(h, stream):
        with _place(h, stream):
            return moe_swiglu_backward(da, h, split, alpha, limit, offset, out)
    code, R, I = _pairs_of(h)
    _check_on(da, "da", h.dtype, (R, I), h.device)
    out = _out(out, "out", h.dtype, (R, 2 * I), h, h, da)
    st = load().moe_swiglu_backward(da.data_ptr(), h.data_ptr(), code, R, I, alpha, limit, offset, 1 if split else 0,
                                    out.data_ptr(), _current_stream(h))
    _raise("moe_swiglu_backward", st)
    return out


def _logits_of(router_logits, token_mask):
    """(T, E) after the checks of the logits and the mask."""
    if not isinstance(router_logits, torch.Tensor):
        raise TypeError("router_logits must be a torch.Tensor")
    if router_logits.dim() != 2:
        raise ValueError(f"router_logits has {router_logits.dim()} dimensions, expected 2")
    T, E = router_logits.shape
    _check(router_logits, "router_logits", torch.float32)
    if token_mask is not None:
        _check_on(token_mask, "token_mask", torch.bool, (T,), router_logits.device)
    return T, E


def moe_balance_loss(router_logits: torch.Tensor, topk_ids: torch.Tensor, token_mask: Optional[torch.Tensor] = None,
                     stream=None):
    """The router's balance loss: E * sum over experts of (its share of the picks) * (its mean
    probability), over the tokens whose token_mask [T] (bool) is True (None: every token).
    router_logits [T, E] float32, topk_ids [T, top_k] int32.  Returns (loss [] float32, counts [E]
    int32, density [E] float32): the picks of every expert, and what moe_balance_loss_backward takes.
    No output ever requires a gradient."""
    if _host is not None and stream is None:
        got = _host.balance_loss(router_logits, topk_ids, token_mask)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(router_logits, stream):
        with _place(router_logits, stream):
            return moe_balance_loss(router_logits, topk_ids, token_mask)
    T, E = _logits_of(router_logits, token_mask)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be a tensor of two dimensions")
    top_k = topk_ids.shape[1]
    _check_on(topk_ids, "topk_ids", torch.int32, (T, top_k), router_logits.device)
    loss, density = router_logits.new_empty(()), router_logits.new_empty((E,))
    counts = topk_ids.new_empty((E,))
    fn = load().moe_balance_loss
    workspace, n = _workspace(fn, router_logits, None, None, None, T, E, top_k, None, None, None)
    st = fn(router_logits.data_ptr(), topk_ids.data_ptr(), _ptr(token_mask), T, E, top_k, loss.data_ptr(),
            counts.data_ptr(), density.data_ptr(), workspace.data_ptr(), ctypes.byref(n),
            _current_stream(router_logits))
    _raise("moe_balance_loss", st)
    return loss, counts, density


def moe_balance_loss_backward(router_logits: torch.Tensor, density: torch.Tensor, d_loss: torch.Tensor,
                              token_mask: Optional[torch.Tensor] = None, add_to: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_balance_loss to the logits, [T, E] float32, for d_loss (a float32 device tensor
    of one element) and density [E] as moe_balance_loss made it; added to add_to [T, E] where that is
    given (moe_route_backward's gradient of the same logits).  out may be add_to itself."""
    if _host is not None and stream is None and out is None:
        got = _host.balance_loss_backward(router_logits, density, d_loss, token_mask, add_to)
        if got is not None:  # None: not a plain call, or one to refuse
            return got
    if _elsewhere(router_logits, stream):
        with _place(router_logits, stream):
            return moe_balance_loss_backward(router_logits, density, d_loss, token_mask, add_to, out)
    T, E = _logits_of(router_logits, token_mask)
    dev = router_logits.device
    _check_on(density, "density", torch.float32, (E,), dev)
    if not isinstance(d_loss, torch.Tensor) or d_loss.numel() != 1:
        raise ValueError("d_loss must be a tensor of one element")
    _check_on(d_loss, "d_loss", torch.float32, d_loss.shape, dev)
    if add_to is not None:
        _check_on(add_to, "add_to", torch.float32, (T, E), dev)
    same = out is not None and add_to is not None and out.data_ptr() == add_to.data_ptr()
    out = _out(out, "out", torch.float32, (T, E), router_logits, router_logits, density, d_loss, token_mask,
               None if same else add_to)
    st = load().moe_balance_loss_backward(router_logits.data_ptr(), density.data_ptr(), d_loss.data_ptr(),
                                          _ptr(token_mask), _ptr(add_to), T, E, out.data_ptr(),
                                          _current_stream(router_logits))
    _raise("moe_balance_loss_backward", st)
    return out


def profile_begin(stage: str, max_calls: int) -> None:
    """Record HIP events around the next ``max_calls`` launches of one kernel stage."""
    st = load().mxfp4moe_profile_begin(STAGES[stage], max_calls)
    _raise("mxfp4moe_profile_begin", st)


def profile_end(capacity: int):
    """Per-launch durations (ms) recorded since profile_begin."""
    buf = (ctypes.c_float * max(capacity, 1))()
    n = load().mxfp4moe_profile_end(buf, capacity)
    if n < 0:
        raise MXFP4MoEError("mxfp4moe_profile_end", n)
    return [float(buf[i]) for i in range(n)]


def layer_to_device(layer, device="cuda"):
    """Host numpy layer (workloads.make_layer) -> device tensors with the binding's dtypes."""
    import numpy as np

    def dev(a, dtype):
        a = np.ascontiguousarray(a)
        if dtype == torch.bfloat16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
        return torch.from_numpy(a).to(device)

    out = {
        "x": dev(layer["x"], torch.bfloat16),
        "router_logits": dev(layer["router_logits"], torch.float32),
        "w13_blocks": dev(layer["w13_blocks"], torch.uint8),
        "w13_scales": dev(layer["w13_scales"], torch.uint8),
        "w13_bias": dev(layer["w13_bias"], torch.bfloat16),
        "w2_blocks": dev(layer["w2_blocks"], torch.uint8),
        "w2_scales": dev(layer["w2_scales"], torch.uint8),
        "w2_bias": dev(layer["w2_bias"], torch.bfloat16),
    }
    for k in ("w13_scale2", "w2_scale2"):  # NVFP4 layers
        if k in layer:
            out[k] = dev(np.asarray(layer[k], dtype=np.float32), torch.float32)
    for k in ("router_w", "router_b"):  # layers with a router projection
        if k in layer:
            out[k] = dev(layer[k], torch.bfloat16)
    return out
