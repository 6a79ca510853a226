"""FP8 block-scaled linear-layer path for NVIDIA GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/fp8bs.h`` (``libfp8bs.so``, built in place
by ``fp8_block_scaled_fp8bs_gb300.build``). Every step of the path runs in the library's CUDA
kernels; this module only marshals arguments (those of the decoder-layer operators in compiled
code, ``csrc/host.cpp``: their smallest calls take a few microseconds). There is no CPU fallback: if the library is
missing or cannot be loaded, importing the binding's functions raises.

Raw entry points (same names and arguments as the C functions; pointers are ints):
    fp8bs_act_quant(x, y, s, M, K, scale_fmt, stream)
    fp8bs_weight_dequant(w, s, y, N, K, stream)
    fp8bs_gemm(a, a_s, b, b_s, c, M, N, K, scale_fmt, stream)
    fp8bs_gemm_ex(a, a_s, b, b_s, c, M, N, K, scale_fmt, flags, stream)
    fp8bs_gemm_plan(M, N, K, scale_fmt, with_workspace) -> dict
    fp8bs_gemm_config(a, a_s, b, b_s, c, M, N, K, scale_fmt, flags, kernel, tile, ksplit,
                      workspace, workspace_bytes, stream)
    fp8bs_gemm_grouped(a, a_s, b, b_s, c, row_offsets, groups, N, K, scale_fmt, stream)
    fp8bs_device_error(clear=True, stream=0) -> int
    fp8bs_probe_wait_timeout(timeout_ns, stream)
    fp8bs_qk_norm_rope(args, stream), fp8bs_paged_attention(args, stream),
    fp8bs_qk_norm_rope_fp8(args, k_scale, v_scale, stream),
    fp8bs_paged_attention_fp8(args, k_scale, v_scale, stream), fp8bs_rms_norm(args, stream),
    fp8bs_moe_route / _experts / _layer: argument structures QkNormRopeArgs, PagedAttentionArgs,
        RmsNormArgs, MoeRouting with the C structures' fields
Tensor conveniences (PyTorch CUDA tensors; outputs allocated with torch):
    act_quant(x, scale_fmt="fp32") -> (y, s)      ("DeepSeek-V3 Administrator & Developer
    weight_dequant(w, s) -> y                        Guide", §8.5.1, §8.5.2, §8.5.3)
    fp8_gemm(a, a_s, b, b_s, scale_fmt="fp32") -> c
    fp8_gemm_grouped(a, a_s, b, b_s, row_offsets, scale_fmt="fp32") -> c
    rms_norm(x, weight, ...) -> NormOut(y, s, n, h)
    qk_norm_rope(q, k, cos, sin, positions, ...) -> q (and k, or the keys and values in a PagedCache or
        PagedCacheFp8)
    paged_attention(q, cache, page_table, q_start, kv_len, ...) -> out (and lse)
    moe_route(x, router_w, ...) -> (weights, ids)      ("DeepSeek-V3 Administrator & Developer
    moe_experts(x, weights, ids, w13, s13, w2, s2) -> y    Guide", §6.4)
    moe_layer(x, router_w, w13, s13, w2, s2, ...) -> y
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Any, NamedTuple

BLOCK = 128
SCALE_FP32 = 0
SCALE_UE8M0 = 1
STATUS = {0: "ok", 1: "invalid argument", 2: "pointer not aligned",
          3: "unsupported device (needs sm_103)", 4: "CUDA error"}
DEVERR_SCALE_NOT_POW2 = 0x10
DEVERR_INDEX = 0x20
DEVERR_PROBE = 0x100

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8bs.so")
GEMM_WEIGHTS_CONSTANT = 0x1
GEMM_QUANT_IN_KERNEL = 0x2
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
MOE_MAX_TOKENS = 64
KERNEL_SWAPPED, KERNEL_PROMOTED, KERNEL_BLOCK_SCALED, KERNEL_BLOCK_SCALED_PAIR = 0, 1, 2, 3
EXPORTS = ("fp8bs_act_quant", "fp8bs_weight_dequant", "fp8bs_gemm", "fp8bs_gemm_ex",
           "fp8bs_gemm_ws", "fp8bs_gemm_workspace_size", "fp8bs_gemm_plan", "fp8bs_gemm_config",
           "fp8bs_gemm_noalloc",
           "fp8bs_act_quant_gemm", "fp8bs_linear_bf16",
           "fp8bs_gemm_grouped",
           "fp8bs_qk_norm_rope", "fp8bs_paged_attention", "fp8bs_paged_attention_workspace_size",
           "fp8bs_qk_norm_rope_fp8", "fp8bs_paged_attention_fp8",
           "fp8bs_paged_attention_fp8_workspace_size", "fp8bs_rms_norm",
           "fp8bs_moe_route", "fp8bs_moe_experts", "fp8bs_moe_layer", "fp8bs_moe_workspace_size",
           "fp8bs_status_string", "fp8bs_device_error", "fp8bs_probe_wait_timeout",
           "fp8bs_probe_occupy")

_lock = threading.Lock()
_lib = None


def _structure(name, doc, **fields):
    return type(name, (ctypes.Structure,), {"_fields_": list(fields.items()), "__doc__": doc,
                                            "__slots__": ()})


_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
KvCache = _structure(
    "KvCache", "fp8bs_kv_cache", k=_vp, v=_vp, pages=_i64, page_size=_i64, heads=_i64, dk=_i64,
    dv=_i64, k_page_stride=_i64, k_slot_stride=_i64, k_head_stride=_i64, v_page_stride=_i64,
    v_slot_stride=_i64, v_head_stride=_i64)
QkNormRopeArgs = _structure(
    "QkNormRopeArgs", "fp8bs_qk_norm_rope_args", q=_vp, k=_vp, v=_vp, q_token_stride=_i64,
    q_head_stride=_i64, k_token_stride=_i64, k_head_stride=_i64, v_token_stride=_i64,
    v_head_stride=_i64, q_weight=_vp, k_weight=_vp, cos=_vp, sin=_vp, positions=_vp, slots=_vp,
    q_out=_vp, cache=KvCache, T=_i64, q_heads=_i64, max_positions=_i64, rot_start=_i64,
    rot_dim=_i64, interleaved=ctypes.c_int, eps=ctypes.c_float)
PagedAttentionArgs = _structure(
    "PagedAttentionArgs", "fp8bs_paged_attention_args", q=_vp, q_token_stride=_i64,
    q_head_stride=_i64, cache=KvCache, page_table=_vp, table_stride=_i64, q_start=_vp, kv_len=_vp,
    out=_vp, lse=_vp, B=_i64, T=_i64, q_heads=_i64, max_q_len=_i64, max_kv_len=_i64, window=_i64,
    causal=ctypes.c_int, scale=ctypes.c_float, workspace=_vp, workspace_bytes=ctypes.c_size_t)
RmsNormArgs = _structure(
    "RmsNormArgs", "fp8bs_rms_norm_args", x=_vp, residual=_vp, weight=_vp, residual_out=_vp,
    norm_out=_vp, y=_vp, s=_vp, x_stride=_i64, residual_stride=_i64, T=_i64, D=_i64,
    scale_fmt=ctypes.c_int, eps=ctypes.c_float)
MoeRouting = _structure(
    "MoeRouting", "fp8bs_moe_routing", router_w=_vp, bias=_vp, top_k=_i64, groups=_i64,
    topk_groups=_i64, score=ctypes.c_int, normalise=ctypes.c_int, route_scale=ctypes.c_float)


class Fp8bsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} (status {status})")
        self.status = status


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libfp8bs.so (building it first if it is missing and nvcc is available)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            from . import build as _build
            _build.build()
        lib = ctypes.CDLL(p)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.fp8bs_act_quant.argtypes = [vp, vp, vp, i64, i64, i32, vp]
        lib.fp8bs_weight_dequant.argtypes = [vp, vp, vp, i64, i64, vp]
        lib.fp8bs_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
        lib.fp8bs_gemm_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.c_uint, vp]
        lib.fp8bs_gemm_ws.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.c_uint, vp,
                                      ctypes.c_size_t, vp]
        lib.fp8bs_gemm_workspace_size.argtypes = [ctypes.POINTER(ctypes.c_size_t)]
        ip = ctypes.POINTER(ctypes.c_int)
        lib.fp8bs_gemm_plan.argtypes = [i64, i64, i64, i32, i32, ip, ip, ip, ip]
        lib.fp8bs_gemm_config.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.c_uint,
                                          i32, i32, i32, vp, ctypes.c_size_t, vp]
        lib.fp8bs_linear_bf16.argtypes = [vp, vp, vp, vp, i64, i64, i64, ctypes.c_uint, vp]
        lib.fp8bs_act_quant_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32,
                                             ctypes.c_uint, vp, ctypes.c_size_t, vp]
        lib.fp8bs_gemm_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.c_uint,
                                           vp]
        lib.fp8bs_gemm_grouped.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int64),
                                           i64, i64, i64, i32, vp]
        lib.fp8bs_qk_norm_rope.argtypes = [ctypes.POINTER(QkNormRopeArgs), vp]
        lib.fp8bs_paged_attention.argtypes = [ctypes.POINTER(PagedAttentionArgs), vp]
        lib.fp8bs_paged_attention_workspace_size.argtypes = [ctypes.POINTER(PagedAttentionArgs),
                                                             ctypes.POINTER(ctypes.c_size_t)]
        lib.fp8bs_qk_norm_rope_fp8.argtypes = [ctypes.POINTER(QkNormRopeArgs), vp, vp, vp]
        lib.fp8bs_paged_attention_fp8.argtypes = [ctypes.POINTER(PagedAttentionArgs), vp, vp, vp]
        lib.fp8bs_paged_attention_fp8_workspace_size.argtypes = [ctypes.POINTER(PagedAttentionArgs),
                                                                 ctypes.POINTER(ctypes.c_size_t)]
        lib.fp8bs_rms_norm.argtypes = [ctypes.POINTER(RmsNormArgs), vp]
        lib.fp8bs_moe_workspace_size.argtypes = [i64] * 5 + [ctypes.POINTER(ctypes.c_size_t)]
        lib.fp8bs_moe_route.argtypes = [vp, ctypes.POINTER(MoeRouting), vp, vp, i64, i64, i64, vp]
        lib.fp8bs_moe_experts.argtypes = [vp] * 8 + [i64] * 5 + [i32, vp, ctypes.c_size_t, vp]
        lib.fp8bs_moe_layer.argtypes = [vp, ctypes.POINTER(MoeRouting)] + [vp] * 5 + [i64] * 4 + \
            [i32, vp, ctypes.c_size_t, vp]
        lib.fp8bs_status_string.argtypes = [i32]
        lib.fp8bs_status_string.restype = ctypes.c_char_p
        lib.fp8bs_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), i32, vp]
        lib.fp8bs_probe_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.fp8bs_probe_occupy.argtypes = [i32, ctypes.c_uint64, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = getattr(lib, name).restype or i32
        lib.fp8bs_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise Fp8bsError(fn, status)


# ----------------------------------------------------------------------- raw entry points

def fp8bs_act_quant(x, y, s, M, K, scale_fmt=SCALE_FP32, stream=0) -> None:
    _check("fp8bs_act_quant", load().fp8bs_act_quant(x, y, s, M, K, scale_fmt, stream))


def fp8bs_weight_dequant(w, s, y, N, K, stream=0) -> None:
    _check("fp8bs_weight_dequant", load().fp8bs_weight_dequant(w, s, y, N, K, stream))


def fp8bs_gemm(a, a_s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, stream=0) -> None:
    _check("fp8bs_gemm", load().fp8bs_gemm(a, a_s, b, b_s, c, M, N, K, scale_fmt, stream))


def fp8bs_gemm_ex(a, a_s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, flags=0, stream=0) -> None:
    _check("fp8bs_gemm_ex", load().fp8bs_gemm_ex(a, a_s, b, b_s, c, M, N, K, scale_fmt, flags,
                                                 stream))


def fp8bs_gemm_ws(a, a_s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, flags=0, workspace=0,
                  workspace_bytes=0, stream=0) -> None:
    _check("fp8bs_gemm_ws", load().fp8bs_gemm_ws(a, a_s, b, b_s, c, M, N, K, scale_fmt, flags,
                                                 workspace, workspace_bytes, stream))


def fp8bs_gemm_noalloc(a, a_s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, flags=0,
                       stream=0) -> None:
    _check("fp8bs_gemm_noalloc", load().fp8bs_gemm_noalloc(a, a_s, b, b_s, c, M, N, K,
                                                           scale_fmt, flags, stream))


def fp8bs_act_quant_gemm(x, y, s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, flags=0,
                         workspace=0, workspace_bytes=0, stream=0) -> None:
    _check("fp8bs_act_quant_gemm", load().fp8bs_act_quant_gemm(
        x, y, s, b, b_s, c, M, N, K, scale_fmt, flags, workspace, workspace_bytes, stream))


def fp8bs_linear_bf16(x, w, w_s, y, M, N, K, flags=0, stream=0) -> None:
    _check("fp8bs_linear_bf16", load().fp8bs_linear_bf16(x, w, w_s, y, M, N, K, flags, stream))


def fp8bs_gemm_workspace_size() -> int:
    out = ctypes.c_size_t(0)
    _check("fp8bs_gemm_workspace_size", load().fp8bs_gemm_workspace_size(ctypes.byref(out)))
    return out.value


def fp8bs_gemm_plan(M, N, K, scale_fmt=SCALE_FP32, with_workspace=True) -> dict:
    """The kernel, tile, K split and stream-K choice fp8bs_gemm_ws (with_workspace) or
    fp8bs_gemm_ex would make for this shape on the current device."""
    out = [ctypes.c_int(0) for _ in range(4)]
    _check("fp8bs_gemm_plan", load().fp8bs_gemm_plan(M, N, K, scale_fmt, int(with_workspace),
                                                     *[ctypes.byref(o) for o in out]))
    return {"kernel": out[0].value, "tile": out[1].value, "ksplit": out[2].value,
            "stream_k": bool(out[3].value)}


def fp8bs_gemm_config(a, a_s, b, b_s, c, M, N, K, scale_fmt=SCALE_FP32, flags=0,
                      kernel=KERNEL_PROMOTED, tile=128, ksplit=1, workspace=0, workspace_bytes=0,
                      stream=0) -> None:
    _check("fp8bs_gemm_config", load().fp8bs_gemm_config(
        a, a_s, b, b_s, c, M, N, K, scale_fmt, flags, kernel, tile, ksplit, workspace,
        workspace_bytes, stream))


def fp8bs_gemm_grouped(a, a_s, b, b_s, c, row_offsets, groups, N, K, scale_fmt=SCALE_FP32,
                       stream=0) -> None:
    """row_offsets: a sequence of groups+1 ints (host memory)."""
    offs = (ctypes.c_int64 * (int(groups) + 1))(*[int(x) for x in row_offsets])
    _check("fp8bs_gemm_grouped", load().fp8bs_gemm_grouped(a, a_s, b, b_s, c, offs, groups, N, K,
                                                           scale_fmt, stream))


def fp8bs_qk_norm_rope(args: QkNormRopeArgs, stream=0) -> None:
    _check("fp8bs_qk_norm_rope", load().fp8bs_qk_norm_rope(ctypes.byref(args), stream))


def fp8bs_paged_attention(args: PagedAttentionArgs, stream=0) -> None:
    _check("fp8bs_paged_attention", load().fp8bs_paged_attention(ctypes.byref(args), stream))


def fp8bs_paged_attention_workspace_size(args: PagedAttentionArgs) -> int:
    out = ctypes.c_size_t(0)
    _check("fp8bs_paged_attention_workspace_size",
           load().fp8bs_paged_attention_workspace_size(ctypes.byref(args), ctypes.byref(out)))
    return out.value


def fp8bs_qk_norm_rope_fp8(args: QkNormRopeArgs, k_scale, v_scale, stream=0) -> None:
    _check("fp8bs_qk_norm_rope_fp8",
           load().fp8bs_qk_norm_rope_fp8(ctypes.byref(args), k_scale, v_scale, stream))


def fp8bs_paged_attention_fp8(args: PagedAttentionArgs, k_scale, v_scale, stream=0) -> None:
    _check("fp8bs_paged_attention_fp8",
           load().fp8bs_paged_attention_fp8(ctypes.byref(args), k_scale, v_scale, stream))


def fp8bs_paged_attention_fp8_workspace_size(args: PagedAttentionArgs) -> int:
    out = ctypes.c_size_t(0)
    _check("fp8bs_paged_attention_fp8_workspace_size",
           load().fp8bs_paged_attention_fp8_workspace_size(ctypes.byref(args), ctypes.byref(out)))
    return out.value


def fp8bs_rms_norm(args: RmsNormArgs, stream=0) -> None:
    _check("fp8bs_rms_norm", load().fp8bs_rms_norm(ctypes.byref(args), stream))


def fp8bs_moe_workspace_size(T, D, I, experts, top_k) -> int:
    out = ctypes.c_size_t(0)
    _check("fp8bs_moe_workspace_size",
           load().fp8bs_moe_workspace_size(T, D, I, experts, top_k, ctypes.byref(out)))
    return out.value


def fp8bs_moe_route(x, routing: MoeRouting, weights, ids, T, D, experts, stream=0) -> None:
    _check("fp8bs_moe_route", load().fp8bs_moe_route(x, ctypes.byref(routing), weights, ids, T, D,
                                                     experts, stream))


def fp8bs_moe_experts(x, weights, ids, w13, s13, w2, s2, y, T, D, I, experts, top_k,
                      scale_fmt=SCALE_FP32, workspace=0, workspace_bytes=0, stream=0) -> None:
    _check("fp8bs_moe_experts", load().fp8bs_moe_experts(
        x, weights, ids, w13, s13, w2, s2, y, T, D, I, experts, top_k, scale_fmt, workspace,
        workspace_bytes, stream))


def fp8bs_moe_layer(x, routing: MoeRouting, w13, s13, w2, s2, y, T, D, I, experts,
                    scale_fmt=SCALE_FP32, workspace=0, workspace_bytes=0, stream=0) -> None:
    _check("fp8bs_moe_layer", load().fp8bs_moe_layer(
        x, ctypes.byref(routing), w13, s13, w2, s2, y, T, D, I, experts, scale_fmt, workspace,
        workspace_bytes, stream))


def fp8bs_device_error(clear: bool = True, stream=0) -> int:
    out = ctypes.c_uint(0)
    _check("fp8bs_device_error", load().fp8bs_device_error(ctypes.byref(out), int(clear), stream))
    return out.value


def fp8bs_probe_wait_timeout(timeout_ns: int, stream=0) -> None:
    _check("fp8bs_probe_wait_timeout", load().fp8bs_probe_wait_timeout(timeout_ns, stream))


def fp8bs_probe_occupy(ctas: int, duration_ns: int, stream=0) -> None:
    _check("fp8bs_probe_occupy", load().fp8bs_probe_occupy(ctas, duration_ns, stream))


# ----------------------------------------------------------------------- tensor helpers

def _fmt(scale_fmt) -> int:
    if scale_fmt in (SCALE_FP32, "fp32", None):
        return SCALE_FP32
    if scale_fmt in (SCALE_UE8M0, "ue8m0"):
        return SCALE_UE8M0
    raise ValueError(f"unknown scale_fmt {scale_fmt!r}")


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _require(t, dtype, ndim, name, host_ok=False):
    """t must be a contiguous CUDA tensor of dtype and rank ndim; with host_ok, a pinned host
    tensor is accepted too (the kernels that read x or write C reach pinned host memory in
    place)."""
    import torch
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or (host_ok and t.is_pinned())):
        raise TypeError(f"{name} must be a CUDA tensor" + (" or a pinned host tensor" if host_ok
                                                          else ""))
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def _output(out, shape, device):
    """The bf16 output: a new CUDA tensor, or the caller's `out` (CUDA or pinned host), checked
    to be a contiguous bf16 tensor of exactly `shape` so that no kernel writes past its end."""
    import torch
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    _require(out, torch.bfloat16, len(shape), "out", host_ok=True)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out.shape)}")
    return out


def _workspace_args(workspace):
    """(pointer, bytes) of a stream-K workspace: None, or a contiguous uint8 CUDA tensor (its
    size is checked by the library against fp8bs_gemm_workspace_size)."""
    import torch
    if workspace is None:
        return 0, 0
    _require(workspace, torch.uint8, workspace.dim() if isinstance(workspace, torch.Tensor) else 1,
             "workspace")
    return workspace.data_ptr(), workspace.numel()


def _cuda_device(*tensors):
    import torch
    for t in tensors:
        if t.is_cuda:
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def act_quant(x, scale_fmt="fp32"):
    """x: bf16 [M,K] (K % 128 == 0) -> (y float8_e4m3fn [M,K], s float32 [M,K/128])."""
    import torch
    _require(x, torch.bfloat16, 2, "x", host_ok=True)
    M, K = x.shape
    dev = _cuda_device(x)
    y = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty((M, K // BLOCK), dtype=torch.float32, device=dev)
    fp8bs_act_quant(x.data_ptr(), y.data_ptr(), s.data_ptr(), M, K, _fmt(scale_fmt), _stream())
    return y, s


def weight_dequant(w, s):
    """w: float8_e4m3fn [N,K], s: float32 [ceil(N/128), ceil(K/128)] -> bf16 [N,K]."""
    import torch
    _require(w, torch.float8_e4m3fn, 2, "w")
    _require(s, torch.float32, 2, "s")
    N, K = w.shape
    if tuple(s.shape) != (-(-N // BLOCK), -(-K // BLOCK)):
        raise ValueError(f"scale shape {tuple(s.shape)} does not match weight {tuple(w.shape)}")
    y = torch.empty((N, K), dtype=torch.bfloat16, device=w.device)
    fp8bs_weight_dequant(w.data_ptr(), s.data_ptr(), y.data_ptr(), N, K, _stream())
    return y


_workspaces = {}


def gemm_workspace(device=None, stream=None):
    """The zero-filled workspace fp8_gemm uses on `device` for calls on `stream` (one per
    device and stream, so that calls that may overlap never share one), allocated on first use."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    key = (dev.index, stream if stream is not None else _stream())
    ws = _workspaces.get(key)
    if ws is None:
        with torch.cuda.device(dev):
            ws = torch.zeros(fp8bs_gemm_workspace_size(), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def _auto_workspace(device, M, N, K, fmt):
    """The workspace of a call that leaves it to us: gemm_workspace's, or in a call that is being
    captured one of its own from the graph's memory, with the counters zeroed by the graph (they
    stand first; the partials behind them are written before they are read). A graph may be
    replayed beside others that were captured on the same stream, and a cached workspace must not
    wait for a replay for its zeros. None where the call would not use one."""
    import torch
    if not torch.cuda.is_current_stream_capturing():
        return gemm_workspace(device)
    if 0 in (M, N, K) or K % BLOCK or not fp8bs_gemm_plan(M, N, K, fmt, True)["stream_k"]:
        return None
    ws = torch.empty(fp8bs_gemm_workspace_size(), dtype=torch.uint8, device=device)
    ws[:4096].zero_()
    return ws


def fp8_gemm(a, a_s, b, b_s, scale_fmt="fp32", out=None, weights_constant=False,
             workspace="auto"):
    """C[M,N] bf16 = A[M,K] . B[N,K]^T with per-128-K-block scales a_s [M,K/128] and
    b_s [ceil(N/128), K/128]. workspace: "auto" (a cached one per device and stream; the
    graph's own in a call that is being captured), None (no split K loops) or a zero-filled uint8
    CUDA tensor of fp8bs_gemm_workspace_size() bytes."""
    import torch
    _require(a, torch.float8_e4m3fn, 2, "a")
    _require(b, torch.float8_e4m3fn, 2, "b")
    _require(a_s, torch.float32, 2, "a_s")
    _require(b_s, torch.float32, 2, "b_s")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or tuple(a_s.shape) != (M, K // BLOCK) or \
            tuple(b_s.shape) != (-(-N // BLOCK), K // BLOCK):
        raise ValueError("operand or scale shapes do not match")
    c = _output(out, (M, N), a.device)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = _auto_workspace(a.device, M, N, K, _fmt(scale_fmt))
    ws_ptr, ws_bytes = _workspace_args(workspace)
    fp8bs_gemm_ws(a.data_ptr(), a_s.data_ptr(), b.data_ptr(), b_s.data_ptr(), c.data_ptr(),
                  M, N, K, _fmt(scale_fmt), GEMM_WEIGHTS_CONSTANT if weights_constant else 0,
                  ws_ptr, ws_bytes, _stream())
    return c


def act_quant_gemm(x, b, b_s, scale_fmt="fp32", weights_constant=False, workspace="auto",
                   quant_in_kernel=False, out=None):
    """linear() on the FP8 path: x bf16 [M,K] -> (c bf16 [M,N], y e4m3 [M,K], s fp32
    [M,K/128]): act_quant then the GEMM (quant_in_kernel: one kernel, M <= 16); see fp8_gemm
    for `workspace`. x and `out` (c) may be pinned host tensors."""
    import torch
    _require(x, torch.bfloat16, 2, "x", host_ok=True)
    _require(b, torch.float8_e4m3fn, 2, "b")
    _require(b_s, torch.float32, 2, "b_s")
    M, K = x.shape
    N = b.shape[0]
    if b.shape[1] != K or tuple(b_s.shape) != (-(-N // BLOCK), K // BLOCK):
        raise ValueError("operand or scale shapes do not match")
    y = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=b.device)
    s = torch.empty((M, K // BLOCK), dtype=torch.float32, device=b.device)
    c = _output(out, (M, N), b.device)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = _auto_workspace(b.device, M, N, K, _fmt(scale_fmt))
    ws_ptr, ws_bytes = _workspace_args(workspace)
    flags = (GEMM_WEIGHTS_CONSTANT if weights_constant else 0) | \
        (GEMM_QUANT_IN_KERNEL if quant_in_kernel else 0)
    fp8bs_act_quant_gemm(x.data_ptr(), y.data_ptr(), s.data_ptr(), b.data_ptr(), b_s.data_ptr(),
                         c.data_ptr(), M, N, K, _fmt(scale_fmt), flags, ws_ptr, ws_bytes,
                         _stream())
    return c, y, s


def linear_bf16(x, w, w_s, weights_constant=False, out=None):
    """bf16 path of linear(): x bf16 [M,K] . bf16(dequant(w, w_s))^T -> y bf16 [M,N]."""
    import torch
    _require(x, torch.bfloat16, 2, "x")
    _require(w, torch.float8_e4m3fn, 2, "w")
    _require(w_s, torch.float32, 2, "w_s")
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or tuple(w_s.shape) != (-(-N // BLOCK), -(-K // BLOCK)):
        raise ValueError("operand or scale shapes do not match")
    y = _output(out, (M, N), x.device)
    fp8bs_linear_bf16(x.data_ptr(), w.data_ptr(), w_s.data_ptr(), y.data_ptr(), M, N, K,
                      GEMM_WEIGHTS_CONSTANT if weights_constant else 0, _stream())
    return y


def fp8_gemm_grouped(a, a_s, b, b_s, row_offsets, scale_fmt="fp32", out=None):
    """Per-group block-scaled GEMMs: a [T,K] e4m3 with rows grouped by row_offsets (groups+1
    host ints), b [G,N,K] e4m3, b_s [G, ceil(N/128), K/128] -> c [T,N] bf16."""
    import torch
    _require(a, torch.float8_e4m3fn, 2, "a")
    _require(b, torch.float8_e4m3fn, 3, "b")
    _require(a_s, torch.float32, 2, "a_s")
    _require(b_s, torch.float32, 3, "b_s")
    T, K = a.shape
    G, N = b.shape[0], b.shape[1]
    offs = [int(x) for x in row_offsets]
    if len(offs) != G + 1 or offs[0] != 0 or offs[-1] != T or b.shape[2] != K or \
            tuple(a_s.shape) != (T, K // BLOCK) or tuple(b_s.shape) != (G, -(-N // BLOCK), K // BLOCK):
        raise ValueError("operand, scale or offset shapes do not match")
    c = _output(out, (T, N), a.device)
    fp8bs_gemm_grouped(a.data_ptr(), a_s.data_ptr(), b.data_ptr(), b_s.data_ptr(), c.data_ptr(),
                       offs, G, N, K, _fmt(scale_fmt), _stream())
    return c


# ------------------------------------------------------------- around the products of a decoder layer
#
# These calls take a few microseconds on the GPU, so their host side (checks, outputs, workspaces) is compiled:
# csrc/host.cpp.

class PagedCache(NamedTuple):
    """Keys [pages, page_size, heads, dk] and values [pages, page_size, heads, dv], bf16 CUDA tensors
    (views of another order too: rows contiguous, the other strides multiples of 8)."""
    k: Any
    v: Any


class PagedCacheFp8(NamedTuple):
    """The same in 8 bits: e4m3 codes k [pages, page_size, heads, dk] and v [pages, page_size, heads, dv]
    (page_size and the strides multiples of 16), each page and head with one scale, fp32 [pages, heads]:
    a code stands for code * scale. The scales are powers of two that qk_norm_rope writes and lets grow
    with the page; zeros say that a page holds nothing yet. paged_attention takes value scales of 2^-80 to
    2^120, within 2^80 of one another among a query's keys."""
    k: Any
    v: Any
    k_scale: Any
    v_scale: Any


class NormOut(NamedTuple):
    """What rms_norm gives; None in the place of what was not asked for."""
    y: Any      # e4m3 [T, D]
    s: Any      # fp32 [T, D/128]
    n: Any      # bf16 [T, D]
    h: Any      # bf16 [T, D], x + residual


HOST_PATH = os.path.join(_HERE, "_host.so")
_host = None


def _load_host():
    """The compiled host side, built if it is missing or was made for another PyTorch."""
    global _host
    lib = load()
    with _lock:
        if _host is None:
            import importlib.util
            import torch  # noqa: F401  (its libraries have to be there first)
            from . import build as _build
            if not _build.host_fits():
                _build.build_host()
            spec = importlib.util.spec_from_file_location("_host", HOST_PATH)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.init(lib._handle, Fp8bsError)
            _host = module
    return _host


def rms_norm(x, weight, eps=1e-6, residual=None, quant=None, norm=None, residual_out=None):
    """RMS norm of x bf16 [T, D] (D a multiple of 128; rows may be strided) with weight bf16 [D], and what
    stands around it between two products, in one pass -> NormOut(y, s, n, h):
    h = x + residual (bf16 [T, D]; into residual_out, which may be x or the residual itself), which then is
    what is normalised; n, the norm in bf16, where no codes are asked for or norm is true; y and s, with
    quant "fp32" or "ue8m0", the norm's e4m3 codes and scales as act_quant's, from unrounded n."""
    if quant is not None:
        quant = _fmt(quant)
    return NormOut(*(_host or _load_host()).rms_norm(x, weight, eps, residual, quant, norm, residual_out))


def qk_norm_rope(q, k, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6, rot_start=0,
                 interleaved=False, cache=None, v=None, slots=None, out=None):
    """RMS norm per head (where a weight is given) and rotation of q bf16 [T, Hq, D] and k bf16
    [T, Hk, D] by positions int32 [T]; cos, sin fp32 [max_positions, R/2] rotate the channels
    rot_start .. rot_start+R-1. With a PagedCache, the keys and v bf16 [T, Hk, Dv] go to its slots
    int64 [T] (negative: not written) and q bf16 [T, Hq, D] is returned; without, (q, k). With a
    PagedCacheFp8 they are held as codes; the tokens that go to one page stand next to one another, in
    rising slots (with gaps or without), and a token in a page's slot 0 begins it anew."""
    return (_host or _load_host()).qk_norm_rope(q, k, cos, sin, positions, q_weight, k_weight, eps, rot_start,
                                                interleaved, cache, v, slots, out)


def paged_attention(q, cache, page_table, q_start, kv_len, scale=None, causal=True, window=0,
                    max_q_len=None, max_kv_len=None, out=None, return_lse=False):
    """Attention of the new tokens q bf16 [T, Hq, Dk] of B sequences (sequence b: rows q_start[b] ..
    q_start[b+1]-1) over a PagedCache or PagedCacheFp8 that holds their kv_len[b] keys, their own included, in the
    pages page_table[b] (int32 [B, n]) -> out bf16 [T, Hq, Dv] (and lse fp32 [T, Hq]). q_start int32
    [B+1] and kv_len int32 [B] are on the GPU; max_q_len and max_kv_len bound them for the host
    (default: T, and what the table can hold; tighter is faster). window > 0: each query sees that
    many keys at most, its own the last. A query without keys gets 0 (lse -inf), one with a score
    that is NaN or +inf gets NaN."""
    return (_host or _load_host()).paged_attention(q, cache, page_table, q_start, kv_len, scale, causal, window,
                                                   max_q_len, max_kv_len, out, return_lse)


def moe_route(x, router_w, top_k, bias=None, score="sigmoid", groups=1, topk_groups=1, normalise=None,
              route_scale=1.0):
    """Expert choice for x bf16 [T, D] with router_w bf16 [E, D] -> (weights fp32 [T, top_k], ids
    int32 [T, top_k], best first). bias fp32 [E] shifts the choice only; groups/topk_groups limit it
    to the best groups of experts; normalise (default: for sigmoid scores) makes a token's weights
    sum to route_scale."""
    return (_host or _load_host()).moe_route(x, router_w, top_k, bias, score, groups, topk_groups, normalise,
                                             route_scale)


def moe_experts(x, weights, ids, w13, s13, w2, s2, scale_fmt="fp32", out=None):
    """The experts of a mixture-of-experts layer for x bf16 [T <= 64, D]: w13 e4m3 [E, 2I, D] (gate
    rows, then up rows), w2 e4m3 [E, D, I], scales per 128 x 128 block; ids int32 [T, top_k] (-1: none)
    and weights fp32 [T, top_k] as moe_route gives them -> y bf16 [T, D]."""
    return (_host or _load_host()).moe_experts(x, weights, ids, w13, s13, w2, s2, _fmt(scale_fmt), out)


def moe_layer(x, router_w, w13, s13, w2, s2, top_k, bias=None, score="sigmoid", groups=1,
              topk_groups=1, normalise=None, route_scale=1.0, scale_fmt="fp32", out=None):
    """A whole mixture-of-experts layer for x bf16 [T <= 64, D]: moe_route, then moe_experts."""
    return (_host or _load_host()).moe_layer(x, router_w, top_k, bias, score, groups, topk_groups, normalise,
                                             route_scale, w13, s13, w2, s2, _fmt(scale_fmt), out)
