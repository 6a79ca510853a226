"""FP8 block-scaled linear-layer path for NVIDIA GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/fp8bs.h`` (``libfp8bs.so``, built in place
by ``fp8_block_scaled_fp8bs_gb300.build``). Every step of the path runs in the library's CUDA
kernels; this module only marshals arguments. There is no CPU fallback: if the library is
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
    fp8bs_moe_route / _experts / _layer: argument structures QkNormRopeArgs, PagedAttentionArgs,
        MoeRouting with the C structures' fields
Tensor conveniences (PyTorch CUDA tensors; outputs allocated with torch):
    act_quant(x, scale_fmt="fp32") -> (y, s)      ("DeepSeek-V3 Administrator & Developer
    weight_dequant(w, s) -> y                        Guide", §8.5.1, §8.5.2, §8.5.3)
    fp8_gemm(a, a_s, b, b_s, scale_fmt="fp32") -> c
    fp8_gemm_grouped(a, a_s, b, b_s, row_offsets, scale_fmt="fp32") -> c
    qk_norm_rope(q, k, cos, sin, positions, ...) -> q (and k, or the keys and values in a PagedCache)
    paged_attention(q, cache, page_table, q_start, kv_len, ...) -> out (and lse)
    moe_route(x, router_w, ...) -> (weights, ids)      ("DeepSeek-V3 Administrator & Developer
    moe_experts(x, weights, ids, w13, s13, w2, s2) -> y    Guide", §6.4)
    moe_layer(x, router_w, w13, s13, w2, s2, ...) -> y
"""
from __future__ import annotations

import ctypes
import os
import struct
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
        # (argument structures: byref of one, or its bytes)
        lib.fp8bs_qk_norm_rope.argtypes = [vp, vp]
        lib.fp8bs_paged_attention.argtypes = [vp, vp]
        lib.fp8bs_paged_attention_workspace_size.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
        lib.fp8bs_moe_workspace_size.argtypes = [i64] * 5 + [ctypes.POINTER(ctypes.c_size_t)]
        lib.fp8bs_moe_route.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        lib.fp8bs_moe_experts.argtypes = [vp] * 8 + [i64] * 5 + [i32, vp, ctypes.c_size_t, vp]
        lib.fp8bs_moe_layer.argtypes = [vp] * 7 + [i64] * 4 + \
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


def fp8_gemm(a, a_s, b, b_s, scale_fmt="fp32", out=None, weights_constant=False,
             workspace="auto"):
    """C[M,N] bf16 = A[M,K] . B[N,K]^T with per-128-K-block scales a_s [M,K/128] and
    b_s [ceil(N/128), K/128]. workspace: "auto" (a cached one per device and stream), None (no
    split K loops) or a zero-filled uint8 CUDA tensor of fp8bs_gemm_workspace_size() bytes."""
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
        workspace = gemm_workspace(a.device)
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
        workspace = gemm_workspace(b.device)
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
# These calls take microseconds on the GPU, so their host side is kept short: one pass over the tensors'
# attributes decides whether everything is as it should be, and only if it is not do the checks that say what
# is wrong run (_explain); the C structures are packed in one go (the ctypes structures above, field by field,
# cost several microseconds a call).

class PagedCache(NamedTuple):
    """Keys [pages, page_size, heads, dk] and values [pages, page_size, heads, dv], bf16 CUDA tensors
    (views of another order too: rows contiguous, the other strides multiples of 8)."""
    k: Any
    v: Any


_KV_FORMAT = "PP11q"
_pack_norm_rope = struct.Struct("@PPP6qPPPPPPP" + _KV_FORMAT + "5qif").pack
_pack_attention = struct.Struct("@Pqq" + _KV_FORMAT + "PqPPPP6qifPN").pack
_pack_routing = struct.Struct("@PP3qiif4x").pack
_KV_SIZE, _NORM_ROPE_SIZE, _ATTENTION_SIZE, _ROUTING_SIZE = (
    struct.calcsize("@" + f) for f in (_KV_FORMAT, "PPP6qPPPPPPP" + _KV_FORMAT + "5qif",
                                       "Pqq" + _KV_FORMAT + "PqPPPP6qifPN", "PP3qiif4x"))
assert (_KV_SIZE, _NORM_ROPE_SIZE, _ATTENTION_SIZE, _ROUTING_SIZE) == tuple(
    ctypes.sizeof(c) for c in (KvCache, QkNormRopeArgs, PagedAttentionArgs, MoeRouting))


class _Types:
    """torch's types, looked up once (the package itself does not import torch)."""
    ready = False

    def load(self):
        import torch
        self.bf16, self.f32, self.i32 = torch.bfloat16, torch.float32, torch.int32
        self.i64, self.e4m3 = torch.int64, torch.float8_e4m3fn
        self.empty = torch.empty
        self.ready = True
        return self


_types = _Types()


def _dense(t, dtype, dev, shape):
    """Whether t is a contiguous tensor of this type and shape on CUDA device `dev`."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _rows(t, ndim, name):
    """A bf16 CUDA tensor whose last axis is contiguous."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != ndim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a {ndim}-D tensor with contiguous rows")
    return t


def _explain(device, rows, dense):
    """The checks of types, devices and layouts, one by one, with what is wrong. rows: {name: (tensor, ndim)}, dense: {name:
    (tensor, dtype, ndim)}."""
    for name, (t, ndim) in rows.items():
        _rows(t, ndim, name)
    for name, (t, dtype, ndim) in dense.items():
        if t is not None:
            _require(t, dtype, ndim, name)
    for name, (t, *_) in (*rows.items(), *dense.items()):
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, like the other tensors")


_stream_of = None


def _raw_stream(dev):
    """The current stream of device `dev` (by torch's own shortcut where it has one: a Stream object
    takes microseconds to make)."""
    global _stream_of
    if _stream_of is None:
        import torch
        _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _stream_of(dev)


def _new_output(out, shape, like):
    """The bf16 output of `shape`: new on the device of `like` (bf16), or the caller's `out`, checked."""
    if out is None:
        return _types.empty(shape, dtype=_types.bf16, device=like.device)
    return _output(out, shape, like.device)


def qk_norm_rope(q, k, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6, rot_start=0,
                 interleaved=False, cache=None, v=None, slots=None, out=None):
    """RMS norm per head (where a weight is given) and rotation of q bf16 [T, Hq, D] and k bf16
    [T, Hk, D] by positions int32 [T]; cos, sin fp32 [max_positions, R/2] rotate the channels
    rot_start .. rot_start+R-1. With a PagedCache, the keys and v bf16 [T, Hk, Dv] go to its slots
    int64 [T] (negative: not written) and q bf16 [T, Hq, D] is returned; without, (q, k)."""
    ty = _types if _types.ready else _types.load()
    bf16 = ty.bf16
    if cache is None:
        if v is not None or slots is not None:
            raise ValueError("v and slots need a cache")
    elif v is None or slots is None:
        raise ValueError("a cache needs v and slots")
    try:
        T, hq, d = q.shape
        hk = k.shape[1]
        max_pos, half = table = cos.shape
        dev = q.get_device()
        q0, q1, q2 = q.stride()
        k0, k1, k2 = k.stride()
        fine = (dev >= 0 and q.dtype is bf16 and q2 == 1 and k.dtype is bf16 and k2 == 1 and
                k.shape == (T, hk, d) and k.get_device() == dev and _dense(cos, ty.f32, dev, table) and
                _dense(sin, ty.f32, dev, table) and _dense(positions, ty.i32, dev, (T,)) and
                (q_weight is None or _dense(q_weight, bf16, dev, (d,))) and
                (k_weight is None or _dense(k_weight, bf16, dev, (d,))))
        if cache is not None:
            ck, cv = cache
            pages, page_size, heads, cd = ck.shape
            dv = cv.shape[3]
            v0, v1, v2 = v.stride()
            ck_strides, cv_strides = ck.stride(), cv.stride()
            fine = (fine and v.dtype is bf16 and v2 == 1 and v.shape == (T, hk, dv) and
                    v.get_device() == dev and ck.dtype is bf16 and ck_strides[3] == 1 and
                    heads == hk and cd == d and ck.get_device() == dev and cv.dtype is bf16 and
                    cv_strides[3] == 1 and cv.shape == (pages, page_size, hk, dv) and
                    cv.get_device() == dev and _dense(slots, ty.i64, dev, (T,)))
    except (AttributeError, ValueError, TypeError):
        fine = False
    if not fine:
        _rows(q, 3, "q")
        _explain(q.device, {"q": (q, 3), "k": (k, 3),
                            **({} if cache is None else {"v": (v, 3), "cache.k": (cache[0], 4),
                                                         "cache.v": (cache[1], 4)})},
                 {"cos": (cos, ty.f32, 2), "sin": (sin, ty.f32, 2), "positions": (positions, ty.i32, 1),
                  "q_weight": (q_weight, bf16, 1), "k_weight": (k_weight, bf16, 1),
                  "slots": (slots, ty.i64, 1)})
        raise ValueError("the shapes of q [T, Hq, D], k [T, Hk, D], v [T, Hk, Dv], cos and sin "
                         "[max_positions, R/2], positions and slots [T], the weights [D] and the cache "
                         "[pages, page_size, Hk, D or Dv] do not match")
    if cache is None:
        k_out = k.new_empty((T, hk, d))
        fields = (k_out.data_ptr(), 0, min(T, 1), max(T, 1), hk, d, d, 0, hk * d, d, 0, 0, 0)
        v_ptr = v0 = v1 = slots_ptr = 0
    else:
        fields = (ck.data_ptr(), cv.data_ptr(), pages, page_size, hk, d, dv, *ck_strides[:3],
                  *cv_strides[:3])
        v_ptr, slots_ptr = v.data_ptr(), slots.data_ptr()
    q_out = _new_output(out, (T, hq, d), q)
    args = _pack_norm_rope(
        q.data_ptr(), k.data_ptr(), v_ptr, q0, q1, k0, k1, v0, v1,
        0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(),
        cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), slots_ptr, q_out.data_ptr(), *fields, T, hq,
        max_pos, rot_start, 2 * half, 1 if interleaved else 0, eps)
    status = (_lib or load()).fp8bs_qk_norm_rope(args, _raw_stream(dev))
    if status:
        raise Fp8bsError("fp8bs_qk_norm_rope", status)
    return q_out if cache is not None else (q_out, k_out)


_scratch = {}


def _scratch_bytes(dev, stream, nbytes):
    """Device memory of at least nbytes for one call on `stream`: one buffer per device and stream (calls on
    one stream follow one another, so they can share it) -> (pointer, bytes, ...). It grows by doubling, and
    the smaller ones before it are kept: a captured graph may still use them."""
    buf = _scratch.get((dev, stream))
    if buf is None or buf[1] < nbytes:
        import torch
        size = max(nbytes, 2 * buf[1] if buf else 1 << 20)
        t = torch.empty(size, dtype=torch.uint8, device=torch.device("cuda", dev))
        buf = _scratch[(dev, stream)] = (t.data_ptr(), size, t, buf)
    return buf


def paged_attention(q, cache, page_table, q_start, kv_len, scale=None, causal=True, window=0,
                    max_q_len=None, max_kv_len=None, out=None, return_lse=False):
    """Attention of the new tokens q bf16 [T, Hq, Dk] of B sequences (sequence b: rows q_start[b] ..
    q_start[b+1]-1) over a PagedCache that holds their kv_len[b] keys, their own included, in the
    pages page_table[b] (int32 [B, n]) -> out bf16 [T, Hq, Dv] (and lse fp32 [T, Hq]). q_start int32
    [B+1] and kv_len int32 [B] are on the GPU; max_q_len and max_kv_len bound them for the host
    (default: T, and what the table can hold; tighter is faster). window > 0: each query sees that
    many keys at most, its own the last."""
    ty = _types if _types.ready else _types.load()
    bf16, i32 = ty.bf16, ty.i32
    ck, cv = cache
    try:
        T, hq, dk = q.shape
        pages, page_size, heads, cdk = ck.shape
        dv = cv.shape[3]
        B, n = table = page_table.shape
        dev = q.get_device()
        q0, q1, q2 = q.stride()
        ck_strides, cv_strides = ck.stride(), cv.stride()
        fine = (dev >= 0 and q.dtype is bf16 and q2 == 1 and dk == cdk and hq % heads == 0 and
                ck.dtype is bf16 and ck_strides[3] == 1 and ck.get_device() == dev and
                cv.dtype is bf16 and cv_strides[3] == 1 and cv.get_device() == dev and
                cv.shape == (pages, page_size, heads, dv) and _dense(page_table, i32, dev, table) and
                _dense(q_start, i32, dev, (B + 1,)) and _dense(kv_len, i32, dev, (B,)))
    except (AttributeError, ValueError, TypeError, ZeroDivisionError):
        fine = False
    if not fine:
        _rows(q, 3, "q")
        _explain(q.device, {"q": (q, 3), "cache.k": (ck, 4), "cache.v": (cv, 4)},
                 {"page_table": (page_table, i32, 2), "q_start": (q_start, i32, 1),
                  "kv_len": (kv_len, i32, 1)})
        raise ValueError("the shapes of q [T, Hq, Dk], the cache [pages, page_size, Hk, Dk or Dv] (Hk "
                         "dividing Hq), page_table [B, n], q_start [B+1] and kv_len [B] do not match")
    o = _new_output(out, (T, hq, dv), q)
    lse = ty.empty((T, hq), dtype=ty.f32, device=q.device) if return_lse else None
    stream = _raw_stream(dev)
    lib = _lib or load()
    # The library says whether the workspace at hand is large enough; if not, it is asked how much it takes.
    ws = _scratch.get((dev, stream)) or (0, 0)
    while True:
        args = _pack_attention(
            q.data_ptr(), q0, q1, ck.data_ptr(), cv.data_ptr(), pages, page_size, heads, dk, dv,
            *ck_strides[:3], *cv_strides[:3], page_table.data_ptr(), n, q_start.data_ptr(),
            kv_len.data_ptr(), o.data_ptr(), 0 if lse is None else lse.data_ptr(), B, T, hq, T if max_q_len is None else max_q_len,
            n * page_size if max_kv_len is None else max_kv_len, window, 1 if causal else 0,
            dk ** -0.5 if scale is None else scale, ws[0], ws[1])
        status = lib.fp8bs_paged_attention(args, stream)
        if status == 0:
            return (o, lse) if return_lse else o
        if status == 1:
            need = ctypes.c_size_t(0)
            if lib.fp8bs_paged_attention_workspace_size(args, ctypes.byref(need)) == 0 and \
                    need.value > ws[1]:
                ws = _scratch_bytes(dev, stream, need.value)
                continue
        raise Fp8bsError("fp8bs_paged_attention", status)


def _routing(x, router_w, bias, top_k, score, groups, topk_groups, normalise, route_scale):
    """(CUDA device, experts, the packed fp8bs_moe_routing), checked."""
    ty = _types if _types.ready else _types.load()
    try:
        T, D = x.shape
        experts = router_w.shape[0]
        dev = x.get_device()
        fine = (dev >= 0 and x.dtype is ty.bf16 and x.is_contiguous() and
                _dense(router_w, ty.bf16, dev, (experts, D)) and
                (bias is None or _dense(bias, ty.f32, dev, (experts,))))
    except (AttributeError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        _require(x, ty.bf16, 2, "x")
        _explain(x.device, {}, {"x": (x, ty.bf16, 2), "router_w": (router_w, ty.bf16, 2),
                                "bias": (bias, ty.f32, 1)})
        raise ValueError("the shapes of x [T, D], router_w [E, D] and bias [E] do not match")
    if score == "sigmoid":
        kind, normalise = SCORE_SIGMOID, 1 if normalise is None else int(normalise)
    elif score == "softmax":
        kind, normalise = SCORE_SOFTMAX, 0 if normalise is None else int(normalise)
    else:
        raise ValueError(f"unknown score {score!r}")
    return dev, experts, _pack_routing(router_w.data_ptr(), 0 if bias is None else bias.data_ptr(), top_k,
                                       groups, topk_groups, kind, normalise, route_scale)


def moe_route(x, router_w, top_k, bias=None, score="sigmoid", groups=1, topk_groups=1, normalise=None,
              route_scale=1.0):
    """Expert choice for x bf16 [T, D] with router_w bf16 [E, D] -> (weights fp32 [T, top_k], ids
    int32 [T, top_k], best first). bias fp32 [E] shifts the choice only; groups/topk_groups limit it
    to the best groups of experts; normalise (default: for sigmoid scores) makes a token's weights
    sum to route_scale."""
    dev, experts, routing = _routing(x, router_w, bias, top_k, score, groups, topk_groups, normalise,
                                     route_scale)
    T, D = x.shape
    weights = x.new_empty((T, top_k), dtype=_types.f32)
    ids = x.new_empty((T, top_k), dtype=_types.i32)
    _check("fp8bs_moe_route", (_lib or load()).fp8bs_moe_route(
        x.data_ptr(), routing, weights.data_ptr(), ids.data_ptr(), T, D, experts, _raw_stream(dev)))
    return weights, ids


def _expert_shapes(x, w13, s13, w2, s2, weights=None, ids=None):
    """(CUDA device, T, D, I, E), checked."""
    ty = _types if _types.ready else _types.load()
    f32, e4m3 = ty.f32, ty.e4m3
    try:
        T, D = x.shape
        E, _, inter = w2.shape
        dev = x.get_device()
        kb, ib = D // BLOCK, inter // BLOCK
        fine = (dev >= 0 and x.dtype is ty.bf16 and x.is_contiguous() and
                _dense(w13, e4m3, dev, (E, 2 * inter, D)) and _dense(w2, e4m3, dev, (E, D, inter)) and
                _dense(s13, f32, dev, (E, 2 * inter // BLOCK, kb)) and _dense(s2, f32, dev, (E, kb, ib)) and
                (ids is None or (_dense(ids, ty.i32, dev, (T, ids.shape[1])) and
                                 _dense(weights, f32, dev, ids.shape))))
    except (AttributeError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        _require(x, ty.bf16, 2, "x")
        _explain(x.device, {}, {"x": (x, ty.bf16, 2), "w13": (w13, e4m3, 3), "s13": (s13, f32, 3),
                                "w2": (w2, e4m3, 3), "s2": (s2, f32, 3), "weights": (weights, f32, 2),
                                "ids": (ids, ty.i32, 2)})
        raise ValueError("the shapes of x [T, D], w13 [E, 2I, D], s13 [E, 2I/128, D/128], w2 [E, D, I], "
                         "s2 [E, D/128, I/128] (and weights, ids [T, top_k]) do not match")
    return dev, T, D, inter, E


def _expert_workspace(lib, dev, stream, T, D, inter, E, top_k):
    need = ctypes.c_size_t(0)
    _check("fp8bs_moe_workspace_size", lib.fp8bs_moe_workspace_size(T, D, inter, E, top_k,
                                                                    ctypes.byref(need)))
    return _scratch_bytes(dev, stream, need.value)


def moe_experts(x, weights, ids, w13, s13, w2, s2, scale_fmt="fp32", out=None):
    """The experts of a mixture-of-experts layer for x bf16 [T <= 64, D]: w13 e4m3 [E, 2I, D] (gate
    rows, then up rows), w2 e4m3 [E, D, I], scales per 128 x 128 block; ids int32 [T, top_k] (-1: none)
    and weights fp32 [T, top_k] as moe_route gives them -> y bf16 [T, D]."""
    dev, T, D, inter, E = _expert_shapes(x, w13, s13, w2, s2, weights, ids)
    k = ids.shape[1]
    y = _new_output(out, (T, D), x)
    stream = _raw_stream(dev)
    lib = _lib or load()
    ws = _expert_workspace(lib, dev, stream, T, D, inter, E, k)
    _check("fp8bs_moe_experts", lib.fp8bs_moe_experts(
        x.data_ptr(), weights.data_ptr(), ids.data_ptr(), w13.data_ptr(), s13.data_ptr(), w2.data_ptr(),
        s2.data_ptr(), y.data_ptr(), T, D, inter, E, k, _fmt(scale_fmt), ws[0], ws[1], stream))
    return y


def moe_layer(x, router_w, w13, s13, w2, s2, top_k, bias=None, score="sigmoid", groups=1,
              topk_groups=1, normalise=None, route_scale=1.0, scale_fmt="fp32", out=None):
    """A whole mixture-of-experts layer for x bf16 [T <= 64, D]: moe_route, then moe_experts."""
    _, experts, routing = _routing(x, router_w, bias, top_k, score, groups, topk_groups, normalise,
                                   route_scale)
    dev, T, D, inter, E = _expert_shapes(x, w13, s13, w2, s2)
    if experts != E:
        raise ValueError("router_w must have one row per expert")
    y = _new_output(out, (T, D), x)
    stream = _raw_stream(dev)
    lib = _lib or load()
    ws = _expert_workspace(lib, dev, stream, T, D, inter, E, top_k)
    _check("fp8bs_moe_layer", lib.fp8bs_moe_layer(
        x.data_ptr(), routing, w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), y.data_ptr(),
        T, D, inter, E, _fmt(scale_fmt), ws[0], ws[1], stream))
    return y
