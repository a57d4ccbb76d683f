"""Thin Python binding of libftq (the C ABI declared in include/ftq.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libftq.so.  PyTorch supplies device memory and the current stream.
There is no fallback: if the library is missing or the device is not a GPU,
the calls raise.

Every call takes the stream to work on (None: the current one).  What a call
allocates belongs to that stream and stays valid for the current one; the tensors
passed to it are the caller's to keep, and to order before the call and after
it, as for any work on another stream.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# FTQ_LIB_PATH: a libftq.so built elsewhere (for example with host sanitizers)
LIB_PATH = os.environ.get("FTQ_LIB_PATH") or os.path.join(_PKG, "libftq.so")

OK, ERR_INVALID_ARG, ERR_WORKSPACE, ERR_LAUNCH, ERR_UNSUPPORTED, ERR_HIP = range(6)
PATH_AUTO, PATH_GEMV, PATH_GROUPED = 0, 1, 2
ACT_SILU, ACT_GELU_TANH = 1, 2
# grouped-path kernels (same bits, different speed); GROUPED_I8 is the default
GROUPED_I8, GROUPED_F16, GROUPED_F16_WS = 0, 1, 2
# weight block types (GGUF type ids) and their block bytes
W_Q4_0, W_Q4_1, W_Q5_0, W_Q5_1, W_Q8_0 = 2, 3, 6, 7, 8
W_BLOCK_BYTES = {W_Q4_0: 18, W_Q4_1: 20, W_Q5_0: 22, W_Q5_1: 24, W_Q8_0: 34}
GEMV_ONLY = (W_Q5_0, W_Q5_1)   # the other types also run on the grouped path
QK, Q4_0_BYTES, Q8_1_BYTES = 32, 18, 36
# element types of the router and the 8-bit floating-point calls
F32, F16, BF16 = 0, 1, 2
_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
FP8, FP8_BLOCK = torch.float8_e4m3fn, 128
EXACT = 0x100   # or'ed to the out type of the 8-bit floating-point matmul

EXPORTS = (
    "ftq_quantize_q8_1", "ftq_quantize_q4_0", "ftq_moe_select_path", "ftq_moe_workspace_bytes",
    "ftq_moe_q4_0_q8_1", "ftq_moe_route", "ftq_moe_q4_0_q8_1_routed", "ftq_moe_q4_0_q8_1_partials",
    "ftq_moe_pairs_workspace_bytes", "ftq_moe_q4_0_q8_1_pairs", "ftq_moe_q4_0_q8_1_pairs_routed",
    "ftq_moe_q4_0_q8_1_pairs_partials", "ftq_moe_combine_topk",
    "ftq_moe_q4_0_q8_1_act", "ftq_moe_q4_0_q8_1_act_routed",
    "ftq_moe_gguf_q8_1", "ftq_moe_gguf_q8_1_partials",
    "ftq_last_error", "ftq_version",
    "ftq_debug_force_block_threads", "ftq_debug_grouped_kernel", "ftq_debug_route_kernels", "ftq_debug_gemv_plan", "ftq_moe_q4_0_q8_1_noalloc",
    "ftq_moe_topk", "ftq_quantize_fp8", "ftq_quantize_fp8_weight",
    "ftq_moe_fp8_select_path", "ftq_moe_fp8_workspace_bytes", "ftq_moe_fp8", "ftq_moe_fp8_route", "ftq_moe_fp8_routed",
    "ftq_moe_balance_workspace_bytes", "ftq_moe_balance", "ftq_moe_topk_backward", "ftq_moe_combine_topk_backward",
    "ftq_lora_select_path", "ftq_lora_workspace_bytes", "ftq_lora", "ftq_lora_backward_workspace_bytes", "ftq_lora_backward",
)


class FtqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"ftq status {status}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libftq.so (built in-tree by quantized_moe_expert_quantize_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FtqError(-1, f"{LIB_PATH} is not built; run `python -m quantized_moe_expert_quantize_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.ftq_quantize_q8_1.argtypes = [P, I64, I64, P, P]
    L.ftq_quantize_q8_1.restype = I32
    L.ftq_quantize_q4_0.argtypes = [P, I64, I64, P, P]
    L.ftq_quantize_q4_0.restype = I32
    L.ftq_moe_select_path.argtypes = [I64, I64, I64, I64, I64]
    L.ftq_moe_select_path.restype = I32
    L.ftq_moe_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I32]
    L.ftq_moe_workspace_bytes.restype = I64
    L.ftq_moe_q4_0_q8_1.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, P, SZ, I32, P]
    L.ftq_moe_q4_0_q8_1.restype = I32
    L.ftq_moe_route.argtypes = [P, I64, I64, I64, P, SZ, I32, P]
    L.ftq_moe_route.restype = I32
    L.ftq_moe_q4_0_q8_1_routed.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, P, SZ, I32, P]
    L.ftq_moe_q4_0_q8_1_routed.restype = I32
    L.ftq_moe_q4_0_q8_1_partials.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, P, SZ, I32, P]
    L.ftq_moe_pairs_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I32]
    L.ftq_moe_pairs_workspace_bytes.restype = I64
    for name in ("ftq_moe_q4_0_q8_1_pairs", "ftq_moe_q4_0_q8_1_pairs_routed", "ftq_moe_q4_0_q8_1_pairs_partials"):
        getattr(L, name).argtypes = [P, P, P, P, I64, I64, I64, I64, I64, P, SZ, I32, P]
        getattr(L, name).restype = I32
    L.ftq_moe_combine_topk.argtypes = [P, P, P, I64, I64, I64, P]
    L.ftq_moe_combine_topk.restype = I32
    for name in ("ftq_moe_q4_0_q8_1_act", "ftq_moe_q4_0_q8_1_act_routed"):
        f = getattr(L, name)
        f.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, I32, P, ctypes.c_size_t, I32, P]
        f.restype = I32
    L.ftq_moe_q4_0_q8_1_partials.restype = I32
    for name in ("ftq_moe_gguf_q8_1", "ftq_moe_gguf_q8_1_partials"):
        f = getattr(L, name)
        f.argtypes = [P, I32, P, P, P, I64, I64, I64, I64, I64, I32, P, SZ, I32, P]
        f.restype = I32
    L.ftq_last_error.restype = ctypes.c_char_p
    L.ftq_version.restype = ctypes.c_char_p
    L.ftq_debug_force_block_threads.argtypes = [I32]
    L.ftq_debug_force_block_threads.restype = None
    L.ftq_debug_grouped_kernel.argtypes = [I32]
    L.ftq_debug_grouped_kernel.restype = I32
    L.ftq_debug_route_kernels.argtypes = [I32]
    L.ftq_debug_route_kernels.restype = None
    L.ftq_debug_gemv_plan.argtypes = [I64, I64, I64, I64, I64, I32, I32, P, P, P]
    L.ftq_debug_gemv_plan.restype = I32
    L.ftq_moe_q4_0_q8_1_noalloc.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, I32, P]
    L.ftq_moe_q4_0_q8_1_noalloc.restype = I32
    F = ctypes.c_float
    L.ftq_moe_topk.argtypes = [P, I32, I64, P, P, P, I64, I64, I64, I32, I64, I64, I32, I32, F, P]
    L.ftq_moe_topk.restype = I32
    L.ftq_quantize_fp8.argtypes = [P, I32, I64, I64, I64, P, P, P]
    L.ftq_quantize_fp8.restype = I32
    L.ftq_quantize_fp8_weight.argtypes = [P, I32, I64, I64, I64, P, P, P]
    L.ftq_quantize_fp8_weight.restype = I32
    L.ftq_moe_fp8_select_path.argtypes = [I64, I64, I64, I64, I64]
    L.ftq_moe_fp8_select_path.restype = I32
    L.ftq_moe_fp8_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I32]
    L.ftq_moe_fp8_workspace_bytes.restype = I64
    for name in ("ftq_moe_fp8", "ftq_moe_fp8_routed"):
        f = getattr(L, name)
        f.argtypes = [P, P, P, P, P, P, I32, I64, I64, I64, I64, I64, I32, I32, P, SZ, I32, P]
        f.restype = I32
    L.ftq_moe_fp8_route.argtypes = [P, I64, I64, I64, P, SZ, I32, P]
    L.ftq_moe_fp8_route.restype = I32
    L.ftq_moe_balance_workspace_bytes.argtypes = [I64, I64, I64, I64]
    L.ftq_moe_balance_workspace_bytes.restype = I64
    L.ftq_moe_balance.argtypes = [P, I32, I64, P, P, P, P, P, P, I64, I64, I64, I64, I32, P, SZ, P]
    L.ftq_moe_balance.restype = I32
    L.ftq_moe_topk_backward.argtypes = [P, I32, I64, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I32, I32, F, P]
    L.ftq_moe_topk_backward.restype = I32
    L.ftq_moe_combine_topk_backward.argtypes = [P, P, P, P, I32, P, I64, I64, I64, P]
    L.ftq_moe_combine_topk_backward.restype = I32
    L.ftq_lora_select_path.argtypes = [I64, I64, I64]
    L.ftq_lora_select_path.restype = I32
    L.ftq_lora_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64, I32, I32]
    L.ftq_lora_workspace_bytes.restype = I64
    L.ftq_lora.argtypes = [P, I64, P, P, P, P, P, I64, P, I64, P, I32, I32, I64, I64, I64, I64, I64, I64, I32, P, SZ, I32, P]
    L.ftq_lora.restype = I32
    L.ftq_lora_backward_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64, I32]
    L.ftq_lora_backward_workspace_bytes.restype = I64
    L.ftq_lora_backward.argtypes = [P, I64, P, I64, P, P, P, P, P, P, P, P, P, I32, I64, I64, I64, I64, I64, I64, I32, P, SZ, P]
    L.ftq_lora_backward.restype = I32
    _lib = L
    return L


def last_error() -> str:
    return lib().ftq_last_error().decode()


def version() -> str:
    return lib().ftq_version().decode()


def _check(status: int):
    if status != OK:
        raise FtqError(status, last_error())


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for work on `stream`, from that stream's pool: a block of the current stream's may still be in use by work
    queued there, which `stream` does not wait for.  The caller goes on with it on the current stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _out(out: torch.Tensor, numel: int, name: str, dtype):
    """A caller's output buffer must hold exactly the elements the call writes."""
    if out.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {out.numel()}")
    return _dev(out, name, dtype)


def quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [T, K] -> uint8 [T, K/32*36] Q8_1 blocks."""
    T, K = x.shape
    if out is None:
        out = _empty((T, K // QK * Q8_1_BYTES), torch.uint8, x.device, stream)
    _check(lib().ftq_quantize_q8_1(_dev(x, "x", torch.float32), T, K, _out(out, T * (K // QK) * Q8_1_BYTES, "out", torch.uint8),
                                   _stream(stream)))
    return out


def quantize_q4_0(w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [..., K] -> uint8 [..., K/32*18] Q4_0 blocks."""
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    if out is None:
        out = _empty(tuple(w.shape[:-1]) + (K // QK * Q4_0_BYTES,), torch.uint8, w.device, stream)
    _check(lib().ftq_quantize_q4_0(_dev(w, "w", torch.float32), rows, K, _out(out, rows * (K // QK) * Q4_0_BYTES, "out", torch.uint8),
                                   _stream(stream)))
    return out


def gemv_plan(E: int, N: int, K: int, T: int, top_k: int, wtype: int = 2, act: int = 0) -> dict:
    """The GEMV path's on-chip plan for these sizes (host arithmetic): K blocks
    per segment, activation rows per pass, workgroups per CU."""
    seg, pc, per_cu = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ftq_debug_gemv_plan(E, N, K, T, top_k, wtype, act, ctypes.addressof(seg), ctypes.addressof(pc),
                                     ctypes.addressof(per_cu)))
    return {"seg": seg.value, "pairs_per_pass": pc.value, "wg_per_cu": per_cu.value}


def grouped_kernel(variant: int):
    """Select the grouped path's kernel for later calls on this thread
    (GROUPED_I8, GROUPED_F16 or GROUPED_F16_WS)."""
    _check(lib().ftq_debug_grouped_kernel(variant))


def route_kernels(split: bool):
    """Bucketing in three kernels at any size (True) or, for small batches, in
    one workgroup (False, the default) for later calls on this thread."""
    lib().ftq_debug_route_kernels(1 if split else 0)


def select_path(E: int, N: int, K: int, T: int, top_k: int) -> int:
    r = lib().ftq_moe_select_path(E, N, K, T, top_k)
    if r < 0:
        raise FtqError(-r, last_error())
    return r


def workspace_bytes(E: int, N: int, K: int, T: int, top_k: int, path: int = PATH_AUTO) -> int:
    r = lib().ftq_moe_workspace_bytes(E, N, K, T, top_k, path)
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def _moe_args(w, a, topk_ids, E, N, K, per_pair=False):
    T, top_k = topk_ids.shape
    nb = K // QK
    if w.numel() != E * N * nb * Q4_0_BYTES:
        raise ValueError("w must hold E*N*(K/32) Q4_0 blocks")
    rows = T * top_k if per_pair else T
    if a.numel() != rows * nb * Q8_1_BYTES:
        raise ValueError(f"a must hold {'T*top_k' if per_pair else 'T'}*(K/32) Q8_1 blocks")
    return T, top_k


def _workspace(ws, need, device, stream):
    if need == 0:
        return None, 0
    if ws is None:
        ws = _empty(need, torch.uint8, device, stream)
    if ws.numel() < need:
        raise ValueError(f"workspace needs {need} bytes")
    return ws, ws.numel()


def moe(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
        path: int = PATH_AUTO, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
        stream=None) -> torch.Tensor:
    """MoE expert matmul: fp32 out [T*top_k, N]."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    if out is None:
        out = _empty((T * top_k, N), torch.float32, a.device, stream)
    need = workspace_bytes(E, N, K, T, top_k, path)
    ws, ws_n = _workspace(workspace, need, a.device, stream)
    _check(lib().ftq_moe_q4_0_q8_1(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k,
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_noalloc(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
                out: torch.Tensor, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """moe() through ftq_moe_q4_0_q8_1_noalloc: no workspace, the library's
    fixed per-device scratch instead.  `out` is the caller's (nothing here
    allocates device memory)."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    _check(lib().ftq_moe_q4_0_q8_1_noalloc(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k, path, _stream(stream)))
    return out


def moe_route(topk_ids: torch.Tensor, E: int, workspace: torch.Tensor | None, path: int = PATH_AUTO,
              stream=None) -> None:
    """Group the pairs by expert into `workspace` (see ftq_moe_route)."""
    T, top_k = topk_ids.shape
    ws_n = workspace.numel() if workspace is not None else 0
    _check(lib().ftq_moe_route(_dev(topk_ids, "topk_ids", torch.int32), E, T, top_k,
                               workspace.data_ptr() if workspace is not None else None, ws_n, path,
                               _stream(stream)))


def moe_routed(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
               out: torch.Tensor, workspace: torch.Tensor | None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """The matmul on pairs already routed into `workspace` by moe_route."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    ws_n = workspace.numel() if workspace is not None else 0
    _check(lib().ftq_moe_q4_0_q8_1_routed(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k,
        workspace.data_ptr() if workspace is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_partials(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
                 path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """Exact integer block partials int32 [T*top_k, N, K/32]."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    out = _empty((T * top_k, N, K // QK), torch.int32, a.device, stream)
    need = workspace_bytes(E, N, K, T, top_k, path)
    ws, ws_n = _workspace(None, need, a.device, stream)
    _check(lib().ftq_moe_q4_0_q8_1_partials(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _dev(out, "partials", torch.int32), E, N, K, T, top_k,
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


# ---- per-pair activations (down projection) and the top-k combine -----------

def pairs_workspace_bytes(E: int, N: int, K: int, T: int, top_k: int, path: int = PATH_AUTO) -> int:
    r = lib().ftq_moe_pairs_workspace_bytes(E, N, K, T, top_k, path)
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def moe_pairs(w: torch.Tensor, a_pairs: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
              path: int = PATH_AUTO, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """MoE expert matmul on per-pair activations a_pairs [T*top_k, K/32 Q8_1 blocks]:
    fp32 out [T*top_k, N]."""
    T, top_k = _moe_args(w, a_pairs, topk_ids, E, N, K, per_pair=True)
    if out is None:
        out = _empty((T * top_k, N), torch.float32, a_pairs.device, stream)
    need = pairs_workspace_bytes(E, N, K, T, top_k, path)
    ws, ws_n = _workspace(workspace, need, a_pairs.device, stream)
    _check(lib().ftq_moe_q4_0_q8_1_pairs(
        _dev(w, "w", torch.uint8), _dev(a_pairs, "a_pairs", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k,
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_pairs_routed(w: torch.Tensor, a_pairs: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
                     out: torch.Tensor, workspace: torch.Tensor | None, path: int = PATH_AUTO,
                     stream=None) -> torch.Tensor:
    """moe_pairs on pairs already routed into `workspace` (sized by pairs_workspace_bytes) by moe_route."""
    T, top_k = _moe_args(w, a_pairs, topk_ids, E, N, K, per_pair=True)
    ws_n = workspace.numel() if workspace is not None else 0
    _check(lib().ftq_moe_q4_0_q8_1_pairs_routed(
        _dev(w, "w", torch.uint8), _dev(a_pairs, "a_pairs", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k,
        workspace.data_ptr() if workspace is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_pairs_partials(w: torch.Tensor, a_pairs: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
                       path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """Exact integer block partials int32 [T*top_k, N, K/32] on per-pair activations."""
    T, top_k = _moe_args(w, a_pairs, topk_ids, E, N, K, per_pair=True)
    out = _empty((T * top_k, N, K // QK), torch.int32, a_pairs.device, stream)
    need = pairs_workspace_bytes(E, N, K, T, top_k, path)
    ws, ws_n = _workspace(None, need, a_pairs.device, stream)
    _check(lib().ftq_moe_q4_0_q8_1_pairs_partials(
        _dev(w, "w", torch.uint8), _dev(a_pairs, "a_pairs", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _dev(out, "partials", torch.int32), E, N, K, T, top_k,
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


# ---- first layer with the gated activation fused (gate rows, then up rows) ----

def moe_act(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int, act: int,
            path: int = PATH_AUTO, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """act(gate) * up: fp32 out [T*top_k, N/2] from N = 2*(N/2) weight rows per expert."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    if out is None:
        out = _empty((T * top_k, N // 2), torch.float32, a.device, stream)
    need = workspace_bytes(E, N, K, T, top_k, path)
    ws, ws_n = _workspace(workspace, need, a.device, stream)
    _check(lib().ftq_moe_q4_0_q8_1_act(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * (N // 2), "out", torch.float32), E, N, K, T, top_k, act,
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_act_routed(w: torch.Tensor, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int, act: int,
                   out: torch.Tensor, workspace: torch.Tensor | None, path: int = PATH_AUTO,
                   stream=None) -> torch.Tensor:
    """moe_act on pairs already routed into `workspace` by moe_route."""
    T, top_k = _moe_args(w, a, topk_ids, E, N, K)
    ws_n = workspace.numel() if workspace is not None else 0
    _check(lib().ftq_moe_q4_0_q8_1_act_routed(
        _dev(w, "w", torch.uint8), _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * (N // 2), "out", torch.float32), E, N, K, T, top_k, act,
        workspace.data_ptr() if workspace is not None else None, ws_n, path, _stream(stream)))
    return out


# ---- the other GGUF weight block types (GEMV path) ---------------------------

def _gguf_args(w, wtype, a, topk_ids, E, N, K, per_pair):
    T, top_k = topk_ids.shape
    nb = K // QK
    if wtype not in W_BLOCK_BYTES:
        raise ValueError(f"unknown weight type {wtype}")
    if w.numel() != E * N * nb * W_BLOCK_BYTES[wtype]:
        raise ValueError("w must hold E*N*(K/32) blocks of the weight type")
    rows = T * top_k if per_pair else T
    if a.numel() != rows * nb * Q8_1_BYTES:
        raise ValueError(f"a must hold {'T*top_k' if per_pair else 'T'}*(K/32) Q8_1 blocks")
    return T, top_k


def moe_gguf(w: torch.Tensor, wtype: int, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
             per_pair: bool = False, path: int = PATH_AUTO, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Matmul with weights of GGUF type `wtype` (W_*): fp32 out [T*top_k, N]."""
    T, top_k = _gguf_args(w, wtype, a, topk_ids, E, N, K, per_pair)
    if out is None:
        out = _empty((T * top_k, N), torch.float32, a.device, stream)
    need = workspace_bytes(E, N, K, T, top_k, PATH_GEMV if wtype in GEMV_ONLY else path)
    ws, ws_n = _workspace(workspace, need, a.device, stream)
    _check(lib().ftq_moe_gguf_q8_1(
        _dev(w, "w", torch.uint8), wtype, _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _out(out, T * top_k * N, "out", torch.float32), E, N, K, T, top_k, int(per_pair),
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


def moe_gguf_partials(w: torch.Tensor, wtype: int, a: torch.Tensor, topk_ids: torch.Tensor, E: int, N: int, K: int,
                      per_pair: bool = False, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """Integer parts sum((q - z) * q8), int32 [T*top_k, N, K/32]."""
    T, top_k = _gguf_args(w, wtype, a, topk_ids, E, N, K, per_pair)
    out = _empty((T * top_k, N, K // QK), torch.int32, a.device, stream)
    need = workspace_bytes(E, N, K, T, top_k, PATH_GEMV if wtype in GEMV_ONLY else path)
    ws, ws_n = _workspace(None, need, a.device, stream)
    _check(lib().ftq_moe_gguf_q8_1_partials(
        _dev(w, "w", torch.uint8), wtype, _dev(a, "a", torch.uint8), _dev(topk_ids, "topk_ids", torch.int32),
        _dev(out, "partials", torch.int32), E, N, K, T, top_k, int(per_pair),
        ws.data_ptr() if ws is not None else None, ws_n, path, _stream(stream)))
    return out


def combine_topk(y: torch.Tensor, gates: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t, n] = sum_j gates[t, j] * y[t*top_k + j, n] (fp32, j ascending)."""
    T, top_k = gates.shape
    if y.dim() != 2 or y.shape[0] != T * top_k:
        raise ValueError("y must be [T*top_k, N]")
    N = y.shape[1]
    if out is None:
        out = _empty((T, N), torch.float32, y.device, stream)
    _check(lib().ftq_moe_combine_topk(_dev(y, "y", torch.float32), _dev(gates, "gates", torch.float32),
                                      _out(out, T * N, "out", torch.float32), T, top_k, N, _stream(stream)))
    return out


# ---- router, and experts in 8-bit floating point -----------------------------

# These calls may take no longer on the GPU than a few microseconds, so the
# marshalling is kept to about one: the raw-handle queries of torch._C stand in
# for torch.cuda.current_device() and current_stream() (0.1 us against 2.8 us).
# They are looked up in the call: a torch without GPU support lacks them.
def _device() -> int:
    return torch._C._cuda_getDevice()


def _raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _device_for(t: torch.Tensor, name: str) -> int:
    """The current device, which the tensors of a call must be on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return _device()


def _refuse(t: torch.Tensor, name: str, dtype, shape, dev: int):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _here(t: torch.Tensor, name: str, dtype, dev: int, shape=None) -> int:
    """Address of a contiguous tensor of this type and shape on the current device."""
    if t.get_device() != dev or t.dtype != dtype or (shape is not None and t.shape != shape) or not t.is_contiguous():
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dev: int):
    """(address, dtype, row stride) of a [rows, columns] tensor with contiguous columns."""
    dt = _DTYPE.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        _refuse(t, name, t.dtype, None, dev)
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, columns]")
    (rows, columns), (ld, one) = t.shape, t.stride()
    if (columns > 1 and one != 1) or (rows > 1 and ld < columns):
        raise ValueError(f"{name} must have contiguous columns and rows that do not overlap")
    return t.data_ptr(), dt, ld if rows > 1 else columns


def _stream_here(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the current device is cuda:{dev}")
    return stream.cuda_stream


def moe_topk(logits: torch.Tensor, top_k: int, score: int = SCORE_SOFTMAX, bias: torch.Tensor | None = None,
             n_group: int = 1, topk_group: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
             ids: torch.Tensor | None = None, gates: torch.Tensor | None = None, stream=None):
    """Router: logits [T, E] (rows may be strided) -> (int32 ids, fp32 gates), each [T, top_k] (see ftq_moe_topk)."""
    dev = _device_for(logits, "logits")
    p, dt, ld = _rows(logits, "logits", dev)
    T, E = logits.shape
    shape = (T, max(top_k, 0))
    if ids is None:
        ids = _empty(shape, torch.int32, logits.device, stream)
    if gates is None:
        gates = _empty(shape, torch.float32, logits.device, stream)
    _check(lib().ftq_moe_topk(p, dt, ld, _here(bias, "bias", torch.float32, dev, (E,)) if bias is not None else None,
                              _here(ids, "ids", torch.int32, dev, shape), _here(gates, "gates", torch.float32, dev, shape),
                              T, E, top_k, score, n_group, topk_group, group_top, int(renorm), scale, _stream_here(stream, dev)))
    return ids, gates


def quantize_fp8(x: torch.Tensor, out: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """x [T, K] (rows may be strided) -> (e4m3 codes [T, K], fp32 scales [T, ceil(K/128)])."""
    dev = _device_for(x, "x")
    p, dt, ld = _rows(x, "x", dev)
    T, K = x.shape
    shape = (T, -(-K // FP8_BLOCK))
    if out is None:
        out = _empty((T, K), FP8, x.device, stream)
    if scales is None:
        scales = _empty(shape, torch.float32, x.device, stream)
    _check(lib().ftq_quantize_fp8(p, dt, ld, T, K, _here(out, "out", FP8, dev, (T, K)),
                                  _here(scales, "scales", torch.float32, dev, shape), _stream_here(stream, dev)))
    return out, scales


def quantize_fp8_weight(w: torch.Tensor, out: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """w [E, N, K] -> (e4m3 codes [E, N, K], fp32 scales [E, ceil(N/128), ceil(K/128)])."""
    if w.dim() != 3 or w.dtype not in _DTYPE:
        raise ValueError("w must be [E, N, K] in float32, float16 or bfloat16")
    dev = _device_for(w, "w")
    E, N, K = w.shape
    shape = (E, -(-N // FP8_BLOCK), -(-K // FP8_BLOCK))
    if out is None:
        out = _empty((E, N, K), FP8, w.device, stream)
    if scales is None:
        scales = _empty(shape, torch.float32, w.device, stream)
    _check(lib().ftq_quantize_fp8_weight(_here(w, "w", w.dtype, dev), _DTYPE[w.dtype], E, N, K, _here(out, "out", FP8, dev, (E, N, K)),
                                         _here(scales, "scales", torch.float32, dev, shape), _stream_here(stream, dev)))
    return out, scales


def fp8_select_path(E: int, N: int, K: int, T: int, top_k: int) -> int:
    r = lib().ftq_moe_fp8_select_path(E, N, K, T, top_k)
    if r < 0:
        raise FtqError(-r, last_error())
    return r


def fp8_workspace_bytes(E: int, N: int, K: int, T: int, top_k: int, path: int = PATH_AUTO) -> int:
    r = lib().ftq_moe_fp8_workspace_bytes(E, N, K, T, top_k, path)
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def _fp8_call(entry, w, w_scale, a, a_scale, topk_ids, E, N, K, per_pair, act, out, workspace, path, exact, stream):
    dev = _device_for(w, "w")
    T, top_k = topk_ids.shape
    rows, nb = T * top_k if per_pair else T, -(-K // FP8_BLOCK)
    if out.dtype not in _DTYPE:
        raise ValueError(f"out must be float32, float16 or bfloat16, got {out.dtype}")
    ws_n = workspace.numel() if workspace is not None else 0
    _check(entry(
        _here(w, "w", FP8, dev, (E, N, K)), _here(w_scale, "w_scale", torch.float32, dev, (E, -(-N // FP8_BLOCK), nb)),
        _here(a, "a", FP8, dev, (rows, K)), _here(a_scale, "a_scale", torch.float32, dev, (rows, nb)),
        _here(topk_ids, "topk_ids", torch.int32, dev), _here(out, "out", out.dtype, dev, (T * top_k, N // 2 if act else N)),
        _DTYPE[out.dtype] | (EXACT if exact else 0), E, N, K, T, top_k, int(per_pair), act,
        _here(workspace, "workspace", torch.uint8, dev) if workspace is not None else None, ws_n, path, _stream_here(stream, dev)))
    return out


def moe_fp8(w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, a_scale: torch.Tensor, topk_ids: torch.Tensor,
            E: int, N: int, K: int, per_pair: bool = False, act: int = 0, path: int = PATH_AUTO,
            out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
            workspace: torch.Tensor | None = None, stream=None, exact: bool = False) -> torch.Tensor:
    """Expert matmul on e4m3 weights [E, N, K] and activations [T or T*top_k, K] with their block scales:
    out [T*top_k, N], or with act (ACT_*) act(gate) * up [T*top_k, N/2].  exact: exact products also for 16-bit
    results of the grouped path, which drop small bits without it (see ftq_moe_fp8)."""
    T, top_k = topk_ids.shape
    if out is None:
        out = _empty((T * top_k, N // 2 if act else N), out_dtype, a.device, stream)
    if workspace is None:
        need = fp8_workspace_bytes(E, N, K, T, top_k, path)
        workspace = _empty(need, torch.uint8, a.device, stream) if need else None
    return _fp8_call(lib().ftq_moe_fp8, w, w_scale, a, a_scale, topk_ids, E, N, K, per_pair, act, out, workspace, path,
                     exact, stream)


def moe_fp8_route(topk_ids: torch.Tensor, E: int, workspace: torch.Tensor | None, path: int, stream=None) -> None:
    """Group the pairs by expert into `workspace` for moe_fp8_routed (see ftq_moe_fp8_route)."""
    dev = _device_for(topk_ids, "topk_ids")
    T, top_k = topk_ids.shape
    ws_n = workspace.numel() if workspace is not None else 0
    _check(lib().ftq_moe_fp8_route(_here(topk_ids, "topk_ids", torch.int32, dev), E, T, top_k,
                                   _here(workspace, "workspace", torch.uint8, dev) if workspace is not None else None, ws_n,
                                   path, _stream_here(stream, dev)))


def moe_fp8_routed(w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, a_scale: torch.Tensor,
                   topk_ids: torch.Tensor, E: int, N: int, K: int, out: torch.Tensor, workspace: torch.Tensor | None,
                   path: int, per_pair: bool = False, act: int = 0, stream=None, exact: bool = False) -> torch.Tensor:
    """moe_fp8 on pairs already routed into `workspace` by moe_fp8_route."""
    return _fp8_call(lib().ftq_moe_fp8_routed, w, w_scale, a, a_scale, topk_ids, E, N, K, per_pair, act, out, workspace,
                     path, exact, stream)


# ---- training the router and low-rank adapters beside frozen experts ---------

def balance_workspace_bytes(T: int, E: int, top_k: int, sequences: int = 1) -> int:
    r = lib().ftq_moe_balance_workspace_bytes(T, E, top_k, sequences)
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def _sequences(offsets, valid, T, dev):
    """(address of offsets, number of sequences, address of valid)."""
    if offsets is not None and (offsets.dim() != 1 or offsets.shape[0] < 2):
        raise ValueError("offsets must be [sequences + 1]")
    return (_here(offsets, "offsets", torch.int32, dev) if offsets is not None else None,
            offsets.shape[0] - 1 if offsets is not None else 1,
            _here(valid, "valid", torch.bool, dev, (T,)) if valid is not None else None)


def _ids(topk_ids, T, dev):
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError(f"topk_ids must be [{T}, top_k]")
    return _here(topk_ids, "topk_ids", torch.int32, dev), topk_ids.shape[1]


def moe_balance(logits: torch.Tensor, topk_ids: torch.Tensor, score: int = SCORE_SOFTMAX, offsets: torch.Tensor | None = None,
                valid: torch.Tensor | None = None, loss: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                tokens: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Balance loss of the sequences offsets [S + 1] delimits (None: one of all rows), rows where valid [T] is False
    left out -> (fp32 loss [S], int32 counts [S, E], int32 tokens [S]) (see ftq_moe_balance)."""
    dev = _device_for(logits, "logits")
    p, dt, ld = _rows(logits, "logits", dev)
    T, E = logits.shape
    ids, top_k = _ids(topk_ids, T, dev)
    off, S, ok = _sequences(offsets, valid, T, dev)
    if loss is None:
        loss = _empty((S,), torch.float32, logits.device, stream)
    if counts is None:
        counts = _empty((S, E), torch.int32, logits.device, stream)
    if tokens is None:
        tokens = _empty((S,), torch.int32, logits.device, stream)
    if workspace is None:
        workspace = _empty(balance_workspace_bytes(T, E, top_k, S), torch.uint8, logits.device, stream)
    _check(lib().ftq_moe_balance(p, dt, ld, ids, ok, off, _here(counts, "counts", torch.int32, dev, (S, E)),
                                 _here(tokens, "tokens", torch.int32, dev, (S,)), _here(loss, "loss", torch.float32, dev, (S,)),
                                 T, E, top_k, S, score, _here(workspace, "workspace", torch.uint8, dev), workspace.numel(),
                                 _stream_here(stream, dev)))
    return loss, counts, tokens


def moe_topk_backward(logits: torch.Tensor, topk_ids: torch.Tensor, d_gates: torch.Tensor | None = None,
                      score: int = SCORE_SOFTMAX, renorm: bool = True, scale: float = 1.0, d_loss: torch.Tensor | None = None,
                      counts: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                      offsets: torch.Tensor | None = None, valid: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of the logits from those of moe_topk's gates and of moe_balance's losses (either may be None), in the
    logits' type (see ftq_moe_topk_backward)."""
    dev = _device_for(logits, "logits")
    p, dt, ld = _rows(logits, "logits", dev)
    T, E = logits.shape
    ids, top_k = _ids(topk_ids, T, dev)
    off, S, ok = _sequences(offsets, valid, T, dev)
    if d_loss is not None and (counts is None or tokens is None):
        raise ValueError("d_loss needs counts and tokens")
    if out is None:
        out = _empty((T, E), logits.dtype, logits.device, stream)
    if out.shape != (T, E) or out.dtype != logits.dtype:
        raise ValueError(f"out must be {logits.dtype} {(T, E)}")
    po, _, ldo = _rows(out, "out", dev)
    _check(lib().ftq_moe_topk_backward(
        p, dt, ld, ids, _here(d_gates, "d_gates", torch.float32, dev, (T, top_k)) if d_gates is not None else None,
        _here(counts, "counts", torch.int32, dev, (S, E)) if d_loss is not None else None,
        _here(tokens, "tokens", torch.int32, dev, (S,)) if d_loss is not None else None,
        _here(d_loss, "d_loss", torch.float32, dev, (S,)) if d_loss is not None else None, ok, off, po, ldo, T, E, top_k, S,
        score, int(renorm), scale, _stream_here(stream, dev)))
    return out


def combine_topk_backward(d_out: torch.Tensor, y: torch.Tensor, gates: torch.Tensor, d_y: torch.Tensor | None = None,
                          d_y_dtype: torch.dtype = torch.float32, d_gates: torch.Tensor | None = None, stream=None):
    """Gradient of combine_topk: fp32 d_out [T, N], y [T*top_k, N], gates [T, top_k] -> (d_y [T*top_k, N] in the type
    of the given buffer or d_y_dtype, fp32 d_gates [T, top_k])."""
    dev = _device_for(d_out, "d_out")
    if d_out.dim() != 2 or gates.dim() != 2:
        raise ValueError("d_out must be [T, N] and gates [T, top_k]")
    (T, N), top_k = d_out.shape, gates.shape[1]
    if d_y is None:
        d_y = _empty((T * top_k, N), d_y_dtype, d_out.device, stream)
    if d_gates is None:
        d_gates = _empty((T, top_k), torch.float32, d_out.device, stream)
    if d_y.dtype not in _DTYPE:
        raise ValueError(f"d_y must be float32, float16 or bfloat16, got {d_y.dtype}")
    _check(lib().ftq_moe_combine_topk_backward(
        _here(d_out, "d_out", torch.float32, dev), _here(y, "y", torch.float32, dev, (T * top_k, N)),
        _here(gates, "gates", torch.float32, dev, (T, top_k)), _here(d_y, "d_y", d_y.dtype, dev, (T * top_k, N)), _DTYPE[d_y.dtype],
        _here(d_gates, "d_gates", torch.float32, dev, (T, top_k)), T, top_k, N, _stream_here(stream, dev)))
    return d_y, d_gates


def lora_select_path(L: int, T: int, top_k: int) -> int:
    r = lib().ftq_lora_select_path(L, T, top_k)
    if r < 0:
        raise FtqError(-r, last_error())
    return r


def lora_workspace_bytes(L: int, R: int, K: int, N: int, T: int, top_k: int, dtype: torch.dtype, path: int = PATH_AUTO) -> int:
    r = lib().ftq_lora_workspace_bytes(L, R, K, N, T, top_k, _DTYPE[dtype], path)
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def lora_backward_workspace_bytes(L: int, R: int, K: int, N: int, T: int, top_k: int, dtype: torch.dtype) -> int:
    r = lib().ftq_lora_backward_workspace_bytes(L, R, K, N, T, top_k, _DTYPE[dtype])
    if r < 0:
        raise FtqError(ERR_INVALID_ARG, last_error())
    return r


def _adapters(x, a, b, topk_ids, per_pair, scale, dev):
    """(L, R, K, N, T, top_k) of a call, with its shapes checked, and the addresses of a, b, scale and topk_ids."""
    if a.dim() != 3 or b.dim() != 3 or topk_ids.dim() != 2 or x.dim() != 2:
        raise ValueError("need x [rows, K], a [L, R, K], b [L, N, R] and topk_ids [T, top_k]")
    (L, R, K), N, (T, top_k) = a.shape, b.shape[1], topk_ids.shape
    rows = T * top_k if per_pair else T
    if x.shape != (rows, K):
        raise ValueError(f"x must have the shape {(rows, K)}, got {tuple(x.shape)}")
    return (L, R, K, N, T, top_k), (_here(a, "a", x.dtype, dev), _here(b, "b", x.dtype, dev, (L, N, R)),
                                    _here(scale, "scale", torch.float32, dev, (L,)) if scale is not None else None,
                                    _here(topk_ids, "topk_ids", torch.int32, dev))


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, topk_ids: torch.Tensor, scale: torch.Tensor | None = None,
         base: torch.Tensor | None = None, per_pair: bool = False, path: int = PATH_AUTO, out: torch.Tensor | None = None,
         out_dtype: torch.dtype | None = None, h: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Low-rank adapters a [L, R, K], b [L, N, R] on the rows x [T or T*top_k, K] (may be strided): out [T*top_k, N] =
    base + scale * b (a x) with the adapter that topk_ids [T, top_k] names (ids outside [0, L): base alone), in base's type,
    without one in out_dtype or else x's.  out may be base itself; h (fp32 [T*top_k, R]) keeps a x for lora_backward (see ftq_lora)."""
    dev = _device_for(x, "x")
    px, dt, ldx = _rows(x, "x", dev)
    (L, R, K, N, T, top_k), (pa, pb, ps, ids) = _adapters(x, a, b, topk_ids, per_pair, scale, dev)
    pairs = T * top_k
    pbase, dbase, ldbase = _rows(base, "base", dev) if base is not None else (None, None, 0)
    if out is None:
        out = _empty((pairs, N), base.dtype if base is not None else out_dtype or x.dtype, x.device, stream)
    if out_dtype is not None and out_dtype != out.dtype:
        raise ValueError(f"out is {out.dtype} (as base or the buffer given), out_dtype {out_dtype}")
    po, do, ldo = _rows(out, "out", dev)
    if out.shape != (pairs, N) or (base is not None and (base.shape != (pairs, N) or dbase != do)):
        raise ValueError(f"out and base must be {(pairs, N)} of one type")
    if workspace is None:
        need = lora_workspace_bytes(L, R, K, N, T, top_k, x.dtype, path)
        workspace = _empty(need, torch.uint8, x.device, stream) if need else None
    _check(lib().ftq_lora(
        px, ldx, pa, pb, ps, ids, pbase, ldbase, po, ldo, _here(h, "h", torch.float32, dev, (pairs, R)) if h is not None else None,
        dt, do, L, R, K, N, T, top_k, int(per_pair), _here(workspace, "workspace", torch.uint8, dev) if workspace is not None else None,
        workspace.numel() if workspace is not None else 0, path, _stream_here(stream, dev)))
    return out


def lora_backward(d_out: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, topk_ids: torch.Tensor,
                  h: torch.Tensor, scale: torch.Tensor | None = None, base: torch.Tensor | None = None, per_pair: bool = False,
                  d_x: torch.Tensor | None = None, d_a: torch.Tensor | None = None, d_b: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None):
    """Gradients of lora: d_out [T*top_k, N] (x's type; may be strided) and the forward call's inputs and h -> (d_x
    [rows, K] in x's type, plus base if given; fp32 d_a [L, R, K], d_b [L, N, R]) (see ftq_lora_backward)."""
    dev = _device_for(x, "x")
    px, dt, ldx = _rows(x, "x", dev)
    (L, R, K, N, T, top_k), (pa, pb, ps, ids) = _adapters(x, a, b, topk_ids, per_pair, scale, dev)
    pd, dd, ldd = _rows(d_out, "d_out", dev)
    if d_out.shape != (T * top_k, N) or dd != dt:
        raise ValueError(f"d_out must be {x.dtype} {(T * top_k, N)}")
    if d_x is None:
        d_x = _empty(tuple(x.shape), x.dtype, x.device, stream)
    if d_a is None:
        d_a = _empty((L, R, K), torch.float32, x.device, stream)
    if d_b is None:
        d_b = _empty((L, N, R), torch.float32, x.device, stream)
    if workspace is None:
        need = lora_backward_workspace_bytes(L, R, K, N, T, top_k, x.dtype)
        workspace = _empty(need, torch.uint8, x.device, stream) if need else None
    shape = tuple(x.shape)
    _check(lib().ftq_lora_backward(
        pd, ldd, px, ldx, pa, pb, ps, ids, _here(h, "h", torch.float32, dev, (T * top_k, R)),
        _here(base, "base", x.dtype, dev, shape) if base is not None else None, _here(d_x, "d_x", x.dtype, dev, shape),
        _here(d_a, "d_a", torch.float32, dev, (L, R, K)), _here(d_b, "d_b", torch.float32, dev, (L, N, R)), dt, L, R, K, N, T, top_k,
        int(per_pair), _here(workspace, "workspace", torch.uint8, dev) if workspace is not None else None,
        workspace.numel() if workspace is not None else 0, _stream_here(stream, dev)))
    return d_x, d_a, d_b
