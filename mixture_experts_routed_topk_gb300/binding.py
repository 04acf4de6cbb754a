"""ctypes binding of ``libmoe_gb300.so`` (the C ABI in ``include/moe_routed_experts.h``).

Argument marshalling only: every function takes torch tensors, checks that they are what the C
entry point expects (device, dtype, contiguity, shape), passes their device pointers and sizes to
the entry point of the same name, and raises :class:`MoeError` on a non-``MOE_OK`` status. All
computation runs in the library's CUDA kernels; there is no fallback of any kind, and a missing
library raises at the first call.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

MOE_OK = 0
MOE_SCORES_F32 = 0
MOE_SCORES_BF16 = 1
MOE_DEV_BAD_EXPERT_ID = 1
MOE_DEV_TIMEOUT = 2
MOE_DEV_BAD_TARGET = 4
MOE_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

WS_REGIONS = (
    "status", "counts", "offsets", "tiles1", "tiles2", "block_counts", "block_bases",
    "perm", "inv", "xp", "h", "rms", "ready", "y", "total",
)
MOE_WEIGHT_W13 = 0
MOE_WEIGHT_W2 = 1
MXWS_REGIONS = (
    "status", "counts", "offsets", "tiles", "tiles2", "block_counts", "block_bases",
    "perm", "inv", "xq", "xs", "hq", "hs", "y", "total",
)

_lock = threading.Lock()
_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {message} (status {status})")
        self.status = status


def library_path() -> str:
    return _build.LIBRARY


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIBRARY
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library {p} is missing; build it with mixture_experts_routed_topk_gb300.build.build()"
            )
        lib = ctypes.CDLL(p)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        sig = {
            "moe_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_workspace_layout": ([i64, i32, i32, i32, i32, vp], ctypes.c_int),
            "moe_routing_workspace_bytes": ([i64, i32, i32], sz),
            "moe_routing": ([vp, i64, i32, i32, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
            "moe_routed_experts_fwd": (
                [vp, vp, vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_mega_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_mega_workspace_layout": ([i64, i32, i32, i32, i32, vp], ctypes.c_int),
            "moe_routed_experts_fwd_mega": (
                [vp, vp, vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_fwd_mega_stages": (
                [vp, vp, vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_routed_experts_fwd_rmsnorm": (
                [vp, vp, vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, ctypes.c_float, vp, sz, vp], ctypes.c_int),
            "moe_fwd_dispatch": ([vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_fwd_gemm1": ([vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_fwd_gemm2": ([vp, i32, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_fwd_combine": ([vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_get_status": ([vp, ctypes.POINTER(ctypes.c_uint32), vp], ctypes.c_int),
            "moe_routing_static_scratch": ([vp, i64, i32, i32, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "moe_selftest_wait_timeout": ([ctypes.c_uint32, vp, vp], ctypes.c_int),
            "moe_bwd_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_routed_experts_bwd": (
                [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_bwd_stages": (
                [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, sz, vp],
                ctypes.c_int),
            "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "moe_mxfp8_weight_bytes": ([i32, i32, i32, i32, vp, vp], ctypes.c_int),
            "moe_mxfp8_prepare_weight": ([i32, vp, i32, i32, i32, vp, sz, vp, sz, vp], ctypes.c_int),
            "moe_mxfp8_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_mxfp8_workspace_layout": ([i64, i32, i32, i32, i32, vp], ctypes.c_int),
            "moe_routed_experts_fwd_mxfp8": (
                [vp, vp, vp, i32, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_nvfp4_weight_bytes": ([i32, i32, i32, i32, vp, vp], ctypes.c_int),
            "moe_nvfp4_prepare_weight": ([i32, vp, i32, i32, i32, vp, sz, vp, sz, vp], ctypes.c_int),
            "moe_nvfp4_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_nvfp4_workspace_layout": ([i64, i32, i32, i32, i32, vp], ctypes.c_int),
            "moe_fwd_nvfp4_stages": (
                [vp, vp, vp, i32, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, i64, i32, i32, i32, i32, i32,
                 i32, vp, sz, vp], ctypes.c_int),
            "moe_routed_experts_fwd_nvfp4": (
                [vp, vp, vp, i32, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, i64, i32, i32, i32, i32, vp, sz,
                 vp], ctypes.c_int),
            "moe_fwd_mxfp8_stages": (
                [vp, vp, vp, i32, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_layernorm_fwd": ([vp, vp, vp, i32, i32, vp, vp, vp, i64, i32, ctypes.c_float, vp], ctypes.c_int),
            "moe_layernorm_bwd_workspace_bytes": ([i64, i32], sz),
            "moe_layernorm_bwd": (
                [vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, i64, i32, vp, sz, vp], ctypes.c_int),
            "moe_router_topk_fwd": ([vp, i32, vp, vp, i64, i32, i32, i32, vp], ctypes.c_int),
            "moe_router_topk_bwd": ([vp, i32, vp, vp, vp, i64, i32, i32, i32, vp], ctypes.c_int),
            "moe_lm_workspace_bytes": ([i64, i32, i32, i32], sz),
            "moe_lm_ce_fwd": ([vp, vp, vp, i32, vp, vp, i64, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_lm_ce_bwd": ([vp, vp, vp, i32, vp, vp, vp, vp, i64, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_lm_distill_fwd": (
                [vp, vp, vp, vp, ctypes.c_float, vp, vp, i64, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_lm_distill_bwd": (
                [vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, i64, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_block_norm_fwd": (
                [vp, vp, vp, vp, i32, vp, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp, i64, i32, vp],
                ctypes.c_int),
            "moe_block_norm_bwd_workspace_bytes": ([i64, i32], sz),
            "moe_block_norm_bwd": (
                [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, i64, i32, vp,
                 sz, vp], ctypes.c_int),
            "moe_few_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
            "moe_routed_experts_fwd_few": (
                [vp, vp, vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_layer_fwd_few": (
                [vp, vp, i32, i32, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp], ctypes.c_int),
            "moe_sample": ([vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, i32, vp], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def moe_status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status, moe_status_string(status))


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_routing_outputs(counts, offsets, perm, inv, T: int, E: int, K: int):
    """int32 CUDA outputs of the routing calls, large enough for what the kernels write: counts [E],
    offsets [E+1], perm and inv [T*K]."""
    for name, t, n in (("counts", counts, E), ("offsets", offsets, E + 1), ("perm", perm, T * K),
                       ("inv", inv, T * K)):
        _need(t, name, torch.int32)
        if t.numel() < n:
            raise ValueError(f"{name} must hold at least {n} int32, got {t.numel()}")


def _need_status_word(t):
    """A caller-owned device status word: the library clears and ORs one whole uint32."""
    _need(t, "device_status", (torch.int32, torch.uint8))
    if t.numel() * t.element_size() < 4:
        raise ValueError(f"device_status must hold at least 4 bytes, got {t.numel() * t.element_size()}")
    if t.data_ptr() % 4:
        raise ValueError("device_status must be 4-byte aligned")


def _dims(x, topk_ids, w13):
    T, D = x.shape
    E, two, F, D2 = w13.shape
    if two != 2 or D2 != D:
        raise ValueError(f"w13 must be [E,2,F,D] with D={D}, got {tuple(w13.shape)}")
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T,K]")
    return T, D, F, E, topk_ids.shape[1]


# ----------------------------------------------------------------------------------- sizes

def moe_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(load().moe_workspace_bytes(T, D, F, E, K))


def moe_workspace_layout(T: int, D: int, F: int, E: int, K: int) -> dict:
    arr = (ctypes.c_size_t * len(WS_REGIONS))()
    _check("moe_workspace_layout", load().moe_workspace_layout(T, D, F, E, K, ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(WS_REGIONS, (int(v) for v in arr)))


def moe_mega_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(load().moe_mega_workspace_bytes(T, D, F, E, K))


def moe_mega_workspace_layout(T: int, D: int, F: int, E: int, K: int) -> dict:
    arr = (ctypes.c_size_t * len(WS_REGIONS))()
    _check("moe_mega_workspace_layout",
           load().moe_mega_workspace_layout(T, D, F, E, K, ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(WS_REGIONS, (int(v) for v in arr)))


def moe_routing_workspace_bytes(T: int, E: int, K: int) -> int:
    return int(load().moe_routing_workspace_bytes(T, E, K))


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A device byte buffer for the workspace (torch's allocator aligns it to 256 bytes or more)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------------------ entry points

def moe_routing(topk_ids, num_experts: int, counts, offsets, perm, inv, workspace, stream=None) -> None:
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, K = topk_ids.shape
    _need_routing_outputs(counts, offsets, perm, inv, T, int(num_experts), K)
    _need(workspace, "workspace", torch.uint8)
    _check("moe_routing", load().moe_routing(
        _ptr(topk_ids), T, int(num_experts), K, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
        _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_routed_experts_fwd(x, topk_ids, topk_scores, w13, w2, out, workspace, stream=None) -> None:
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w13, "w13", torch.bfloat16, 4)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    T, D, F, E, K = _dims(x, topk_ids, w13)
    if tuple(w2.shape) != (E, D, F) or tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K):
        raise ValueError("inconsistent shapes among w2 [E,D,F], out [T,D], topk_scores [T,K]")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_routed_experts_fwd", load().moe_routed_experts_fwd(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13), _ptr(w2), _ptr(out),
        T, D, F, E, K, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_routed_experts_fwd_mega(x, topk_ids, topk_scores, w13, w2, out, workspace, stream=None) -> None:
    """The forward pass with both grouped GEMMs in one fused pipeline; the workspace is
    moe_mega_workspace_bytes(T, D, F, E, K) bytes. Bit-identical to moe_routed_experts_fwd."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w13, "w13", torch.bfloat16, 4)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    T, D, F, E, K = _dims(x, topk_ids, w13)
    if tuple(w2.shape) != (E, D, F) or tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K):
        raise ValueError("inconsistent shapes among w2 [E,D,F], out [T,D], topk_scores [T,K]")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_routed_experts_fwd_mega", load().moe_routed_experts_fwd_mega(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13), _ptr(w2), _ptr(out),
        T, D, F, E, K, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


MEGA_STAGES = 3  # dispatch, both GEMMs in one grid, combine


def moe_fwd_mega_stages(x, topk_ids, topk_scores, w13, w2, out, workspace, stage_begin: int, stage_end: int,
                        stream=None) -> None:
    """Stages [stage_begin, stage_end) of moe_routed_experts_fwd_mega (MEGA_STAGES in all)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w13, "w13", torch.bfloat16, 4)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    T, D, F, E, K = _dims(x, topk_ids, w13)
    if tuple(w2.shape) != (E, D, F) or tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K):
        raise ValueError("inconsistent shapes among w2 [E,D,F], out [T,D], topk_scores [T,K]")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_fwd_mega_stages", load().moe_fwd_mega_stages(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13), _ptr(w2), _ptr(out),
        T, D, F, E, K, int(stage_begin), int(stage_end), _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_routed_experts_fwd_rmsnorm(x, topk_ids, topk_scores, w13, w2, out, workspace, eps: float = 1e-6,
                                   stream=None) -> None:
    """The forward pass with route-wise RMSNorm of each expert output before the score weighting."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w13, "w13", torch.bfloat16, 4)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    T, D, F, E, K = _dims(x, topk_ids, w13)
    if tuple(w2.shape) != (E, D, F) or tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K):
        raise ValueError("inconsistent shapes among w2 [E,D,F], out [T,D], topk_scores [T,K]")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_routed_experts_fwd_rmsnorm", load().moe_routed_experts_fwd_rmsnorm(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13), _ptr(w2), _ptr(out),
        T, D, F, E, K, float(eps), _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_fwd_dispatch(x, topk_ids, dims, workspace, stream=None) -> None:
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, D, F, E, K = dims
    _check("moe_fwd_dispatch", load().moe_fwd_dispatch(
        _ptr(x), _ptr(topk_ids), T, D, F, E, K, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_fwd_gemm1(w13, dims, workspace, stream=None) -> None:
    _need(w13, "w13", torch.bfloat16, 4)
    T, D, F, E, K = dims
    _check("moe_fwd_gemm1", load().moe_fwd_gemm1(
        _ptr(w13), T, D, F, E, K, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_fwd_gemm2(topk_scores, w2, dims, workspace, stream=None) -> None:
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w2, "w2", torch.bfloat16, 3)
    T, D, F, E, K = dims
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_fwd_gemm2", load().moe_fwd_gemm2(
        _ptr(topk_scores), sd, _ptr(w2), T, D, F, E, K, _ptr(workspace), workspace.numel(),
        _stream_handle(stream)))


def moe_fwd_combine(topk_ids, out, dims, workspace, stream=None) -> None:
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(out, "out", torch.bfloat16, 2)
    T, D, F, E, K = dims
    _check("moe_fwd_combine", load().moe_fwd_combine(
        _ptr(topk_ids), _ptr(out), T, D, F, E, K, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_routing_static_scratch(topk_ids, num_experts: int, counts, offsets, perm, inv, device_status=None,
                               stream=None) -> None:
    """Routing without a workspace: its scratch is a fixed ~2 MiB array inside the library.

    For callers that cannot allocate device memory where they call the layer (an engine whose
    device memory is all owned by another allocator, a host program with no allocator at hand).
    The first call on a device looks up the array's address; make it before any stream capture.
    Calls share the array, so calls whose GPU work overlaps race: order them on one stream.
    """
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, K = topk_ids.shape
    _need_routing_outputs(counts, offsets, perm, inv, T, int(num_experts), K)
    if device_status is not None:
        _need_status_word(device_status)
    _check("moe_routing_static_scratch", load().moe_routing_static_scratch(
        _ptr(topk_ids), T, int(num_experts), K, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
        _ptr(device_status), _stream_handle(stream)))


def moe_bwd_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(load().moe_bwd_workspace_bytes(T, D, F, E, K))


BWD_STAGES = 7  # dispatch, recompute, dgrad down, dgrad gate/up, wgrad down, wgrad gate/up, reduce
BWD_STAGE_NAMES = ("dispatch", "recompute", "dgrad_down", "dgrad_gate_up", "wgrad_down", "wgrad_gate_up", "reduce")


def moe_routed_experts_bwd(x, topk_ids, topk_scores, w13, w2, dout, dx, dscores, dw13, dw2, workspace,
                           stream=None) -> None:
    """Gradients of the layer: dx [T,D] bf16, dscores [T,K] fp32, dw13 [E,2,F,D] and dw2 [E,D,F] bf16."""
    args, dims = _bwd_args(x, topk_ids, topk_scores, w13, w2, dout, dx, dscores, dw13, dw2, workspace)
    _check("moe_routed_experts_bwd", load().moe_routed_experts_bwd(
        *args, *dims, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def moe_bwd_stages(x, topk_ids, topk_scores, w13, w2, dout, dx, dscores, dw13, dw2, workspace, stage_begin: int,
                   stage_end: int, stream=None) -> None:
    """Backward stages stage_begin .. stage_end-1 (BWD_STAGE_NAMES) on one workspace, in order."""
    args, dims = _bwd_args(x, topk_ids, topk_scores, w13, w2, dout, dx, dscores, dw13, dw2, workspace)
    _check("moe_bwd_stages", load().moe_bwd_stages(
        *args, *dims, int(stage_begin), int(stage_end), _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def _bwd_args(x, topk_ids, topk_scores, w13, w2, dout, dx, dscores, dw13, dw2, workspace):
    """Checked pointer arguments and (T, D, F, E, K) of the backward entry points."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(w13, "w13", torch.bfloat16, 4)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(dout, "dout", torch.bfloat16, 2)
    _need(dx, "dx", torch.bfloat16, 2)
    _need(dscores, "dscores", torch.float32, 2)
    _need(dw13, "dw13", torch.bfloat16, 4)
    _need(dw2, "dw2", torch.bfloat16, 3)
    _need(workspace, "workspace", torch.uint8)
    T, D, F, E, K = _dims(x, topk_ids, w13)
    for name, t, shape in (("w2", w2, (E, D, F)), ("dout", dout, (T, D)), ("dx", dx, (T, D)),
                           ("dscores", dscores, (T, K)), ("dw13", dw13, (E, 2, F, D)), ("dw2", dw2, (E, D, F)),
                           ("topk_scores", topk_scores, (T, K))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    return ((_ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13), _ptr(w2), _ptr(dout), _ptr(dx),
             _ptr(dscores), _ptr(dw13), _ptr(dw2)), (T, D, F, E, K))


def moe_selftest_wait_timeout(timeout_us: int, device_status, stream=None) -> None:
    """Runs a kernel whose bounded wait must run out; device_status receives MOE_DEV_TIMEOUT."""
    _need_status_word(device_status)
    _check("moe_selftest_wait_timeout", load().moe_selftest_wait_timeout(
        int(timeout_us), _ptr(device_status), _stream_handle(stream)))


def moe_get_status(workspace, stream=None) -> int:
    """The device status bits of a workspace (synchronises the stream)."""
    _need(workspace, "workspace", torch.uint8)
    bits = ctypes.c_uint32(0)
    _check("moe_get_status", load().moe_get_status(_ptr(workspace), ctypes.byref(bits), _stream_handle(stream)))
    return int(bits.value)


# ------------------------------------------------------------------------------------- MXFP8

def moe_mxfp8_weight_bytes(which: int, D: int, F: int, E: int) -> tuple[int, int]:
    """(data bytes, scale bytes) of a prepared MXFP8 weight (which = MOE_WEIGHT_W13 or _W2)."""
    data, scales = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_mxfp8_weight_bytes", load().moe_mxfp8_weight_bytes(
        int(which), D, F, E, ctypes.byref(data), ctypes.byref(scales)))
    return int(data.value), int(scales.value)


def moe_mxfp8_prepare_weight(which: int, w, data=None, scales=None, stream=None):
    """Quantizes w13 [E,2,F,D] (which = MOE_WEIGHT_W13) or w2 [E,D,F] (MOE_WEIGHT_W2) to MXFP8.

    Returns (data, scales): uint8 device tensors of E4M3 codes (w's element order) and UE8M0
    scales (grouped per GEMM tile); pass them to preallocate.
    """
    _need(w, "w", torch.bfloat16)
    if which == MOE_WEIGHT_W13:
        if w.dim() != 4 or w.shape[1] != 2:
            raise ValueError(f"w13 must be [E,2,F,D], got {tuple(w.shape)}")
        E, _, F, D = w.shape
    elif which == MOE_WEIGHT_W2:
        if w.dim() != 3:
            raise ValueError(f"w2 must be [E,D,F], got {tuple(w.shape)}")
        E, D, F = w.shape
    else:
        raise ValueError("which must be MOE_WEIGHT_W13 or MOE_WEIGHT_W2")
    nd, ns = moe_mxfp8_weight_bytes(which, D, F, E)
    if data is None:
        data = torch.empty(nd, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(ns, dtype=torch.uint8, device=w.device)
    _need(data, "data", torch.uint8)
    _need(scales, "scales", torch.uint8)
    _check("moe_mxfp8_prepare_weight", load().moe_mxfp8_prepare_weight(
        int(which), _ptr(w), D, F, E, _ptr(data), data.numel(), _ptr(scales), scales.numel(),
        _stream_handle(stream)))
    return data, scales


def moe_mxfp8_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(load().moe_mxfp8_workspace_bytes(T, D, F, E, K))


def moe_mxfp8_workspace_layout(T: int, D: int, F: int, E: int, K: int) -> dict:
    arr = (ctypes.c_size_t * len(MXWS_REGIONS))()
    _check("moe_mxfp8_workspace_layout",
           load().moe_mxfp8_workspace_layout(T, D, F, E, K, ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(MXWS_REGIONS, (int(v) for v in arr)))


MX_STAGES = 4


def moe_routed_experts_fwd_mxfp8(x, topk_ids, topk_scores, w13_mx, w2_mx, out, workspace, dims_FE=None,
                                 stream=None) -> None:
    """The MXFP8 forward. w13_mx, w2_mx: (data, scales) from moe_mxfp8_prepare_weight.

    dims_FE = (F, E); the prepared weights are flat byte tensors, so F and E come from here.
    """
    moe_fwd_mxfp8_stages(x, topk_ids, topk_scores, w13_mx, w2_mx, out, workspace, dims_FE, 0, MX_STAGES, stream)


def moe_fwd_mxfp8_stages(x, topk_ids, topk_scores, w13_mx, w2_mx, out, workspace, dims_FE, stage_begin: int,
                         stage_end: int, stream=None) -> None:
    """Stages [stage_begin, stage_end) of the MXFP8 forward (0 dispatch, 1 gate/up, 2 down, 3 combine)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    for name, t in (("w13 data", w13_mx[0]), ("w13 scales", w13_mx[1]), ("w2 data", w2_mx[0]),
                    ("w2 scales", w2_mx[1])):
        _need(t, name, torch.uint8)
    if dims_FE is None:
        raise ValueError("dims_FE = (F, E) is required")
    T, D = x.shape
    K = topk_ids.shape[1]
    F, E = (int(v) for v in dims_FE)
    if tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K) or topk_ids.shape[0] != T:
        raise ValueError("inconsistent shapes among x [T,D], topk_ids/topk_scores [T,K], out [T,D]")
    for which, (d, sc) in ((MOE_WEIGHT_W13, w13_mx), (MOE_WEIGHT_W2, w2_mx)):
        nd, ns = moe_mxfp8_weight_bytes(which, D, F, E)
        if d.numel() < nd or sc.numel() < ns:
            raise ValueError("prepared weight buffers are smaller than moe_mxfp8_weight_bytes")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_fwd_mxfp8_stages", load().moe_fwd_mxfp8_stages(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13_mx[0]), _ptr(w13_mx[1]), _ptr(w2_mx[0]),
        _ptr(w2_mx[1]), _ptr(out), T, D, F, E, K, int(stage_begin), int(stage_end), _ptr(workspace),
        workspace.numel(), _stream_handle(stream)))


# ------------------------------------------------------------------------------------- NVFP4

def moe_nvfp4_weight_bytes(which: int, D: int, F: int, E: int) -> tuple[int, int]:
    """(data bytes, scale bytes) of a prepared NVFP4 weight (which = MOE_WEIGHT_W13 or _W2)."""
    data, scales = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_nvfp4_weight_bytes", load().moe_nvfp4_weight_bytes(
        int(which), D, F, E, ctypes.byref(data), ctypes.byref(scales)))
    return int(data.value), int(scales.value)


def moe_nvfp4_prepare_weight(which: int, w, data=None, scales=None, stream=None):
    """Quantizes w13 [E,2,F,D] or w2 [E,D,F] to NVFP4. Returns (data, scales) uint8 device tensors:
    packed E2M1 codes, and a 256-byte header holding the tensor scale followed by the UE4M3 scales."""
    _need(w, "w", torch.bfloat16)
    if which == MOE_WEIGHT_W13:
        if w.dim() != 4 or w.shape[1] != 2:
            raise ValueError(f"w13 must be [E,2,F,D], got {tuple(w.shape)}")
        E, _, F, D = w.shape
    elif which == MOE_WEIGHT_W2:
        if w.dim() != 3:
            raise ValueError(f"w2 must be [E,D,F], got {tuple(w.shape)}")
        E, D, F = w.shape
    else:
        raise ValueError("which must be MOE_WEIGHT_W13 or MOE_WEIGHT_W2")
    nd, ns = moe_nvfp4_weight_bytes(which, D, F, E)
    if data is None:
        data = torch.empty(nd, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(ns, dtype=torch.uint8, device=w.device)
    _need(data, "data", torch.uint8)
    _need(scales, "scales", torch.uint8)
    _check("moe_nvfp4_prepare_weight", load().moe_nvfp4_prepare_weight(
        int(which), _ptr(w), D, F, E, _ptr(data), data.numel(), _ptr(scales), scales.numel(), _stream_handle(stream)))
    return data, scales


def moe_nvfp4_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    return int(load().moe_nvfp4_workspace_bytes(T, D, F, E, K))


def moe_nvfp4_workspace_layout(T: int, D: int, F: int, E: int, K: int) -> dict:
    arr = (ctypes.c_size_t * len(MXWS_REGIONS))()
    _check("moe_nvfp4_workspace_layout",
           load().moe_nvfp4_workspace_layout(T, D, F, E, K, ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(MXWS_REGIONS, (int(v) for v in arr)))


def moe_routed_experts_fwd_nvfp4(x, topk_ids, topk_scores, w13_nv, w2_nv, out, workspace, dims_FE, x_scale: float,
                                 h_scale: float, stream=None) -> None:
    """The NVFP4 forward. w13_nv, w2_nv: (data, scales) from moe_nvfp4_prepare_weight; dims_FE = (F, E);
    x_scale, h_scale: the activations' tensor scales (calibration constants)."""
    moe_fwd_nvfp4_stages(x, topk_ids, topk_scores, w13_nv, w2_nv, out, workspace, dims_FE, x_scale, h_scale, 0,
                         MX_STAGES, stream)


def moe_fwd_nvfp4_stages(x, topk_ids, topk_scores, w13_nv, w2_nv, out, workspace, dims_FE, x_scale: float,
                         h_scale: float, stage_begin: int, stage_end: int, stream=None) -> None:
    """Stages [stage_begin, stage_end) of the NVFP4 forward (0 dispatch, 1 gate/up, 2 down, 3 combine)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_scores, "topk_scores", (torch.float32, torch.bfloat16), 2)
    _need(out, "out", torch.bfloat16, 2)
    _need(workspace, "workspace", torch.uint8)
    for name, t in (("w13 data", w13_nv[0]), ("w13 scales", w13_nv[1]), ("w2 data", w2_nv[0]),
                    ("w2 scales", w2_nv[1])):
        _need(t, name, torch.uint8)
    T, D = x.shape
    K = topk_ids.shape[1]
    F, E = (int(v) for v in dims_FE)
    if tuple(out.shape) != (T, D) or tuple(topk_scores.shape) != (T, K) or topk_ids.shape[0] != T:
        raise ValueError("inconsistent shapes among x [T,D], topk_ids/topk_scores [T,K], out [T,D]")
    for which, (d, sc) in ((MOE_WEIGHT_W13, w13_nv), (MOE_WEIGHT_W2, w2_nv)):
        nd, ns = moe_nvfp4_weight_bytes(which, D, F, E)
        if d.numel() < nd or sc.numel() < ns:
            raise ValueError("prepared weight buffers are smaller than moe_nvfp4_weight_bytes")
    sd = MOE_SCORES_BF16 if topk_scores.dtype == torch.bfloat16 else MOE_SCORES_F32
    _check("moe_fwd_nvfp4_stages", load().moe_fwd_nvfp4_stages(
        _ptr(x), _ptr(topk_ids), _ptr(topk_scores), sd, _ptr(w13_nv[0]), _ptr(w13_nv[1]), _ptr(w2_nv[0]),
        _ptr(w2_nv[1]), float(x_scale), float(h_scale), _ptr(out), T, D, F, E, K, int(stage_begin),
        int(stage_end), _ptr(workspace), workspace.numel(), _stream_handle(stream)))


# ------------------------------------- layer norm, norms around a block, router and vocabulary losses
#
# These calls are short on the GPU (a few microseconds at the smallest sizes), so their checks are too:
# one comparison per property and tensor, and the words for a refusal only once it is one.

def _refuse(t, name: str, dtype, shape, device: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _operand(t, name: str, dtype, shape, device: int) -> int:
    """The device pointer of a contiguous tensor of this dtype, shape and device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device)


_INT32_MAX = (1 << 31) - 1


def _int32(n: int, name: str) -> int:
    """A size that the library takes as a 32-bit number (ctypes would wrap a larger one around)."""
    if n > _INT32_MAX:
        raise ValueError(f"{name}: a size of {n} does not fit 32 bits")
    return n


def _rows(x, name: str, dtypes):
    """T, D, device and pointer of a contiguous [T, D] tensor of one of the dtypes."""
    if isinstance(x, torch.Tensor) and x.dtype in dtypes and x.dim() == 2 and x.is_cuda and x.is_contiguous():
        T, D = x.shape
        return T, _int32(D, name), x.get_device(), x.data_ptr()
    _need(x, name, tuple(dtypes), 2)


def _workspace(t, device: int) -> int:
    return _operand(t, "workspace", torch.uint8, (t.numel(),) if isinstance(t, torch.Tensor) else (0,), device)


def _stream_of(stream, device: int) -> int:
    """The handle of the call's stream. The library launches on the current device, so that has to be the tensors'."""
    current = torch._C._cuda_getDevice()
    if device != current:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(current)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != current:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{current}")
        return stream.cuda_stream
    return int(stream)


def _norm_params(x, D: int, device: int, *params):
    """The common MOE_DTYPE of the (name, [D] tensor or None) pairs, and their pointers (0 for None)."""
    dtype, ptrs = None, []
    for name, p in params:
        if p is None:
            ptrs.append(0)
            continue
        if dtype is None:
            if not isinstance(p, torch.Tensor) or p.dtype not in MOE_DTYPE:
                _need(p, name, tuple(MOE_DTYPE), 1)
            dtype = p.dtype
        ptrs.append(_operand(p, name, dtype, (D,), device))
    return MOE_DTYPE[dtype if dtype is not None else x.dtype], ptrs


def moe_layernorm_fwd(x, gamma, beta, y, mean, rstd, eps: float = 1e-5, stream=None) -> None:
    """Layer norm of the rows of x [T,D] (fp32, bf16 or fp16) into y; mean and rstd [T] fp32 are kept for
    the backward pass. gamma and beta [D] may be None (1 and 0), and have one dtype of their own. y may be x."""
    T, D, dev, px = _rows(x, "x", MOE_DTYPE)
    pd, (pg, pb) = _norm_params(x, D, dev, ("gamma", gamma), ("beta", beta))
    _check("moe_layernorm_fwd", load().moe_layernorm_fwd(
        px, pg, pb, MOE_DTYPE[x.dtype], pd, _operand(y, "y", x.dtype, (T, D), dev),
        _operand(mean, "mean", torch.float32, (T,), dev), _operand(rstd, "rstd", torch.float32, (T,), dev), T, D,
        float(eps), _stream_of(stream, dev)))


def moe_layernorm_bwd_workspace_bytes(T: int, D: int) -> int:
    return int(load().moe_layernorm_bwd_workspace_bytes(T, D)) if D <= _INT32_MAX else 0


def moe_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace, stream=None) -> None:
    """Layer norm's backward pass: dx, and dgamma and dbeta (either may be None) in the parameters' dtype.
    The workspace is moe_layernorm_bwd_workspace_bytes(T, D) bytes (None when neither is wanted). dx may be dy or x."""
    T, D, dev, px = _rows(x, "x", MOE_DTYPE)
    pd, (pg, pdg, pdb) = _norm_params(x, D, dev, ("gamma", gamma), ("dgamma", dgamma), ("dbeta", dbeta))
    _check("moe_layernorm_bwd", load().moe_layernorm_bwd(
        _operand(dy, "dy", x.dtype, (T, D), dev), px, pg, _operand(mean, "mean", torch.float32, (T,), dev),
        _operand(rstd, "rstd", torch.float32, (T,), dev), MOE_DTYPE[x.dtype], pd,
        _operand(dx, "dx", x.dtype, (T, D), dev), pdg, pdb, T, D, 0 if workspace is None else _workspace(workspace, dev),
        0 if workspace is None else workspace.numel(), _stream_of(stream, dev)))


def _gate(gate, x, T: int, D: int, device: int):
    """Whether the gate is one per token ([T,D] of x's dtype; else [D] of the parameters' or None), and its pointer."""
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        return 1, _operand(gate, "gate", x.dtype, (T, D), device)
    return 0, 0


def _optional(t, name: str, dtype, shape, device: int) -> int:
    return 0 if t is None else _operand(t, name, dtype, shape, device)


def moe_block_norm_fwd(block, residual, post_gamma, gate, pre_gamma, stream_out, normed, post_rstd, pre_rstd,
                       residual_scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """The RMS norms after and before a block, its gate and the residual's scale, in one pass over rows [T,D] (fp32,
    bf16 or fp16): stream_out = residual_scale residual + gate rms(block) post_gamma, normed = rms(stream_out) pre_gamma.
    post_rstd and pre_rstd [T] fp32 are kept for the backward pass; post_rstd None: no norm after the block. The gammas
    and a gate [D] (each may be None: 1) have one dtype of their own; a gate [T,D] has the rows'."""
    T, D, dev, pb = _rows(block, "block", MOE_DTYPE)
    per_token, pg = _gate(gate, block, T, D, dev)
    pd, (pp, pc, pn) = _norm_params(block, D, dev, ("post_gamma", post_gamma), ("gate", None if per_token else gate),
                                    ("pre_gamma", pre_gamma))
    dt, f32 = block.dtype, torch.float32
    _check("moe_block_norm_fwd", load().moe_block_norm_fwd(
        pb, _operand(residual, "residual", dt, (T, D), dev), pp, pg or pc, per_token, pn, MOE_DTYPE[dt], pd,
        float(residual_scale), float(eps), _operand(stream_out, "stream_out", dt, (T, D), dev),
        _operand(normed, "normed", dt, (T, D), dev), _optional(post_rstd, "post_rstd", f32, (T,), dev),
        _operand(pre_rstd, "pre_rstd", f32, (T,), dev), T, D, _stream_of(stream, dev)))


def moe_block_norm_bwd_workspace_bytes(T: int, D: int) -> int:
    return int(load().moe_block_norm_bwd_workspace_bytes(T, D)) if D <= _INT32_MAX else 0


def moe_block_norm_bwd(dstream, dnormed, block, stream_in, post_gamma, gate, pre_gamma, post_rstd, pre_rstd, dblock,
                       dresidual, dpost_gamma, dgate, dpre_gamma, workspace, residual_scale: float = 1.0,
                       stream=None) -> None:
    """The way back of moe_block_norm_fwd: dblock and dresidual [T,D], and dpost_gamma, dgate and dpre_gamma (each may
    be None), for the gradients dstream (None: 0) and dnormed of its outputs. stream_in is its stream_out; block may be
    None without a gate and a norm after the block. The workspace is moe_block_norm_bwd_workspace_bytes(T, D) bytes
    (None when no gradient of a [D] parameter is asked for)."""
    T, D, dev, pdn = _rows(dnormed, "dnormed", MOE_DTYPE)
    per_token, pg = _gate(gate, dnormed, T, D, dev)
    pd, (pp, pc, pn, pdp, pdc, pdpre) = _norm_params(
        dnormed, D, dev, ("post_gamma", post_gamma), ("gate", None if per_token else gate), ("pre_gamma", pre_gamma),
        ("dpost_gamma", dpost_gamma), ("dgate", None if per_token else dgate), ("dpre_gamma", dpre_gamma))
    dt, f32 = dnormed.dtype, torch.float32
    if per_token:
        pdc = _optional(dgate, "dgate", dt, (T, D), dev)
    _check("moe_block_norm_bwd", load().moe_block_norm_bwd(
        _optional(dstream, "dstream", dt, (T, D), dev), pdn, _optional(block, "block", dt, (T, D), dev),
        _operand(stream_in, "stream_in", dt, (T, D), dev), pp, pg or pc, per_token, pn,
        _optional(post_rstd, "post_rstd", f32, (T,), dev), _operand(pre_rstd, "pre_rstd", f32, (T,), dev),
        MOE_DTYPE[dt], pd, float(residual_scale), _operand(dblock, "dblock", dt, (T, D), dev),
        _operand(dresidual, "dresidual", dt, (T, D), dev), pdp, pdc, pdpre, T, D,
        0 if workspace is None else _workspace(workspace, dev), 0 if workspace is None else workspace.numel(),
        _stream_of(stream, dev)))


_LOGIT_DTYPES = (torch.float32, torch.bfloat16)


def _choices(topk_ids, T: int, dev: int):
    """K and the pointer of topk_ids [T, K]."""
    K = topk_ids.shape[1] if isinstance(topk_ids, torch.Tensor) and topk_ids.dim() == 2 else 0
    return _int32(K, "topk_ids"), _operand(topk_ids, "topk_ids", torch.int32, (T, K), dev)


def moe_router_topk_fwd(logits, topk_ids, topk_scores, normalize: bool = True, stream=None) -> None:
    """The K largest of each row of logits [T,E] (fp32 or bf16) into topk_ids [T,K] int32 and their scores
    into topk_scores [T,K] fp32: the softmax over the chosen (normalize) or over all E experts."""
    T, E, dev, pz = _rows(logits, "logits", _LOGIT_DTYPES)
    K, pi = _choices(topk_ids, T, dev)
    _check("moe_router_topk_fwd", load().moe_router_topk_fwd(
        pz, MOE_DTYPE[logits.dtype], pi, _operand(topk_scores, "topk_scores", torch.float32, (T, K), dev), T, E, K,
        1 if normalize else 0, _stream_of(stream, dev)))


def moe_router_topk_bwd(logits, topk_ids, dscores, dlogits, normalize: bool = True, stream=None) -> None:
    """dlogits [T,E] from dscores [T,K] (as moe_routed_experts_bwd writes them), for the logits, ids and
    normalize of moe_router_topk_fwd."""
    T, E, dev, pz = _rows(logits, "logits", _LOGIT_DTYPES)
    K, pi = _choices(topk_ids, T, dev)
    _check("moe_router_topk_bwd", load().moe_router_topk_bwd(
        pz, MOE_DTYPE[logits.dtype], pi, _operand(dscores, "dscores", torch.float32, (T, K), dev),
        _operand(dlogits, "dlogits", logits.dtype, (T, E), dev), T, E, K, 1 if normalize else 0,
        _stream_of(stream, dev)))


def moe_lm_workspace_bytes(T: int, D: int, V: int, K: int = 1) -> int:
    """Workspace of the moe_lm_* calls; K is the number of teacher entries per row (1 for cross entropy)."""
    return int(load().moe_lm_workspace_bytes(T, D, V, K)) if max(D, V, K) <= _INT32_MAX else 0


_BF16 = (torch.bfloat16,)


def _head(x, w):
    """T, D, V, device and the pointers of x [T, D] and w [V, D]."""
    T, D, dev, px = _rows(x, "x", _BF16)
    V = w.shape[0] if isinstance(w, torch.Tensor) and w.dim() == 2 else 0
    return T, D, _int32(V, "w"), dev, px, _operand(w, "w", torch.bfloat16, (V, D), dev)


def _teacher(teacher_ids, teacher_logits, T: int, dev: int):
    """K and the pointers of teacher_ids and teacher_logits [T, K]."""
    K = teacher_ids.shape[1] if isinstance(teacher_ids, torch.Tensor) and teacher_ids.dim() == 2 else 0
    return (_int32(K, "teacher_ids"), _operand(teacher_ids, "teacher_ids", torch.int32, (T, K), dev),
            _operand(teacher_logits, "teacher_logits", torch.float32, (T, K), dev))


def _vector(t, name: str, T: int, dev: int) -> int:
    return _operand(t, name, torch.float32, (T,), dev)


def _ignored(ignore_index) -> int:
    """ignore_index as a label can have it."""
    i = int(ignore_index)
    if not -_INT32_MAX - 1 <= i <= _INT32_MAX:
        raise ValueError(f"ignore_index {i} does not fit 32 bits, as the targets do")
    return i


def _grad(t, name: str, shape, dev: int) -> int:
    return 0 if t is None else _operand(t, name, torch.bfloat16, shape, dev)


def moe_lm_ce_fwd(x, w, targets, loss, lse, workspace, ignore_index: int = -100, stream=None) -> None:
    """Softmax cross entropy of the head z = x w^T without keeping z: loss and lse [T] fp32 for x [T,D] and
    w [V,D] (bf16) and targets [T] int32. Rows of ignore_index have loss 0; a target outside [0, V) sets
    MOE_DEV_BAD_TARGET in the workspace's status word and counts as ignored."""
    T, D, V, dev, px, pw = _head(x, w)
    _check("moe_lm_ce_fwd", load().moe_lm_ce_fwd(
        px, pw, _operand(targets, "targets", torch.int32, (T,), dev), _ignored(ignore_index), _vector(loss, "loss", T, dev),
        _vector(lse, "lse", T, dev), T, D, V, _workspace(workspace, dev), workspace.numel(), _stream_of(stream, dev)))


def moe_lm_ce_bwd(x, w, targets, lse, dloss, dx, dw, workspace, ignore_index: int = -100, stream=None) -> None:
    """dx [T,D] and dw [V,D] (bf16; either may be None) for the losses' gradients dloss [T] and the lse of
    moe_lm_ce_fwd."""
    T, D, V, dev, px, pw = _head(x, w)
    _check("moe_lm_ce_bwd", load().moe_lm_ce_bwd(
        px, pw, _operand(targets, "targets", torch.int32, (T,), dev), _ignored(ignore_index), _vector(lse, "lse", T, dev),
        _vector(dloss, "dloss", T, dev), _grad(dx, "dx", (T, D), dev), _grad(dw, "dw", (V, D), dev), T, D, V,
        _workspace(workspace, dev), workspace.numel(), _stream_of(stream, dev)))


def moe_lm_distill_fwd(x, w, teacher_ids, teacher_logits, loss, lse, workspace, temperature: float = 1.0,
                       stream=None) -> None:
    """tau^2 KL(p || q) of the head z = x w^T without keeping z: p is the softmax of a row's teacher_logits
    [T,K] fp32 at the temperature over the entries with teacher_ids [T,K] int32 >= 0, q the softmax of z at
    the temperature over the whole vocabulary. Rows without entries have loss 0."""
    T, D, V, dev, px, pw = _head(x, w)
    K, pi, pl = _teacher(teacher_ids, teacher_logits, T, dev)
    _check("moe_lm_distill_fwd", load().moe_lm_distill_fwd(
        px, pw, pi, pl, float(temperature), _vector(loss, "loss", T, dev), _vector(lse, "lse", T, dev), T, D, V, K,
        _workspace(workspace, dev), workspace.numel(), _stream_of(stream, dev)))


def moe_lm_distill_bwd(x, w, teacher_ids, teacher_logits, lse, dloss, dx, dw, workspace, temperature: float = 1.0,
                       stream=None) -> None:
    """dx [T,D] and dw [V,D] (bf16; either may be None) for the losses' gradients dloss [T] and the lse of
    moe_lm_distill_fwd."""
    T, D, V, dev, px, pw = _head(x, w)
    K, pi, pl = _teacher(teacher_ids, teacher_logits, T, dev)
    _check("moe_lm_distill_bwd", load().moe_lm_distill_bwd(
        px, pw, pi, pl, float(temperature), _vector(lse, "lse", T, dev), _vector(dloss, "dloss", T, dev),
        _grad(dx, "dx", (T, D), dev), _grad(dw, "dw", (V, D), dev), T, D, V, K, _workspace(workspace, dev),
        workspace.numel(), _stream_of(stream, dev)))


# ------------------------------------------------------------------------ a decoding step

def moe_few_workspace_bytes(T: int, D: int, F: int, E: int, K: int) -> int:
    """Workspace of moe_routed_experts_fwd_few and moe_layer_fwd_few."""
    return int(load().moe_few_workspace_bytes(T, D, F, E, K)) if max(D, F, E, K) <= _INT32_MAX else 0


def _experts(x, w13, w2):
    """T, D, F, E, device and the pointers of x [T,D], w13 [E,2,F,D] and w2 [E,D,F]."""
    T, D, dev, px = _rows(x, "x", _BF16)
    E, F = (w13.shape[0], w13.shape[2]) if isinstance(w13, torch.Tensor) and w13.dim() == 4 else (0, 0)
    return (T, D, _int32(F, "w13"), _int32(E, "w13"), dev, px, _operand(w13, "w13", torch.bfloat16, (E, 2, F, D), dev),
            _operand(w2, "w2", torch.bfloat16, (E, D, F), dev))


def moe_routed_experts_fwd_few(x, topk_ids, topk_scores, w13, w2, out, workspace, stream=None) -> None:
    """The layer for 1 to 32 tokens (T K at most 512), as moe_routed_experts_fwd: each chosen expert's weights are
    streamed once, by two kernels. The workspace is moe_few_workspace_bytes(T, D, F, E, K) bytes."""
    T, D, F, E, dev, px, p13, p2 = _experts(x, w13, w2)
    K, pi = _choices(topk_ids, T, dev)
    bf16 = isinstance(topk_scores, torch.Tensor) and topk_scores.dtype is torch.bfloat16
    ps = _operand(topk_scores, "topk_scores", torch.bfloat16 if bf16 else torch.float32, (T, K), dev)
    _check("moe_routed_experts_fwd_few", load().moe_routed_experts_fwd_few(
        px, pi, ps, MOE_SCORES_BF16 if bf16 else MOE_SCORES_F32, p13, p2,
        _operand(out, "out", torch.bfloat16, (T, D), dev), T, D, F, E, K, _workspace(workspace, dev), workspace.numel(),
        _stream_of(stream, dev)))


def moe_layer_fwd_few(x, logits, w13, w2, topk_ids, topk_scores, out, workspace, normalize: bool = True,
                      stream=None) -> None:
    """moe_router_topk_fwd on logits [T,E] (fp32 or bf16) into topk_ids and topk_scores, and the layer on its choice,
    without a launch between them. Limits and workspace as for moe_routed_experts_fwd_few."""
    T, D, F, E, dev, px, p13, p2 = _experts(x, w13, w2)
    K, pi = _choices(topk_ids, T, dev)
    bf16 = isinstance(logits, torch.Tensor) and logits.dtype is torch.bfloat16
    pz = _operand(logits, "logits", torch.bfloat16 if bf16 else torch.float32, (T, E), dev)
    _check("moe_layer_fwd_few", load().moe_layer_fwd_few(
        px, pz, 1 if bf16 else 0, 1 if normalize else 0, p13, p2, pi,
        _operand(topk_scores, "topk_scores", torch.float32, (T, K), dev), _operand(out, "out", torch.bfloat16, (T, D), dev),
        T, D, F, E, K, _workspace(workspace, dev), workspace.numel(), _stream_of(stream, dev)))


def moe_sample(logits, uniform, token, logprob=None, temperature=None, top_k=None, top_p=None, min_p=None,
               stream=None) -> None:
    """The next token [T] int32 of each row of logits [T,V] (fp32, bf16 or fp16) for the numbers uniform [T] fp32 in
    [0, 1), and the logarithm [T] fp32 of its probability among the tokens that were kept (None: not wanted).
    temperature, top_p and min_p [T] fp32 and top_k [T] int32 hold each row's own (None: 1, and off); a temperature of 0
    takes the largest logit. A row without a choice (nothing but -inf, or a NaN) gets token -1."""
    T, V, dev, pz = _rows(logits, "logits", MOE_DTYPE)
    f32, one = torch.float32, (T,)
    _check("moe_sample", load().moe_sample(
        pz, MOE_DTYPE[logits.dtype], _operand(uniform, "uniform", f32, one, dev),
        _optional(temperature, "temperature", f32, one, dev), _optional(top_k, "top_k", torch.int32, one, dev),
        _optional(top_p, "top_p", f32, one, dev), _optional(min_p, "min_p", f32, one, dev),
        _operand(token, "token", torch.int32, one, dev), _optional(logprob, "logprob", f32, one, dev), T, V,
        _stream_of(stream, dev)))
