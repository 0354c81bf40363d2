"""ctypes binding to libbfp8 (include/bfp8.h).

Argument marshalling only: every step of the computation runs in libbfp8's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There
is no fallback: if the library is missing or the device is not an sm_103
part, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libbfp8.so")

BFP8_OK = 0
BFP8_IN_BF16 = 0
BFP8_IN_F32 = 1
SCALE_FP32, SCALE_UE8M0 = 0, 1
SCHEDULE_AUTO, SCHEDULE_SWAP_AB, SCHEDULE_WIDE, SCHEDULE_GEMV = 0, 1, 2, 3
KSPLIT_AUTO, KSPLIT_STREAM_K, KSPLIT_CLUSTER, KSPLIT_NONE = 0, 1, 2, 3
PAIRS_AUTO, PAIRS_NEVER, PAIRS_ALWAYS = 0, 1, 2
STATUS_NAMES = {0: "BFP8_OK", 1: "BFP8_ERR_INVALID_ARG", 2: "BFP8_ERR_ALIGNMENT",
                3: "BFP8_ERR_UNSUPPORTED", 4: "BFP8_ERR_CUDA", 5: "BFP8_ERR_WORKSPACE",
                6: "BFP8_ERR_DEVICE_TIMEOUT"}

# Every symbol include/bfp8.h declares.
EXPORTS = ("bfp8_group_quant", "bfp8_group_quant_ex", "bfp8_scale_ceil_ue8m0", "bfp8_scale_ld", "bfp8_gemm", "bfp8_gemm_ex",
           "bfp8_gemm_workspace_size", "bfp8_gemm_plan", "bfp8_plan_unit", "bfp8_last_error",
           "bfp8_status_string", "bfp8_device_status", "bfp8_selftest_bounded_wait",
           "bfp8_version", "bfp8_gemm_noalloc", "bfp8_gemm_grouped",
           "bfp8_gemm_grouped_workspace_size", "bfp8_gemm_fused", "bfp8_gemm_fused_workspace_size",
           "bfp8_linear", "bfp8_linear_workspace_size", "bfp8_rmsnorm_quant", "bfp8_kv_cache_write",
           "bfp8_kv_cache_read", "bfp8_paged_attention", "bfp8_paged_attention_workspace_size",
           "bfp8_shared_prefix_attention", "bfp8_shared_prefix_attention_workspace_size", "bfp8_kv_cache_weigh",
           "bfp8_kv_cache_weigh_workspace_size", "bfp8_kv_cache_evict", "bfp8_kv_cache_evict_workspace_size",
           "bfp8_stream_capture_id")


class BFP8Error(RuntimeError):
    def __init__(self, status: int, where: str, reason: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {reason}")
        self.status = status


class GemmOptions(ctypes.Structure):
    _fields_ = [("schedule", ctypes.c_int), ("max_ctas", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("prefetch_weights", ctypes.c_int), ("k_split", ctypes.c_int),
                ("cluster_size", ctypes.c_int), ("pairs", ctypes.c_int),
                ("reserved", ctypes.c_int * 1)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("swap_ab", ctypes.c_int), ("tile_n", ctypes.c_int), ("stages", ctypes.c_int),
                ("grid", ctypes.c_int), ("tiles", ctypes.c_int64), ("k_blocks", ctypes.c_int64),
                ("dp_tiles", ctypes.c_int64), ("sk_units", ctypes.c_int64),
                ("relayout", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t),
                ("cluster", ctypes.c_int), ("gemv", ctypes.c_int), ("pair", ctypes.c_int)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("reserved", ctypes.c_int),
                ("stride_page", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("scale_stride_page", ctypes.c_int64),
                ("scale_stride_head", ctypes.c_int64)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("total_q", ctypes.c_int64), ("num_heads", ctypes.c_int), ("batch", ctypes.c_int),
                ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("max_pages", ctypes.c_int), ("max_q_len", ctypes.c_int), ("max_kv_len", ctypes.c_int64),
                ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("softmax_scale", ctypes.c_float),
                ("causal", ctypes.c_int), ("window", ctypes.c_int), ("reserved", ctypes.c_int)]


class PrefixArgs(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("prefixes", ctypes.c_int), ("cu_q", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("max_q_len", ctypes.c_int), ("reserved", ctypes.c_int), ("max_len", ctypes.c_int64)]


class EvictArgs(ctypes.Structure):
    _fields_ = [("weights", ctypes.c_void_p), ("weights_stride_page", ctypes.c_int64),
                ("weights_stride_head", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("out_table", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("max_out_pages", ctypes.c_int), ("kv_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
                ("max_kv_len", ctypes.c_int64), ("budget", ctypes.c_int64), ("recent", ctypes.c_int64),
                ("first", ctypes.c_int64), ("batch", ctypes.c_int), ("reserved", ctypes.c_int)]


# The structures as packed bytes: half the host time of filling a ctypes Structure field by field.
_pack_cache = struct.Struct("@PPPPqiiiiqqqqq")
_pack_attention = struct.Struct("@PPPqiiqqqqPqiiqPPfiii")
_pack_prefix = struct.Struct("@PqiiPPiiq")
_pack_evict = struct.Struct("@PqqPqPqiiPPqqqqii")
assert _pack_cache.size == ctypes.sizeof(KVCacheDesc) and _pack_attention.size == ctypes.sizeof(AttentionArgs)
assert _pack_prefix.size == ctypes.sizeof(PrefixArgs) and _pack_evict.size == ctypes.sizeof(EvictArgs)

_lock = threading.Lock()
_lib = None


def lib():
    """The loaded libbfp8 (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libbfp8 is not built ({LIB_PATH} missing): run "
                    "`python -m block_scaled_fp8_02_gb300.build` or __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.bfp8_group_quant.restype = i32
            L.bfp8_group_quant.argtypes = [P, i32, i64, i64, i64, i32, i32, P, i64, P, i64, P]
            L.bfp8_group_quant_ex.restype = i32
            L.bfp8_group_quant_ex.argtypes = [P, i32, i64, i64, i64, i32, i32, i32, P, i64, P, i64, P]
            L.bfp8_scale_ceil_ue8m0.restype = i32
            L.bfp8_scale_ceil_ue8m0.argtypes = [P, P, i64, P]
            L.bfp8_scale_ld.restype = i64
            L.bfp8_scale_ld.argtypes = [i64]
            L.bfp8_gemm.restype = i32
            L.bfp8_gemm.argtypes = [P, P, P, i32, i64, P, P, i64, i64, i64, P, sz, P]
            L.bfp8_gemm_ex.restype = i32
            L.bfp8_gemm_ex.argtypes = [P, P, P, i32, i64, P, P, i64, i64, i64, P, sz,
                                       ctypes.POINTER(GemmOptions), P]
            L.bfp8_gemm_workspace_size.restype = i32
            L.bfp8_gemm_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(GemmOptions), i32,
                                                   ctypes.POINTER(sz)]
            L.bfp8_gemm_plan.restype = i32
            L.bfp8_gemm_plan.argtypes = [i64, i64, i64, i32, ctypes.POINTER(GemmOptions), i32,
                                         ctypes.POINTER(PlanInfo)]
            L.bfp8_plan_unit.restype = i32
            L.bfp8_plan_unit.argtypes = [i64, i64, i64, i32, ctypes.POINTER(GemmOptions), i32, i64,
                                         ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)]
            L.bfp8_last_error.restype = ctypes.c_char_p
            L.bfp8_last_error.argtypes = []
            L.bfp8_status_string.restype = ctypes.c_char_p
            L.bfp8_status_string.argtypes = [i32]
            L.bfp8_device_status.restype = i32
            L.bfp8_device_status.argtypes = [ctypes.POINTER(i32), i32]
            L.bfp8_selftest_bounded_wait.restype = i32
            L.bfp8_selftest_bounded_wait.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64), P]
            L.bfp8_version.restype = i32
            L.bfp8_version.argtypes = []
            L.bfp8_gemm_noalloc.restype = i32
            L.bfp8_gemm_noalloc.argtypes = [P, P, P, i32, i64, P, P, i64, i64, i64, P]
            L.bfp8_gemm_grouped.restype = i32
            L.bfp8_gemm_grouped.argtypes = [P, P, P, i32, i64, P, P, i32, P, i64, i64, i64, P, sz,
                                            ctypes.POINTER(GemmOptions), P]
            L.bfp8_gemm_fused.restype = i32
            L.bfp8_gemm_fused.argtypes = [P, P, P, i32, i64, P, P, P, P, P, i32, i64, i64, i64, i64,
                                          P, sz, ctypes.POINTER(GemmOptions), P]
            L.bfp8_gemm_fused_workspace_size.restype = i32
            L.bfp8_gemm_fused_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(GemmOptions),
                                                         i32, ctypes.POINTER(sz)]
            L.bfp8_linear.restype = i32
            L.bfp8_linear.argtypes = [P, i64, P, P, P, i64, i64, i64, P, sz,
                                      ctypes.POINTER(GemmOptions), P]
            L.bfp8_linear_workspace_size.restype = i32
            L.bfp8_linear_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(GemmOptions), i32,
                                                     ctypes.POINTER(sz)]
            L.bfp8_gemm_grouped_workspace_size.restype = i32
            L.bfp8_gemm_grouped_workspace_size.argtypes = [i64, i64, i64, i32,
                                                           ctypes.POINTER(GemmOptions), i32,
                                                           ctypes.POINTER(sz)]
            L.bfp8_rmsnorm_quant.restype = i32
            L.bfp8_rmsnorm_quant.argtypes = [P, i32, i64, P, i64, P, i64, P, i32, ctypes.c_float, i64, i64,
                                             P, i64, i32, i32, P, i64, P, i64, P]
            L.bfp8_kv_cache_write.restype = i32
            L.bfp8_kv_cache_write.argtypes = [P, P, i32, i64, i64, i64, i64, P, i64, i32,
                                              P, P]
            L.bfp8_kv_cache_read.restype = i32
            L.bfp8_kv_cache_read.argtypes = [P, P, i64, i32, P, i64, P, i64, P]
            L.bfp8_paged_attention.restype = i32
            L.bfp8_paged_attention.argtypes = [P, P, P, sz, P]
            L.bfp8_paged_attention_workspace_size.restype = i32
            L.bfp8_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
            L.bfp8_shared_prefix_attention.restype = i32
            L.bfp8_shared_prefix_attention.argtypes = [P, P, P, P, sz, P]
            L.bfp8_shared_prefix_attention_workspace_size.restype = i32
            L.bfp8_shared_prefix_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, ctypes.POINTER(sz)]
            L.bfp8_kv_cache_weigh.restype = i32
            L.bfp8_kv_cache_weigh.argtypes = [P, P, P, i64, i64, i32, P, sz, P]
            L.bfp8_kv_cache_weigh_workspace_size.restype = i32
            L.bfp8_kv_cache_weigh_workspace_size.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
            L.bfp8_kv_cache_evict.restype = i32
            L.bfp8_kv_cache_evict.argtypes = [P, P, P, sz, P]
            L.bfp8_kv_cache_evict_workspace_size.restype = i32
            L.bfp8_kv_cache_evict_workspace_size.argtypes = [i32, i32, i64, i64, ctypes.POINTER(sz)]
            L.bfp8_stream_capture_id.restype = i32
            L.bfp8_stream_capture_id.argtypes = [P, ctypes.POINTER(ctypes.c_ulonglong)]
            _lib = L
    return _lib


def bfp8_last_error() -> str:
    return lib().bfp8_last_error().decode()


def _check(status: int, where: str):
    if status != BFP8_OK:
        raise BFP8Error(status, where, bfp8_last_error())


def _stream_ptr(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _opts(options) -> ctypes.POINTER(GemmOptions) | None:
    if options is None:
        return None
    if isinstance(options, GemmOptions):
        return ctypes.pointer(options)
    o = GemmOptions()
    o.schedule = int(options.get("schedule", 0))
    o.max_ctas = int(options.get("max_ctas", 0))
    o.tile_n = int(options.get("tile_n", 0))
    o.prefetch_weights = int(options.get("prefetch_weights", 0))
    o.k_split = int(options.get("k_split", 0))
    o.cluster_size = int(options.get("cluster_size", 0))
    o.pairs = int(options.get("pairs", 0))
    unknown = set(options) - {"schedule", "max_ctas", "tile_n", "prefetch_weights", "k_split",
                              "cluster_size", "pairs"}
    if unknown:
        raise ValueError(f"unknown GEMM options {sorted(unknown)}")
    return ctypes.pointer(o)


def bfp8_version() -> int:
    return int(lib().bfp8_version())


def bfp8_scale_ld(M: int) -> int:
    return int(lib().bfp8_scale_ld(M))


def bfp8_group_quant(x: torch.Tensor, col_major: bool = True, group: int = 128,
                     q: torch.Tensor | None = None, s_storage: torch.Tensor | None = None,
                     stream=None, ue8m0: bool = False):
    """Quantise x [M, K] (bf16 or fp32, CUDA, unit inner stride) per 128-group.

    Returns (q, s): q [M, K] float8_e4m3fn and s [M, G] fp32; for col_major the
    scales live in a [G, bfp8_scale_ld(M)] buffer and s is its transposed view
    (stride (1, ld)), the layout the pages hand to the GEMM.  ue8m0: every
    scale rounded up to a power of two (the UE8M0 variant).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit inner stride")
    if x.dtype == torch.bfloat16:
        in_dtype = BFP8_IN_BF16
    elif x.dtype == torch.float32:
        in_dtype = BFP8_IN_F32
    else:
        raise ValueError(f"x dtype {x.dtype}: expected bfloat16 or float32")
    M, K = x.shape
    G = (K + 127) // 128
    if q is None:
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    if col_major:
        ld_s = bfp8_scale_ld(M) if s_storage is None else s_storage.shape[1]
        if s_storage is None:
            s_storage = torch.empty((G, max(ld_s, 1)), dtype=torch.float32, device=x.device)
        s_view = s_storage[:, :M].t()
    else:
        ld_s = G if s_storage is None else s_storage.shape[1]
        if s_storage is None:
            s_storage = torch.empty((M, max(ld_s, 1)), dtype=torch.float32, device=x.device)
        s_view = s_storage[:, :G]
    st = lib().bfp8_group_quant_ex(x.data_ptr(), in_dtype, M, K, x.stride(0), group, int(col_major),
                                   SCALE_UE8M0 if ue8m0 else SCALE_FP32, q.data_ptr(),
                                   q.stride(0) if M > 0 else K, s_storage.data_ptr(), ld_s,
                                   _stream_ptr(stream))
    _check(st, "bfp8_group_quant")
    return q, s_view


def bfp8_scale_ceil_ue8m0(s: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Every element of the fp32 scale tensor s rounded up to a power of two
    (contiguous tensors; out may be s itself)."""
    if s.dtype != torch.float32 or not s.is_contiguous():
        raise ValueError("s must be a contiguous float32 tensor")
    if out is None:
        out = torch.empty_like(s)
    if out.shape != s.shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 tensor shaped like s")
    _check(lib().bfp8_scale_ceil_ue8m0(s.data_ptr(), out.data_ptr(), s.numel(), _stream_ptr(stream)),
           "bfp8_scale_ceil_ue8m0")
    return out


def _as_layout(As: torch.Tensor, M: int, G: int):
    """(col_major, ld) of an As tensor of shape [M, G]."""
    if As.shape != (M, G):
        raise ValueError(f"As has shape {tuple(As.shape)}, expected ({M}, {G})")
    s0, s1 = As.stride()
    if s0 == 1 and (G == 1 or s1 >= M):
        return 1, (s1 if G > 1 else max(M, 1))
    if s1 == 1 and (M == 1 or s0 >= G):
        return 0, (s0 if M > 1 else G)
    raise ValueError(f"As strides {As.stride()} are neither row- nor column-major")


_ws_cache: dict[tuple[int, int], torch.Tensor] = {}
# (device, stream) -> (capture, buffer allocated in it); buffers of _ws_cache that a graph holds the address of
_ws_graph: dict[tuple[int, int], tuple[int, torch.Tensor]] = {}
_ws_held: dict[int, torch.Tensor] = {}


def _capture_id(stream, sp: int) -> int:
    """The number of the graph capture that the stream is in, 0 outside of any."""
    if stream is None and not torch.cuda.is_current_stream_capturing():
        return 0
    n = ctypes.c_ulonglong(0)
    _check(lib().bfp8_stream_capture_id(sp, ctypes.byref(n)), "bfp8_stream_capture_id")
    return int(n.value)


def workspace_for(nbytes: int, device: torch.device, stream=None) -> torch.Tensor:
    """A zero-initialised workspace of at least nbytes on `device` for calls
    on `stream` (None: the current stream), cached per (device, stream).

    libbfp8 leaves the workspace zeroed after every completed call, so one
    buffer serves every call issued in order on one stream; calls on streams
    without ordering between them get separate buffers.  A new buffer is
    allocated and zeroed on that stream, so its zeroing is ordered before the
    calls that use it, and a replaced buffer is only ever reused by later work
    on the same stream (the caching allocator's stream-ordered reuse).

    A call that is being captured gets the stream's buffer if that is large
    enough, which is then kept for good: the graph holds its address.  Otherwise
    it gets a buffer of this capture's own, zeroed by a node of the graph, which
    no call outside the capture is given (it is zero only when the graph runs)."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    sp = _stream_ptr(stream)
    ws = _ws_cache.get((idx, sp))
    capture = _capture_id(stream, sp)
    if capture:
        if ws is not None and ws.numel() >= nbytes:
            _ws_held[ws.data_ptr()] = ws
            return ws
        born, ws = _ws_graph.get((idx, sp), (0, None))
        if born != capture:
            ws = None
    if ws is None or ws.numel() < nbytes:
        s = stream if isinstance(stream, torch.cuda.Stream) else (
            torch.cuda.current_stream(device) if stream is None else
            torch.cuda.ExternalStream(sp, device=device))
        with torch.cuda.stream(s):
            ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        if capture:
            _ws_graph[(idx, sp)] = (capture, ws)
        else:
            _ws_cache[(idx, sp)] = ws
    return ws


def drop_workspaces() -> None:
    """Forget every cached workspace (after a kernel gave up on a wait, one may
    hold non-zero stream-K counters).  Those that captured graphs use stay and
    are zeroed, with the device idle before and after."""
    _ws_cache.clear()
    for ws in _ws_held.values():
        torch.cuda.synchronize(ws.device)
        ws.zero_()
        torch.cuda.synchronize(ws.device)


def bfp8_gemm_workspace_size(M: int, N: int, K: int, options=None,
                             operands_unaligned: bool = False) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_gemm_workspace_size(M, N, K, _opts(options), int(operands_unaligned),
                                          ctypes.byref(n)), "bfp8_gemm_workspace_size")
    return int(n.value)


def bfp8_gemm_plan(M: int, N: int, K: int, num_sms: int, options=None,
                   operands_unaligned: bool = False) -> dict:
    info = PlanInfo()
    _check(lib().bfp8_gemm_plan(M, N, K, num_sms, _opts(options), int(operands_unaligned),
                                ctypes.byref(info)), "bfp8_gemm_plan")
    return {f: getattr(info, f) for f, _ in PlanInfo._fields_}


def bfp8_plan_unit(M: int, N: int, K: int, num_sms: int, cta: int, j: int = -1, options=None):
    n, t, kb = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
    _check(lib().bfp8_plan_unit(M, N, K, num_sms, _opts(options), cta, j, ctypes.byref(n),
                                ctypes.byref(t), ctypes.byref(kb)), "bfp8_plan_unit")
    return int(n.value), int(t.value), int(kb.value)


def bfp8_gemm(A: torch.Tensor, B: torch.Tensor, As: torch.Tensor, Bs: torch.Tensor,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              options=None, stream=None) -> torch.Tensor:
    """out [M, N] bf16 = blocked-FP8 GEMM of A [M, K], B [N, K] (float8_e4m3fn),
    As [M, G] (row- or column-major strides) and Bs [ceil(N/128), G]."""
    if A.dtype != torch.float8_e4m3fn or B.dtype != torch.float8_e4m3fn:
        raise ValueError("A and B must be float8_e4m3fn")
    if not (A.is_contiguous() and B.is_contiguous() and Bs.is_contiguous()):
        raise ValueError("A, B and Bs must be contiguous")
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError("A and B disagree on K")
    G = (K + 127) // 128
    if Bs.shape != ((N + 127) // 128, G) or Bs.dtype != torch.float32:
        raise ValueError(f"Bs must be float32 of shape {((N + 127) // 128, G)}")
    col, ld = _as_layout(As, M, G)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    unaligned = (A.data_ptr() % 16 != 0) or (B.data_ptr() % 16 != 0)
    if workspace is None:
        need = bfp8_gemm_workspace_size(M, N, K, options, unaligned)
        workspace = workspace_for(need, A.device, stream)
    st = lib().bfp8_gemm_ex(A.data_ptr(), B.data_ptr(), As.data_ptr(), col, ld, Bs.data_ptr(),
                            out.data_ptr(), M, N, K, workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _opts(options),
                            _stream_ptr(stream))
    _check(st, "bfp8_gemm")
    return out


def bfp8_gemm_grouped_workspace_size(M: int, N: int, K: int, num_experts: int, options=None,
                                     operands_unaligned: bool = False) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_gemm_grouped_workspace_size(M, N, K, num_experts, _opts(options),
                                                  int(operands_unaligned), ctypes.byref(n)),
           "bfp8_gemm_grouped_workspace_size")
    return int(n.value)


def bfp8_gemm_grouped(A: torch.Tensor, B: torch.Tensor, As: torch.Tensor, Bs: torch.Tensor,
                      grouped_layout: torch.Tensor, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, options=None,
                      stream=None) -> torch.Tensor:
    """M-grouped (mixture-of-experts) blocked-FP8 GEMM: A [M, K] rows grouped by
    expert in 128-aligned blocks, B [E, N, K], Bs [E, ceil(N/128), G],
    grouped_layout int32 [E] = cumulative aligned row counts (device).  Rows
    past the last expert's block are left untouched in `out`."""
    if A.dtype != torch.float8_e4m3fn or B.dtype != torch.float8_e4m3fn:
        raise ValueError("A and B must be float8_e4m3fn")
    if B.dim() != 3:
        raise ValueError("B must be [experts, N, K]")
    if not (A.is_contiguous() and B.is_contiguous() and Bs.is_contiguous()
            and grouped_layout.is_contiguous()):
        raise ValueError("A, B, Bs and grouped_layout must be contiguous")
    M, K = A.shape
    E, N, K2 = B.shape
    if K2 != K:
        raise ValueError("A and B disagree on K")
    G = (K + 127) // 128
    if Bs.shape != (E, (N + 127) // 128, G) or Bs.dtype != torch.float32:
        raise ValueError(f"Bs must be float32 of shape {(E, (N + 127) // 128, G)}")
    if grouped_layout.dtype != torch.int32 or grouped_layout.shape != (E,):
        raise ValueError(f"grouped_layout must be int32 of shape ({E},)")
    col, ld = _as_layout(As, M, G)
    if out is None:
        out = torch.zeros((M, N), dtype=torch.bfloat16, device=A.device)
    unaligned = (A.data_ptr() % 16 != 0) or (B.data_ptr() % 16 != 0)
    if workspace is None:
        need = bfp8_gemm_grouped_workspace_size(M, N, K, E, options, unaligned)
        workspace = workspace_for(need, A.device, stream)
    st = lib().bfp8_gemm_grouped(A.data_ptr(), B.data_ptr(), As.data_ptr(), col, ld,
                                 Bs.data_ptr(), grouped_layout.data_ptr(), E, out.data_ptr(),
                                 M, N, K, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _opts(options),
                                 _stream_ptr(stream))
    _check(st, "bfp8_gemm_grouped")
    return out


def bfp8_gemm_fused(A: torch.Tensor, B: torch.Tensor, As: torch.Tensor, Bs: torch.Tensor,
                    bias: torch.Tensor | None = None, want_out: bool = True,
                    quantise: bool = True, s_col_major: bool = True,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    options=None, stream=None):
    """Blocked-FP8 GEMM with the fused epilogue: y = bf16(bf16(A B^T scaled) +
    bias), returned as (out or None, q or None, s or None); q, s = the 1x128
    group quantisation of y (s a [M, G] view, column-major storage by default)."""
    if A.dtype != torch.float8_e4m3fn or B.dtype != torch.float8_e4m3fn:
        raise ValueError("A and B must be float8_e4m3fn")
    if not (A.is_contiguous() and B.is_contiguous() and Bs.is_contiguous()):
        raise ValueError("A, B and Bs must be contiguous")
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError("A and B disagree on K")
    G = (K + 127) // 128
    if Bs.shape != ((N + 127) // 128, G) or Bs.dtype != torch.float32:
        raise ValueError(f"Bs must be float32 of shape {((N + 127) // 128, G)}")
    if bias is not None and (bias.dtype != torch.bfloat16 or bias.shape != (N,)
                             or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous bfloat16 tensor of shape ({N},)")
    col, ld = _as_layout(As, M, G)
    if want_out and out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    if not want_out:
        out = None
    q = s_view = s_st = None
    Gn = (N + 127) // 128
    ld_s = 0
    if quantise:
        q = torch.empty((M, N), dtype=torch.float8_e4m3fn, device=A.device)
        if s_col_major:
            ld_s = bfp8_scale_ld(M)
            s_st = torch.zeros((Gn, ld_s), dtype=torch.float32, device=A.device)
            s_view = s_st[:, :M].t()
        else:
            ld_s = Gn
            s_st = torch.zeros((M, Gn), dtype=torch.float32, device=A.device)
            s_view = s_st
    unaligned = (A.data_ptr() % 16 != 0) or (B.data_ptr() % 16 != 0)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(lib().bfp8_gemm_fused_workspace_size(M, N, K, _opts(options), int(unaligned),
                                                    ctypes.byref(n)),
               "bfp8_gemm_fused_workspace_size")
        workspace = workspace_for(int(n.value), A.device, stream)
    st = lib().bfp8_gemm_fused(
        A.data_ptr(), B.data_ptr(), As.data_ptr(), col, ld, Bs.data_ptr(),
        bias.data_ptr() if bias is not None else None, out.data_ptr() if out is not None else None,
        q.data_ptr() if q is not None else None, s_st.data_ptr() if s_st is not None else None,
        int(s_col_major), ld_s, M, N, K, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _opts(options), _stream_ptr(stream))
    _check(st, "bfp8_gemm_fused")
    return out, q, s_view


def bfp8_device_status(clear: bool = True) -> int:
    """The device failure word (0: no kernel gave up on a wait).  A nonzero
    word also drops the cached workspaces, which may hold stale counters."""
    code = ctypes.c_int(0)
    _check(lib().bfp8_device_status(ctypes.byref(code), int(clear)), "bfp8_device_status")
    if code.value != 0:
        drop_workspaces()
    return int(code.value)


def bfp8_selftest_bounded_wait(limit_cycles: int, stream=None):
    """Returns (status, elapsed_cycles); status BFP8_ERR_DEVICE_TIMEOUT (6) is
    the expected outcome: the wait gave up instead of hanging."""
    el = ctypes.c_uint64(0)
    st = lib().bfp8_selftest_bounded_wait(limit_cycles, ctypes.byref(el), _stream_ptr(stream))
    return int(st), int(el.value)


def bfp8_linear_workspace_size(M: int, N: int, K: int, options=None,
                               weights_unaligned: bool = False) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_linear_workspace_size(M, N, K, _opts(options), int(weights_unaligned),
                                            ctypes.byref(n)), "bfp8_linear_workspace_size")
    return int(n.value)


def bfp8_linear(x: torch.Tensor, B: torch.Tensor, Bs: torch.Tensor, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, options=None, stream=None) -> torch.Tensor:
    """out [M, N] bf16 = the blocked linear layer of bf16 x [M, K] (rows may be
    strided) against e4m3 weights B [N, K] with scales Bs: the 1 x 128 group
    quantisation into the workspace, then the GEMM, in one library call."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 tensor with unit column stride")
    if B.dtype != torch.float8_e4m3fn or not B.is_contiguous() or not Bs.is_contiguous():
        raise ValueError("B must be contiguous float8_e4m3fn and Bs contiguous")
    M, K = x.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError("x and B disagree on K")
    G = (K + 127) // 128
    if Bs.shape != ((N + 127) // 128, G) or Bs.dtype != torch.float32:
        raise ValueError(f"Bs must be float32 of shape {((N + 127) // 128, G)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        need = bfp8_linear_workspace_size(M, N, K, options, B.data_ptr() % 16 != 0)
        workspace = workspace_for(need, x.device, stream)
    st = lib().bfp8_linear(x.data_ptr(), x.stride(0), B.data_ptr(), Bs.data_ptr(), out.data_ptr(),
                           M, N, K, workspace.data_ptr(),
                           workspace.numel() * workspace.element_size(), _opts(options),
                           _stream_ptr(stream))
    _check(st, "bfp8_linear")
    return out


def linear(x: torch.Tensor, B: torch.Tensor, Bs: torch.Tensor, out: torch.Tensor | None = None,
           stream=None, ue8m0: bool = False) -> torch.Tensor:
    """The whole W8A8 blocked linear layer: quantise x per 128-group (column-major
    scales) and run the blocked GEMM against e4m3 weights B with scales Bs
    (bfp8_linear).  ue8m0: the UE8M0 variant (activation scales rounded up to
    powers of two; pass weight scales rounded the same way, e.g. by
    bfp8_scale_ceil_ue8m0) and fp32 activations run as two calls."""
    if not ue8m0 and x.dtype == torch.bfloat16:
        return bfp8_linear(x, B, Bs, out=out, stream=stream)
    q, s = bfp8_group_quant(x, col_major=True, stream=stream, ue8m0=ue8m0)
    # the quantisation kernel writes neither B nor Bs: the GEMM may start
    # streaming the weights while it runs
    return bfp8_gemm(q, B, s, Bs, out=out, options={"prefetch_weights": 1}, stream=stream)


_IN_DTYPE = {torch.bfloat16: BFP8_IN_BF16, torch.float32: BFP8_IN_F32}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(stream) -> int:
    """_stream_ptr without building a Stream object for the current one (3 us of a small call's 10)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(_current_device())
    return _stream_ptr(stream)


def _on(dev: torch.device, *tensors) -> None:
    """All on one device: an address of another one (a length left on the host, say) would fault in the kernel."""
    index = dev.index                          # (a comparison of numbers: half the time of one of devices)
    for t in tensors:
        if t is not None and t.get_device() != index and t.device != dev:
            raise ValueError(f"a tensor is on {t.device}, the others on {dev}")


def _rows(t: torch.Tensor, name: str, shape, dtype) -> int:
    """Row stride of a tensor of the given 2-D shape with unit inner stride."""
    st = t.stride()
    if t.shape != shape or t.dtype != dtype or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} with unit inner stride")
    return st[0] if shape[0] > 1 else shape[1]


def _col_major_scales(M: int, G: int, ld: int, dev) -> torch.Tensor:
    """[M, G] fp32 with strides (1, ld), whose columns the GEMM copies in 16-byte lines.  ld - M < 4 and the columns begin on
    lines, so the last one's line holds at least one of the tensor's floats, and CUDA memory is never handed out in
    parts of a line.  (A slice of a buffer with the ld - M floats too costs 4 us of a small call's 15.)"""
    return torch.empty_strided((M, G), (1, ld), dtype=torch.float32, device=dev)


def bfp8_rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor | None, residual: torch.Tensor | None = None,
                       residual_out: torch.Tensor | None = None, eps: float = 1e-6,
                       col_major: bool = True, ue8m0: bool = False, want_y: bool = False,
                       quantise: bool = True, stream=None):
    """Residual addition, RMS norm and 1 x 128 group quantisation of x [M, K] (bf16 or fp32) in one pass.

    h = x + residual goes to residual_out (default: residual itself, in place); y = h * rsqrt(mean(h^2) +
    eps) * weight.  Returns (q, s), the codes and scales of y as bfp8_group_quant returns them; with
    want_y, (q, s, y) with y in bf16; without quantise q and s are None."""
    if x.dim() != 2 or x.dtype not in _IN_DTYPE:
        raise ValueError("x must be a 2-D bfloat16 or float32 tensor")
    shape, dtype, dev = x.shape, x.dtype, x.device
    M, K = shape
    ld_x = _rows(x, "x", shape, dtype)
    r_ptr = ro_ptr = w_ptr = y_ptr = q_ptr = s_ptr = None
    ld_r = ld_ro = ld_q = ld_s = K
    if residual is not None:
        ld_r = _rows(residual, "residual", shape, dtype)
        r_ptr = residual.data_ptr()
        if residual_out is None:
            residual_out = residual
    if residual_out is not None:
        ld_ro = ld_r if residual_out is residual else _rows(residual_out, "residual_out", shape, dtype)
        ro_ptr = residual_out.data_ptr()
    w_dtype = BFP8_IN_BF16
    if weight is not None:
        if weight.dtype not in _IN_DTYPE or weight.shape != (K,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous bfloat16 or float32 tensor of shape ({K},)")
        w_dtype, w_ptr = _IN_DTYPE[weight.dtype], weight.data_ptr()
    _on(dev, residual, residual_out if residual_out is not residual else None, weight)
    q = s = y = None
    if quantise:
        G = (K + 127) // 128
        q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        if col_major:                          # [M, G] over a [G, ld_s] buffer, as bfp8_group_quant returns it
            ld_s = (M + 3) // 4 * 4
            s = _col_major_scales(M, G, ld_s, dev)
        else:
            ld_s = G
            s = torch.empty((M, G), dtype=torch.float32, device=dev)
        q_ptr, s_ptr = q.data_ptr(), s.data_ptr()
    if want_y:
        y = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        y_ptr = y.data_ptr()
    rc = (_lib or lib()).bfp8_rmsnorm_quant(x.data_ptr(), _IN_DTYPE[dtype], ld_x, r_ptr, ld_r, ro_ptr, ld_ro, w_ptr,
                                            w_dtype, eps, M, K, y_ptr, K, int(col_major),
                                            SCALE_UE8M0 if ue8m0 else SCALE_FP32, q_ptr, ld_q, s_ptr, ld_s,
                                            _stream_of(stream))
    _check(rc, "bfp8_rmsnorm_quant")
    return (q, s, y) if want_y else (q, s)


class KVCache:
    """A paged e4m3 cache: codes k, v [pages, kv_heads, page_size, head_dim] (float8_e4m3fn, any strides with
    unit inner stride) and fp32 scales k_scale, v_scale [pages, kv_heads, page_size] (unit inner stride).
    The tensors stay the caller's; slot = page * page_size + offset."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "_desc")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        shape, st, ss = k.shape, k.stride(), k_scale.stride()
        if len(shape) != 4 or v.shape != shape or k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
            raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim], the scales [pages, kv_heads, page_size]")
        if k.dtype != torch.float8_e4m3fn or v.dtype != torch.float8_e4m3fn:
            raise ValueError("k and v must be float8_e4m3fn")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise ValueError("k_scale and v_scale must be float32")
        if st[3] != 1 or ss[2] != 1 or v.stride() != st or v_scale.stride() != ss:
            raise ValueError("k and v (and the two scale tensors) must have the same strides, the inner one 1")
        _on(k.device, v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        P, H, page, D = shape
        self._desc = _pack_cache.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), P, page, H, D, 0,
                                 st[0], st[1] if H > 1 else max(st[1], page * D), st[2], ss[0],
                                 ss[1] if H > 1 else max(ss[1], page))

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int, head_dim: int, device) -> "KVCache":
        """A zero-filled cache of its own."""
        def codes():
            return torch.zeros((pages, kv_heads, page_size, head_dim), dtype=torch.uint8,
                               device=device).view(torch.float8_e4m3fn)

        def scales():
            return torch.zeros((pages, kv_heads, page_size), dtype=torch.float32, device=device)
        return cls(codes(), codes(), scales(), scales())

    @property
    def shape(self):
        return self.k.shape


def _check_slots(slots: torch.Tensor, T: int | None = None) -> int:
    if slots.dtype != torch.int64 or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous 1-D int64 tensor")
    if T is not None and slots.shape[0] != T:
        raise ValueError(f"slots has {slots.shape[0]} entries for {T} tokens")
    return slots.shape[0]


def bfp8_kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slots: torch.Tensor,
                        ue8m0: bool = False, stream=None) -> None:
    """Quantise new keys and values k, v [T, kv_heads, head_dim] (bf16 or fp32; token and head strides free)
    into the cache at slots [T] (int64; negative: skipped), one fp32 scale per (token, head)."""
    _, H, _, D = cache.k.shape
    if k.dim() != 3 or k.shape[1:] != (H, D) or v.shape != k.shape:
        raise ValueError(f"k and v must be [T, {H}, {D}]")
    if k.dtype not in _IN_DTYPE or v.dtype != k.dtype:
        raise ValueError("k and v must both be bfloat16 or float32")
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("k and v must have unit inner stride")
    T = _check_slots(slots, k.shape[0])
    _on(k.device, v, slots, cache.k)
    _check((_lib or lib()).bfp8_kv_cache_write(k.data_ptr(), v.data_ptr(), _IN_DTYPE[k.dtype], k.stride(0), k.stride(1),
                                     v.stride(0), v.stride(1), slots.data_ptr(), T,
                                     SCALE_UE8M0 if ue8m0 else SCALE_FP32, cache._desc,
                                     _stream_of(stream)), "bfp8_kv_cache_write")


def bfp8_kv_cache_read(cache: KVCache, slots: torch.Tensor, dtype=torch.bfloat16, stream=None):
    """The keys and values of slots [T] (int64; negative: zeros) as (k, v) [T, kv_heads, head_dim] in bf16 or fp32."""
    if dtype not in _IN_DTYPE:
        raise ValueError("dtype must be bfloat16 or float32")
    T = _check_slots(slots)
    _on(slots.device, cache.k)
    _, H, _, D = cache.k.shape
    k = torch.empty((T, H, D), dtype=dtype, device=slots.device)
    v = torch.empty((T, H, D), dtype=dtype, device=slots.device)
    _check((_lib or lib()).bfp8_kv_cache_read(cache._desc, slots.data_ptr(), T, _IN_DTYPE[dtype], k.data_ptr(),
                                    H * D, v.data_ptr(), H * D, _stream_of(stream)), "bfp8_kv_cache_read")
    return k, v


def bfp8_paged_attention_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_paged_attention_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len, ctypes.byref(n)),
           "bfp8_paged_attention_workspace_size")
    return int(n.value)


# From one token more than the kernel for few rows takes of any group (32 rows) the size is the same for all lengths:
# asked for as one, or the cache below would grow by an entry for every prompt's length.
_LONG_Q = 33


@functools.lru_cache(maxsize=None)
def _attention_workspace(device, num_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int) -> int:
    return bfp8_paged_attention_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len)


def _check_query(q: torch.Tensor, cache: KVCache) -> None:
    D = cache.k.shape[3]
    qs = q.shape
    if len(qs) != 3 or qs[2] != D or q.dtype != torch.bfloat16 or q.stride(2) != 1:
        raise ValueError(f"q must be bfloat16 [total_q, heads, {D}] with unit inner stride")


def _check_context(table: torch.Tensor, cu_q: torch.Tensor, lens: torch.Tensor, names=("block_table", "cu_q", "kv_lens")):
    """Checks the tables and lengths of sequences (or prefixes); how many there are, the table's row stride and width."""
    ts, tst, ls = table.shape, table.stride(), lens.shape
    B = ls[0] if len(ls) == 1 else -1
    if B < 0 or cu_q.shape != (B + 1,) or not lens.is_contiguous() or not cu_q.is_contiguous():
        raise ValueError(f"{names[2]} must be a contiguous [batch] tensor and {names[1]} a contiguous [batch + 1] one")
    if len(ts) != 2 or ts[0] != B or (B > 0 and ts[1] > 1 and tst[1] != 1):
        raise ValueError(f"{names[0]} must be [{B}, max_pages] with unit inner stride")
    if table.dtype != torch.int32 or cu_q.dtype != torch.int32 or lens.dtype != torch.int32:
        raise ValueError(f"{', '.join(names[:2])} and {names[2]} must be int32")
    return B, tst[0] if B > 1 else ts[1], ts[1]


def _workspace(need: int, dev, stream, sp: int) -> torch.Tensor:
    """workspace_for without its lookups where the stream's buffer will do."""
    ws = _ws_cache.get((dev.index, sp))
    if ws is None or ws.numel() < need or _capture_id(stream, sp):
        ws = workspace_for(need, dev, stream)
    return ws


def _axis(T: int, n: int, D: int, st) -> tuple[int, int]:
    """Token and head strides; the stride of an axis of one means nothing: any will do."""
    return D if T == 1 else st[0], D if n == 1 else st[1]


def bfp8_paged_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, cu_q: torch.Tensor,
                         kv_lens: torch.Tensor, max_q_len: int, max_kv_len: int, scale: float | None = None,
                         causal: bool = True, window: int = 0, return_lse: bool = False,
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of the newest tokens q [total_q, heads, head_dim] (bf16) of each sequence over its context in the
    paged cache: sequence b's rows are cu_q[b] .. cu_q[b+1] (int32 [batch + 1]), its context kv_lens[b] tokens
    (int32 [batch], the new ones included) on the pages block_table[b] (int32 [batch, max_pages]).  max_q_len and
    max_kv_len bound the lengths; scale defaults to head_dim ** -0.5.  Returns out (bf16, like q), or (out, lse)
    with lse fp32 [total_q, heads]."""
    _check_query(q, cache)
    _, H, _, D = cache.k.shape
    qs, dev = q.shape, q.device
    T, Hq, _ = qs
    B, ld_table, width = _check_context(block_table, cu_q, kv_lens)
    if out is None:
        out = torch.empty(qs, dtype=torch.bfloat16, device=dev)
    elif out.shape != qs or out.dtype != torch.bfloat16 or out.stride(2) != 1:
        raise ValueError("out must be bfloat16, shaped like q, with unit inner stride")
    _on(dev, cache.k, block_table, cu_q, kv_lens, out, workspace)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if return_lse else None
    sp = _stream_of(stream)
    if workspace is None:
        workspace = _workspace(_attention_workspace(dev, Hq, H, D, min(max_q_len, _LONG_Q)) if T and B else 0, dev, stream, sp)
    (qt, qh), (ot, oh) = _axis(T, Hq, D, q.stride()), _axis(T, Hq, D, out.stride())
    a = _pack_attention.pack(q.data_ptr(), out.data_ptr(), lse.data_ptr() if return_lse else 0, T, Hq, B, qt, qh,
                      ot, oh, block_table.data_ptr(), ld_table, width, max_q_len,
                      max_kv_len, cu_q.data_ptr(), kv_lens.data_ptr(), D ** -0.5 if scale is None else scale,
                      causal, window, 0)
    _check((_lib or lib()).bfp8_paged_attention(a, cache._desc, workspace.data_ptr(),
                                                workspace.numel() * workspace.element_size(), sp),
           "bfp8_paged_attention")
    return (out, lse) if return_lse else out


def bfp8_shared_prefix_attention_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int, max_prefix_q_len: int,
                                                max_q_len: int, total_q: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_shared_prefix_attention_workspace_size(num_heads, num_kv_heads, head_dim, max_prefix_q_len, max_q_len,
                                                             total_q, ctypes.byref(n)),
           "bfp8_shared_prefix_attention_workspace_size")
    return int(n.value)


@functools.lru_cache(maxsize=None)
def _shared_workspace(device, num_heads: int, num_kv_heads: int, head_dim: int, max_prefix_q_len: int, max_q_len: int) -> tuple[int, int]:
    """The bytes of a call without rows, and those that each row of q adds."""
    none, one = (bfp8_shared_prefix_attention_workspace_size(num_heads, num_kv_heads, head_dim, max_prefix_q_len, max_q_len, n)
                 for n in (0, 1))
    return none, one - none


def bfp8_shared_prefix_attention(q: torch.Tensor, cache: KVCache, prefix_table: torch.Tensor, prefix_cu_q: torch.Tensor,
                                 prefix_lens: torch.Tensor, max_prefix_q_len: int, max_prefix_len: int,
                                 block_table: torch.Tensor, cu_q: torch.Tensor, kv_lens: torch.Tensor, max_q_len: int,
                                 max_kv_len: int, scale: float | None = None, causal: bool = True,
                                 return_lse: bool = False, out: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None, stream=None):
    """bfp8_paged_attention for sequences that begin with the same text, whose tokens are read once for all of
    them: prefix f's prefix_lens[f] tokens (int32 [prefixes]), on the pages prefix_table[f] (int32 [prefixes, max_pages]),
    are seen by the rows prefix_cu_q[f] .. prefix_cu_q[f+1] of q (int32 [prefixes + 1]; max_prefix_q_len bounds how many
    they are, max_prefix_len the lengths).  block_table, cu_q, kv_lens and their bounds are those of the sequences' own
    tokens behind the prefix.  Returns out or (out, lse), of one softmax over both parts.  (The workspace holds the
    prefixes' part in fp32, and in some calls the own one: 4 or 8 (head_dim + 1) bytes a row and head, 1.1 GB for 32768
    rows of 64 heads of 128.  A stream's own workspace keeps the largest call's size until drop_workspaces.)"""
    _check_query(q, cache)
    _, H, _, D = cache.k.shape
    qs, dev = q.shape, q.device
    T, Hq, _ = qs
    B, ld_table, width = _check_context(block_table, cu_q, kv_lens)
    F, ld_prefix, prefix_width = _check_context(prefix_table, prefix_cu_q, prefix_lens,
                                                ("prefix_table", "prefix_cu_q", "prefix_lens"))
    if out is None:
        out = torch.empty(qs, dtype=torch.bfloat16, device=dev)
    elif out.shape != qs or out.dtype != torch.bfloat16 or out.stride(2) != 1:
        raise ValueError("out must be bfloat16, shaped like q, with unit inner stride")
    _on(dev, cache.k, prefix_table, prefix_cu_q, prefix_lens, block_table, cu_q, kv_lens, out, workspace)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if return_lse else None
    sp = _stream_of(stream)
    if workspace is None:
        need = 0
        if T and B:
            mq = min(max_q_len, _LONG_Q)
            need, per_row = _shared_workspace(dev, Hq, H, D, min(max_prefix_q_len, _LONG_Q) if F else mq, mq)
            need += per_row * T if F else 0
        workspace = _workspace(need, dev, stream, sp)
    (qt, qh), (ot, oh) = _axis(T, Hq, D, q.stride()), _axis(T, Hq, D, out.stride())
    a = _pack_attention.pack(q.data_ptr(), out.data_ptr(), lse.data_ptr() if return_lse else 0, T, Hq, B, qt, qh,
                             ot, oh, block_table.data_ptr(), ld_table, width, max_q_len, max_kv_len, cu_q.data_ptr(),
                             kv_lens.data_ptr(), D ** -0.5 if scale is None else scale, causal, 0, 0)
    f = _pack_prefix.pack(prefix_table.data_ptr(), ld_prefix, prefix_width, F, prefix_cu_q.data_ptr(),
                          prefix_lens.data_ptr(), max_prefix_q_len, 0, max_prefix_len)
    _check((_lib or lib()).bfp8_shared_prefix_attention(a, f, cache._desc, workspace.data_ptr(),
                                                        workspace.numel() * workspace.element_size(), sp),
           "bfp8_shared_prefix_attention")
    return (out, lse) if return_lse else out


def _weight_strides(weights: torch.Tensor, cache: KVCache) -> tuple[int, int]:
    """Page and head strides of the sums of a cache's tokens."""
    P, H, page, _ = cache.k.shape
    if weights.shape != (P, H, page) or weights.dtype != torch.float32 or weights.stride(2) != 1:
        raise ValueError(f"weights must be float32 [{P}, {H}, {page}] with unit inner stride")
    sp, sh, _ = weights.stride()
    return sp if P > 1 else max(sp, H * page), sh if H > 1 else max(sh, page)


def bfp8_kv_cache_weigh_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_kv_cache_weigh_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len, ctypes.byref(n)),
           "bfp8_kv_cache_weigh_workspace_size")
    return int(n.value)


@functools.lru_cache(maxsize=None)
def _weigh_workspace(device, num_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int) -> int:
    return bfp8_kv_cache_weigh_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len)


def bfp8_kv_cache_weigh(q: torch.Tensor, lse: torch.Tensor, cache: KVCache, weights: torch.Tensor,
                        block_table: torch.Tensor, cu_q: torch.Tensor, kv_lens: torch.Tensor, max_q_len: int,
                        max_kv_len: int, scale: float | None = None, causal: bool = True, window: int = 0,
                        accumulate: bool = True, workspace: torch.Tensor | None = None, stream=None) -> None:
    """Adds to weights [pages, kv_heads, page_size] (fp32) the attention weight that each cached token receives from
    the new tokens q, summed over them and over the query heads of a kv head.  lse [total_q, heads] (fp32) is what
    bfp8_paged_attention or bfp8_shared_prefix_attention returned for the same q; the other arguments are as
    there.  With accumulate the sums of the new tokens begin here (causal) and those of the earlier ones go on; without
    it all sums of the context begin here.  Unlike in attention, no page may stand in two sequences' tables of one
    call (their sums would overwrite each other's): what sequences share is weighed once, as a prefix."""
    _check_query(q, cache)
    _, H, _, D = cache.k.shape
    T, Hq, _ = q.shape
    dev = q.device
    B, ld_table, width = _check_context(block_table, cu_q, kv_lens)
    if lse.shape != (T, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape ({T}, {Hq})")
    wp, wh = _weight_strides(weights, cache)
    _on(dev, lse, cache.k, weights, block_table, cu_q, kv_lens, workspace)
    sp = _stream_of(stream)
    if workspace is None:
        workspace = _workspace(_weigh_workspace(dev, Hq, H, D, min(max_q_len, _LONG_Q)) if T and B else 0, dev, stream, sp)
    qt, qh = _axis(T, Hq, D, q.stride())
    a = _pack_attention.pack(q.data_ptr(), 0, lse.data_ptr(), T, Hq, B, qt, qh, 0, 0, block_table.data_ptr(), ld_table,
                             width, max_q_len, max_kv_len, cu_q.data_ptr(), kv_lens.data_ptr(),
                             D ** -0.5 if scale is None else scale, causal, window, 0)
    _check((_lib or lib()).bfp8_kv_cache_weigh(a, cache._desc, weights.data_ptr(), wp, wh, int(accumulate),
                                               workspace.data_ptr(), workspace.numel() * workspace.element_size(), sp),
           "bfp8_kv_cache_weigh")


def bfp8_kv_cache_evict_workspace_size(batch: int, num_kv_heads: int, max_kv_len: int, budget: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().bfp8_kv_cache_evict_workspace_size(batch, num_kv_heads, max_kv_len, budget, ctypes.byref(n)),
           "bfp8_kv_cache_evict_workspace_size")
    return int(n.value)


# It goes by the budget alone where anything can be evicted, and is the same for all lengths where nothing can.
@functools.lru_cache(maxsize=256)
def _evict_workspace(batch: int, num_kv_heads: int, budget: int) -> int:
    return bfp8_kv_cache_evict_workspace_size(batch, num_kv_heads, budget + 1 if budget else 0, budget or 1)


def bfp8_kv_cache_evict(cache: KVCache, weights: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
                        max_kv_len: int, budget: int, recent: int = 0, first: int = 0,
                        out_table: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Shortens sequences to budget tokens: every kv head keeps its first `first`, its last `recent` and of the others
    the heaviest by weights [pages, kv_heads, page_size] (fp32, as bfp8_kv_cache_weigh sums them), in their order.
    They move with codes, scales and weights to the pages out_table (int32 [batch, max_pages], none of them among
    those of block_table; shorter sequences are copied whole), or, without one, to the first pages of block_table
    (so too where out_table is block_table or a view of its first columns; a copy of them is not, and not allowed).
    No page may stand in two sequences' tables of one call.
    Returns the new lengths min(kv_lens, budget) (int32 [batch], into new_lens if given; not kv_lens itself)."""
    _, H, page, _ = cache.k.shape
    wp, wh = _weight_strides(weights, cache)
    ls = kv_lens.shape
    if len(ls) != 1 or kv_lens.dtype != torch.int32 or not kv_lens.is_contiguous():
        raise ValueError("kv_lens must be a contiguous [batch] int32 tensor")
    B, dev = ls[0], kv_lens.device

    def table(t, name):
        ts, st = t.shape, t.stride()
        if len(ts) != 2 or ts[0] != B or t.dtype != torch.int32 or (B > 0 and ts[1] > 1 and st[1] != 1):
            raise ValueError(f"{name} must be int32 [{B}, max_pages] with unit inner stride")
        return t.data_ptr(), st[0] if B > 1 else ts[1], ts[1]

    tp, ld, width = table(block_table, "block_table")
    op, ld_out, out_width = (0, 0, 0) if out_table is None else table(out_table, "out_table")
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    elif new_lens.shape != (B,) or new_lens.dtype != torch.int32 or not new_lens.is_contiguous():
        raise ValueError(f"new_lens must be a contiguous [{B}] int32 tensor")
    _on(dev, cache.k, weights, block_table, out_table, new_lens, workspace)
    sp = _stream_of(stream)
    if workspace is None:
        workspace = _workspace(_evict_workspace(B, H, budget if max_kv_len > budget else 0) if B else 0, dev, stream, sp)
    a = _pack_evict.pack(weights.data_ptr(), wp, wh, tp, ld, op, ld_out, width, out_width, kv_lens.data_ptr(),
                         new_lens.data_ptr(), max_kv_len, budget, recent, first, B, 0)
    _check((_lib or lib()).bfp8_kv_cache_evict(a, cache._desc, workspace.data_ptr(),
                                               workspace.numel() * workspace.element_size(), sp), "bfp8_kv_cache_evict")
    return new_lens
