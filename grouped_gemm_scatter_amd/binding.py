"""ctypes binding of libep_combine.so (the C ABI in include/ep_combine.h).

Argument marshalling only: every step of the EP-combine path runs in the HIP
kernels of the library.  Functions keep the C names; device arguments are
torch tensors on the current HIP device (PyTorch supplies device memory and
streams), passed as raw pointers.  The library must have been built
(``python -m grouped_gemm_scatter_amd.build``); loading fails loudly otherwise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_combine.so")

EP_OK = 0
EP_ERR_INVALID_ARG = -1
EP_ERR_UNSUPPORTED = -2
EP_ERR_HIP = -3
EP_ERR_SLOT_OOB = 0x1
EP_ERR_FLAG_TIMEOUT = 0x2
EP_ERR_BAD_GROUP = 0x4
EP_DTYPE_BF16 = 0
EP_DTYPE_FP8_E4M3_B128 = 1
EP_FLAG_SYSTEM_SCOPE = 0x1
EP_FLAG_PER_EXPERT_RELEASE = 0x2
EP_FLAG_EPILOGUE_ONLY = 0x4
EP_FLAG_TRACE = 0x8
EP_FLAG_W_SLICE_MAJOR = 0x10
EP_FLAG_DEVICE_EPOCH = 0x20
EP_FLAG_SEND_TILE = 0x40
EP_MAX_RANKS = 8
EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_GROUP_MAX = 0
EP_GROUP_TOP2 = 1
EP_LOGITS_F32 = 0
EP_LOGITS_BF16 = 1
EP_LOGITS_F16 = 2
EP_MAX_ROUTED_EXPERTS = 1024
EP_MAX_ROUTE_GROUPS = 64
EP_W4_INT4 = 0
EP_W4_E2M1 = 1
EP_W4_SCALE_BF16 = 0
EP_W4_SCALE_F16 = 1

EXPORTED = ("ep_combine_init", "ep_combine_destroy", "ep_gemm_tile", "ep_group_local_picks",
            "ep_dispatch_rows", "ep_pack_weights", "ep_advance_epoch",
            "ep_grouped_gemm_scatter", "ep_grouped_gemm_scatter_noalloc", "ep_grouped_gemm_swiglu",
            "ep_grouped_gemm_swiglu_fp8", "ep_grouped_gemm_swiglu_w4", "ep_grouped_gemm_scatter_w4",
            "ep_pack_weights_w4", "ep_route_topk", "ep_route_topk_backward", "ep_combine_backward",
            "ep_grouped_gemm_scatter_combine", "ep_signal_completion",
            "ep_combine_reduce", "ep_combine_query_error", "ep_combine_strerror",
            "ep_combine_version")


class EpCombineParams(ctypes.Structure):
    _fields_ = [
        ("n_ranks", ctypes.c_int32),
        ("p2p_world_size", ctypes.c_int32),
        ("my_rank", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("msg_bytes", ctypes.c_int32),
        ("max_tokens_per_rank", ctypes.c_int32),
        ("n_experts_per_device", ctypes.c_int32),
        ("hidden_k", ctypes.c_int32),
        ("hidden_n", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("send_waves", ctypes.c_int32),
        ("flag_spin_limit", ctypes.c_int64),
    ]


class EpCombineBuffers(ctypes.Structure):
    _fields_ = [
        ("recv_buf", ctypes.c_void_p * EP_MAX_RANKS),
        ("recv_count", ctypes.c_void_p),
        ("rank_counter", ctypes.c_void_p),
        ("tile_counter", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
        ("trace", ctypes.c_void_p),
        ("trace_records", ctypes.c_int64),
        ("epoch_word", ctypes.c_void_p),
    ]


class EpRouteParams(ctypes.Structure):
    _fields_ = [
        ("n_experts", ctypes.c_int32),
        ("n_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("logits_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class EpW4Format(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("scales", ctypes.c_int32),
    ]


class EpError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_lib = None


def load_library(path: str | None = None):
    """Loads the HIP library once (torch is imported first so that the library
    binds to the HIP runtime torch already loaded)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"HIP library {path} is missing; build it with "
            "`python -m grouped_gemm_scatter_amd.build` (there is no fallback path)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    lib.ep_combine_init.argtypes = [ctypes.POINTER(EpCombineParams),
                                    ctypes.POINTER(EpCombineBuffers), ctypes.POINTER(vp)]
    lib.ep_combine_init.restype = ctypes.c_int
    lib.ep_combine_destroy.argtypes = [vp]
    lib.ep_combine_destroy.restype = None
    lib.ep_grouped_gemm_scatter.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, u64, vp]
    lib.ep_grouped_gemm_scatter.restype = ctypes.c_int
    lib.ep_grouped_gemm_scatter_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, vp,
                                                    u64, vp]
    lib.ep_grouped_gemm_scatter_noalloc.restype = ctypes.c_int
    lib.ep_grouped_gemm_scatter_combine.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32,
                                                    vp, u64, vp]
    lib.ep_grouped_gemm_scatter_combine.restype = ctypes.c_int
    lib.ep_grouped_gemm_swiglu.argtypes = [vp, vp, vp, vp, i32, vp, vp]
    lib.ep_grouped_gemm_swiglu_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
    lib.ep_grouped_gemm_swiglu_fp8.restype = ctypes.c_int
    lib.ep_grouped_gemm_swiglu.restype = ctypes.c_int
    lib.ep_gemm_tile.argtypes = [vp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.ep_gemm_tile.restype = ctypes.c_int
    lib.ep_group_local_picks.argtypes = [vp, vp, i32, vp, vp, vp]
    lib.ep_dispatch_rows.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, vp]
    lib.ep_dispatch_rows.restype = ctypes.c_int
    lib.ep_pack_weights.argtypes = [vp, vp, vp, vp]
    lib.ep_advance_epoch.argtypes = [vp, vp]
    lib.ep_advance_epoch.restype = ctypes.c_int
    lib.ep_pack_weights.restype = ctypes.c_int
    lib.ep_group_local_picks.restype = ctypes.c_int
    lib.ep_signal_completion.argtypes = [vp, vp, vp, vp, i32, u64, vp]
    lib.ep_signal_completion.restype = ctypes.c_int
    lib.ep_combine_reduce.argtypes = [vp, vp, vp, i32, vp, u64, vp]
    lib.ep_combine_reduce.restype = ctypes.c_int
    route, w4 = ctypes.POINTER(EpRouteParams), ctypes.POINTER(EpW4Format)
    lib.ep_route_topk.argtypes = [vp, route, vp, vp, i32, vp, vp, vp]
    lib.ep_route_topk.restype = ctypes.c_int
    lib.ep_route_topk_backward.argtypes = [vp, route, vp, vp, vp, i32, vp, vp]
    lib.ep_route_topk_backward.restype = ctypes.c_int
    lib.ep_combine_backward.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp]
    lib.ep_combine_backward.restype = ctypes.c_int
    lib.ep_pack_weights_w4.argtypes = [vp, w4, vp, vp, i32, i32, vp, vp, vp]
    lib.ep_pack_weights_w4.restype = ctypes.c_int
    lib.ep_grouped_gemm_swiglu_w4.argtypes = [vp, w4, vp, vp, vp, vp, i32, vp, vp]
    lib.ep_grouped_gemm_swiglu_w4.restype = ctypes.c_int
    lib.ep_grouped_gemm_scatter_w4.argtypes = [vp, w4, vp, vp, vp, vp, vp, i32, i32, vp, u64, vp]
    lib.ep_grouped_gemm_scatter_w4.restype = ctypes.c_int
    lib.ep_combine_query_error.argtypes = [vp, vp]
    lib.ep_combine_query_error.restype = ctypes.c_int
    lib.ep_combine_strerror.argtypes = [ctypes.c_int]
    lib.ep_combine_strerror.restype = ctypes.c_char_p
    lib.ep_combine_version.argtypes = []
    lib.ep_combine_version.restype = ctypes.c_int
    del i64
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load_library().ep_combine_strerror(int(code)).decode()


def _ptr(t, dtype=None, name="tensor", allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t.data_ptr()


# the current stream's handle without the stream object around it (2.5 us less a call)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _current_raw_stream is not None:
            return _current_raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise EpError(rc, what)
    return rc


def make_params(*, n_ranks, my_rank, top_k, msg_bytes, max_tokens_per_rank,
                n_experts_per_device, hidden_k, hidden_n, dtype=EP_DTYPE_BF16, flags=0,
                flag_spin_limit=0, p2p_world_size=None, send_waves=0) -> EpCombineParams:
    return EpCombineParams(n_ranks, n_ranks if p2p_world_size is None else p2p_world_size,
                           my_rank, top_k, msg_bytes, max_tokens_per_rank,
                           n_experts_per_device, hidden_k, hidden_n, dtype, flags, send_waves,
                           flag_spin_limit)


def ep_combine_init(params: EpCombineParams, recv_bufs, recv_count, rank_counter,
                    tile_counter, error_word, trace=None, epoch_word=None) -> int:
    """Returns an opaque handle (int).  Buffers are device tensors that must
    outlive the handle; `trace` is an int64 [records][4] tensor, used with
    EP_FLAG_TRACE only; `epoch_word` one int64, with EP_FLAG_DEVICE_EPOCH only."""
    lib = load_library()
    b = EpCombineBuffers()
    if len(recv_bufs) > EP_MAX_RANKS:
        raise ValueError("at most 8 receive buffers")
    for i, rb in enumerate(recv_bufs):
        b.recv_buf[i] = _ptr(rb, torch.uint8, f"recv_buf[{i}]")
    b.recv_count = _ptr(recv_count, (torch.int64, torch.uint64), "recv_count")
    b.rank_counter = _ptr(rank_counter, torch.int32, "rank_counter")
    b.tile_counter = _ptr(tile_counter, torch.int32, "tile_counter")
    b.error_word = _ptr(error_word, torch.int32, "error_word")
    if trace is not None:
        if trace.dim() != 2 or trace.shape[1] != 4:
            raise ValueError("trace must be [records][4]")
        b.trace = _ptr(trace, (torch.int64, torch.uint64), "trace")
        b.trace_records = trace.shape[0]
    if epoch_word is not None:
        b.epoch_word = _ptr(epoch_word, (torch.int64, torch.uint64), "epoch_word")
    h = ctypes.c_void_p()
    _check(lib.ep_combine_init(ctypes.byref(params), ctypes.byref(b), ctypes.byref(h)),
           "ep_combine_init")
    return h.value


def ep_combine_destroy(h: int) -> None:
    if h:
        load_library().ep_combine_destroy(h)


def ep_grouped_gemm_scatter(h, x, w, x_scale, w_scale, offsets, src_info, m_total,
                            p3_control=0, c_local=None, epoch=1, stream=None,
                            noalloc=False) -> int:
    """The GEMM + scatter call; ``noalloc`` selects the allocation-free entry
    point ep_grouped_gemm_scatter_noalloc (library-held counters)."""
    lib = load_library()
    name = "ep_grouped_gemm_scatter_noalloc" if noalloc else "ep_grouped_gemm_scatter"
    rc = getattr(lib, name)(
        h, _ptr(x, None, "x", allow_none=True), _ptr(w, None, "w"),
        _ptr(x_scale, torch.float32, "x_scale", allow_none=True),
        _ptr(w_scale, torch.float32, "w_scale", allow_none=True),
        _ptr(offsets, torch.int32, "offsets"),
        _ptr(src_info, torch.int32, "src_info", allow_none=True),
        int(m_total), int(p3_control), _ptr(c_local, torch.bfloat16, "c_local", allow_none=True),
        int(epoch), _stream(stream))
    return _check(rc, name)


def ep_grouped_gemm_scatter_combine(h, x, w, x_scale, w_scale, offsets, src_info, m_total,
                                    topk_ids, topk_w, tokens_per_rank, out, epoch=1,
                                    stream=None) -> int:
    lib = load_library()
    rc = lib.ep_grouped_gemm_scatter_combine(
        h, _ptr(x, None, "x", allow_none=True), _ptr(w, None, "w"),
        _ptr(x_scale, torch.float32, "x_scale", allow_none=True),
        _ptr(w_scale, torch.float32, "w_scale", allow_none=True),
        _ptr(offsets, torch.int32, "offsets"),
        _ptr(src_info, torch.int32, "src_info", allow_none=True), int(m_total),
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(topk_w, torch.float32, "topk_w"),
        int(tokens_per_rank), _ptr(out, torch.bfloat16, "out"), int(epoch), _stream(stream))
    return _check(rc, "ep_grouped_gemm_scatter_combine")


def ep_gemm_tile(h, m_total) -> tuple:
    """(tile kind, tile rows, tile columns) ep_grouped_gemm_scatter uses for
    m_total rows on handle h."""
    lib = load_library()
    r, c = ctypes.c_int32(), ctypes.c_int32()
    kind = _check(lib.ep_gemm_tile(h, int(m_total), ctypes.byref(r), ctypes.byref(c)),
                  "ep_gemm_tile")
    return kind, r.value, c.value


def ep_dispatch_rows(h, tokens_x, tokens_per_rank, row_bytes, offsets, src_info, m_total,
                     x_out, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_dispatch_rows(h, _ptr(tokens_x, None, "tokens_x", allow_none=True),
                              int(tokens_per_rank), int(row_bytes),
                              _ptr(offsets, torch.int32, "offsets"),
                              _ptr(src_info, torch.int32, "src_info", allow_none=True),
                              int(m_total), _ptr(x_out, None, "x_out", allow_none=True),
                              _stream(stream))
    return _check(rc, "ep_dispatch_rows")


def ep_advance_epoch(h, stream=None) -> int:
    lib = load_library()
    return _check(lib.ep_advance_epoch(h, _stream(stream)), "ep_advance_epoch")


def ep_pack_weights(h, w, w_out, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_pack_weights(h, _ptr(w, torch.bfloat16, "w"), _ptr(w_out, torch.bfloat16, "w_out"),
                             _stream(stream))
    return _check(rc, "ep_pack_weights")


def ep_group_local_picks(h, topk_ids, tokens_per_rank, offsets, src_info, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_group_local_picks(h, _ptr(topk_ids, torch.int32, "topk_ids", allow_none=True),
                                  int(tokens_per_rank), _ptr(offsets, torch.int32, "offsets"),
                                  _ptr(src_info, torch.int32, "src_info", allow_none=True),
                                  _stream(stream))
    return _check(rc, "ep_group_local_picks")


def ep_grouped_gemm_swiglu(h, x1, w1, offsets, m_total, h_out, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_grouped_gemm_swiglu(
        h, _ptr(x1, torch.bfloat16, "x1", allow_none=True), _ptr(w1, torch.bfloat16, "w1"),
        _ptr(offsets, torch.int32, "offsets"), int(m_total),
        _ptr(h_out, torch.bfloat16, "h_out", allow_none=True), _stream(stream))
    return _check(rc, "ep_grouped_gemm_swiglu")


def ep_grouped_gemm_swiglu_fp8(h, x1, x1_scale, w1, w1_scale, offsets, m_total, h_out, h_scale,
                               stream=None) -> int:
    lib = load_library()
    rc = lib.ep_grouped_gemm_swiglu_fp8(
        h, _ptr(x1, torch.uint8, "x1", allow_none=True),
        _ptr(x1_scale, torch.float32, "x1_scale", allow_none=True), _ptr(w1, torch.uint8, "w1"),
        _ptr(w1_scale, torch.float32, "w1_scale"), _ptr(offsets, torch.int32, "offsets"),
        int(m_total), _ptr(h_out, torch.uint8, "h_out", allow_none=True),
        _ptr(h_scale, torch.float32, "h_scale", allow_none=True), _stream(stream))
    return _check(rc, "ep_grouped_gemm_swiglu_fp8")


def ep_signal_completion(h, expert, dst_rank, signal, n, epoch, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_signal_completion(h, _ptr(expert, torch.int32, "expert", allow_none=True),
                                  _ptr(dst_rank, torch.int32, "dst_rank", allow_none=True),
                                  _ptr(signal, (torch.int64, torch.uint64), "signal",
                                       allow_none=True),
                                  int(n), int(epoch), _stream(stream))
    return _check(rc, "ep_signal_completion")


def ep_combine_reduce(h, topk_ids, topk_w, tokens_per_rank, out, epoch, stream=None) -> int:
    lib = load_library()
    rc = lib.ep_combine_reduce(h, _ptr(topk_ids, torch.int32, "topk_ids"),
                               _ptr(topk_w, torch.float32, "topk_w"), int(tokens_per_rank),
                               _ptr(out, torch.bfloat16, "out"), int(epoch), _stream(stream))
    return _check(rc, "ep_combine_reduce")


_LOGITS = {torch.float32: EP_LOGITS_F32, torch.bfloat16: EP_LOGITS_BF16,
           torch.float16: EP_LOGITS_F16}
_W4_SCALES = {torch.bfloat16: EP_W4_SCALE_BF16, torch.float16: EP_W4_SCALE_F16}


def make_route_params(*, n_experts, logits_dtype, n_groups=1, topk_groups=1,
                      score=EP_SCORE_SOFTMAX, group_score=EP_GROUP_MAX, renormalize=True,
                      scale=1.0) -> EpRouteParams:
    if logits_dtype not in _LOGITS:
        raise ValueError(f"logits must be float32, bfloat16 or float16, not {logits_dtype}")
    return EpRouteParams(n_experts, n_groups, topk_groups, score, group_score, int(renormalize),
                         _LOGITS[logits_dtype], scale)


def make_w4_format(*, codes, group, scale_dtype) -> EpW4Format:
    if scale_dtype not in _W4_SCALES:
        raise ValueError(f"scales must be bfloat16 or float16, not {scale_dtype}")
    return EpW4Format(codes, group, _W4_SCALES[scale_dtype])


def ep_route_topk(h, params: EpRouteParams, logits, bias, tokens_per_rank, topk_ids, topk_w,
                  stream=None) -> int:
    rc = load_library().ep_route_topk(
        h, ctypes.byref(params), _ptr(logits, tuple(_LOGITS), "logits", allow_none=True),
        _ptr(bias, torch.float32, "bias", allow_none=True), int(tokens_per_rank),
        _ptr(topk_ids, torch.int32, "topk_ids", allow_none=True),
        _ptr(topk_w, torch.float32, "topk_w", allow_none=True), _stream(stream))
    return _check(rc, "ep_route_topk")


def ep_route_topk_backward(h, params: EpRouteParams, logits, topk_ids, grad_w, tokens_per_rank,
                           grad_logits, stream=None) -> int:
    rc = load_library().ep_route_topk_backward(
        h, ctypes.byref(params), _ptr(logits, tuple(_LOGITS), "logits", allow_none=True),
        _ptr(topk_ids, torch.int32, "topk_ids", allow_none=True),
        _ptr(grad_w, torch.float32, "grad_w", allow_none=True), int(tokens_per_rank),
        _ptr(grad_logits, tuple(_LOGITS), "grad_logits", allow_none=True), _stream(stream))
    return _check(rc, "ep_route_topk_backward")


def ep_combine_backward(h, grad_out, topk_ids, topk_w, tokens_per_rank, offsets, src_info, m_total,
                        grad_rows, grad_w, stream=None) -> int:
    rc = load_library().ep_combine_backward(
        h, _ptr(grad_out, torch.bfloat16, "grad_out", allow_none=True),
        _ptr(topk_ids, torch.int32, "topk_ids", allow_none=True),
        _ptr(topk_w, torch.float32, "topk_w", allow_none=True), int(tokens_per_rank),
        _ptr(offsets, torch.int32, "offsets", allow_none=True),
        _ptr(src_info, torch.int32, "src_info", allow_none=True), int(m_total),
        _ptr(grad_rows, torch.bfloat16, "grad_rows", allow_none=True),
        _ptr(grad_w, torch.float32, "grad_w", allow_none=True), _stream(stream))
    return _check(rc, "ep_combine_backward")


def ep_pack_weights_w4(h, fmt: EpW4Format, codes, scales, rows, k, codes_out, scales_out,
                       stream=None) -> int:
    two = tuple(_W4_SCALES)
    rc = load_library().ep_pack_weights_w4(
        h, ctypes.byref(fmt), _ptr(codes, torch.uint8, "codes"), _ptr(scales, two, "scales"),
        int(rows), int(k), _ptr(codes_out, torch.uint8, "codes_out"),
        _ptr(scales_out, two, "scales_out"), _stream(stream))
    return _check(rc, "ep_pack_weights_w4")


def ep_grouped_gemm_swiglu_w4(h, fmt: EpW4Format, x1, w1, w1_scale, offsets, m_total, h_out,
                              stream=None) -> int:
    rc = load_library().ep_grouped_gemm_swiglu_w4(
        h, ctypes.byref(fmt), _ptr(x1, torch.bfloat16, "x1", allow_none=True),
        _ptr(w1, torch.uint8, "w1"), _ptr(w1_scale, tuple(_W4_SCALES), "w1_scale"),
        _ptr(offsets, torch.int32, "offsets"), int(m_total),
        _ptr(h_out, torch.bfloat16, "h_out", allow_none=True), _stream(stream))
    return _check(rc, "ep_grouped_gemm_swiglu_w4")


def ep_grouped_gemm_scatter_w4(h, fmt: EpW4Format, x, w, w_scale, offsets, src_info, m_total,
                               p3_control=0, c_local=None, epoch=1, stream=None) -> int:
    rc = load_library().ep_grouped_gemm_scatter_w4(
        h, ctypes.byref(fmt), _ptr(x, torch.bfloat16, "x", allow_none=True),
        _ptr(w, torch.uint8, "w"), _ptr(w_scale, tuple(_W4_SCALES), "w_scale"),
        _ptr(offsets, torch.int32, "offsets"),
        _ptr(src_info, torch.int32, "src_info", allow_none=True), int(m_total), int(p3_control),
        _ptr(c_local, torch.bfloat16, "c_local", allow_none=True), int(epoch), _stream(stream))
    return _check(rc, "ep_grouped_gemm_scatter_w4")


def ep_combine_query_error(h, stream=None) -> int:
    return _check(load_library().ep_combine_query_error(h, _stream(stream)),
                  "ep_combine_query_error")


def ep_combine_strerror(code: int) -> str:
    return strerror(code)


def ep_combine_version() -> int:
    return load_library().ep_combine_version()
