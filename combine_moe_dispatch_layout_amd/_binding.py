"""ctypes binding of libmoe_ep.so (include/moe_ep.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  torch provides device memory (torch.empty on the current device) and
the stream (torch.cuda.current_stream()).  There is no fallback: if the library
is missing or a call fails, an exception is raised.
"""
import ctypes
import functools
import os
from operator import index as _index

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_ep.so")

# ---------------------------------------------------------------- constants
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CAPACITY = 3
MOE_ERR_HANDLE = 4
MOE_ERR_HIP = 5
MOE_ERR_BAD_TOPK = 6
MOE_ERR_DEVICE_BOUNDS = 7
MOE_ERR_STALE_LAYOUT = 8
MOE_ERR_NONFINITE = 9
# moe_poll_error's raw bits
ERR_FLAG_BAD_TOPK, ERR_FLAG_BOUNDS, ERR_FLAG_CAPACITY, ERR_FLAG_STALE, ERR_FLAG_NONFINITE = 1, 2, 4, 8, 16
_POLL_STATUSES = (MOE_OK, MOE_ERR_BAD_TOPK, MOE_ERR_CAPACITY, MOE_ERR_DEVICE_BOUNDS, MOE_ERR_STALE_LAYOUT,
                  MOE_ERR_NONFINITE)

MOE_QUANT_BF16 = 0
MOE_QUANT_FP8_E4M3 = 1
MOE_LAYOUT_CONTIGUOUS = 0
MOE_LAYOUT_PADDED_LL = 1

(MOE_BUF_SEND_ROWS, MOE_BUF_SEND_SCALES, MOE_BUF_RECV_ROWS, MOE_BUF_RECV_SCALES, MOE_BUF_EXPERT_OUT,
 MOE_BUF_COMBINE_OUT, MOE_BUF_HANDLE_POS, MOE_BUF_HANDLE_EXPERT_OFFSETS, MOE_BUF_HANDLE_RANK_OFFSETS,
 MOE_BUF_HANDLE_SEND_SRC, MOE_BUF_HANDLE_RECV_SRC, MOE_BUF_HANDLE_RECV_COUNTS,
 MOE_BUF_LAYOUT_EXPERT_COUNTS, MOE_BUF_LAYOUT_RANK_COUNTS, MOE_BUF_LAYOUT_TOKEN_IN_RANK,
 MOE_BUF_WORKSPACE) = range(16)

(MOE_KERNEL_LAYOUT, MOE_KERNEL_DISPATCH, MOE_KERNEL_COMBINE, MOE_KERNEL_DISPATCH_BWD,
 MOE_KERNEL_COMBINE_BWD, MOE_KERNEL_EXPERT_GEMM, MOE_KERNEL_EXPERT_BWD_ROWS, MOE_KERNEL_EXPERT_BWD_WEIGHTS,
 MOE_KERNEL_SWIGLU, MOE_KERNEL_SWIGLU_BWD, MOE_KERNEL_ROUTE, MOE_KERNEL_ROUTE_BWD, MOE_KERNEL_LINEAR,
 MOE_KERNEL_LINEAR_BWD, MOE_KERNEL_LAYER) = range(15)
KERNEL_NAMES = ("layout", "dispatch", "combine", "dispatch_bwd", "combine_bwd", "expert_gemm", "expert_bwd_rows",
                "expert_bwd_weights", "swiglu", "swiglu_bwd", "route", "route_bwd", "linear", "linear_bwd", "layer")

# order of a row buffer of the expert products and the activation
MOE_ROWS_RECV, MOE_ROWS_PACKED = 0, 1
MOE_GRAD_BF16, MOE_GRAD_F32 = 0, 1
MOE_MAX_FEATURES = 65536

# the router, the dense product, the layer of a few tokens
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_LOGIT_F32, MOE_LOGIT_BF16 = 0, 1
MOE_MAX_GROUPS = 64
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SWIGLU = range(6)
MOE_OUT_BF16, MOE_OUT_F32 = 0, 1
MOE_LAYER_MAX_ROWS = 1024


class MoeError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s" % (what, status_str(status)))


# ctypes passes the lower 32 bits of a number that is longer: sizes and settings are looked at before.
_INT_MAX = 2 ** 31 - 1


def _int32(*values):
    for v in values:
        if not -_INT_MAX <= v <= _INT_MAX:
            raise MoeError(MOE_ERR_UNSUPPORTED, "a size or setting of %d" % v)


def _tokens(n):
    """A batch's tokens, which no context has more than 2^31 - 1 of."""
    if n > _INT_MAX:
        raise MoeError(MOE_ERR_CAPACITY, "a batch of %d tokens" % n)
    return n


# ---------------------------------------------------------------- C structs
class moe_config(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_ranks", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("src_rank", ctypes.c_int32),
                ("quant", ctypes.c_int32), ("layout", ctypes.c_int32)]


class moe_dispatch_buffers(ctypes.Structure):
    _fields_ = [("send_rows", ctypes.c_void_p), ("send_scales", ctypes.c_void_p),
                ("recv_rows", ctypes.c_void_p), ("recv_scales", ctypes.c_void_p)]


class moe_handle(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("rank_offsets", ctypes.c_void_p), ("send_src_idx", ctypes.c_void_p),
                ("recv_src_idx", ctypes.c_void_p), ("recv_counts", ctypes.c_void_p),
                ("num_tokens", ctypes.c_int32), ("tag", ctypes.c_uint32)]


class moe_router(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("normalize", ctypes.c_int32), ("scale", ctypes.c_float)]


# the full list of symbols include/moe_ep.h declares
EXPORTS = ("moe_status_str", "moe_size_hint", "moe_ctx_create", "moe_ctx_destroy", "moe_ctx_config",
           "moe_ctx_tune", "moe_dispatch_layout", "moe_dispatch", "moe_combine", "moe_dispatch_backward",
           "moe_combine_backward", "moe_ctx_set_max_workgroups", "moe_hook_create", "moe_hook_destroy",
           "moe_hook_record", "moe_hook_wait", "moe_poll_error", "moe_timing_begin", "moe_timing_end",
           "moe_timing_launches", "moe_dispatch_noalloc",
           "moe_dispatch_layout_prefetch", "moe_expert_gemm", "moe_expert_gemm_fp8",
           "moe_expert_gemm_backward_rows", "moe_expert_gemm_backward_weights", "moe_swiglu", "moe_swiglu_fp8",
           "moe_swiglu_backward", "moe_route", "moe_route_backward", "moe_linear", "moe_linear_backward",
           "moe_linear_workspace", "moe_linear_backward_workspace", "moe_layer", "moe_layer_fp8")

_lib = None


def load_library(path=LIB_PATH):
    """Open libmoe_ep.so (raises if it has not been built) and declare the ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libmoe_ep.so is not built (%s); run `python __graft_entry__.py` "
                           "or combine_moe_dispatch_layout_amd/_build.py" % path)
    lib = ctypes.CDLL(path)
    vp, i32, u32p = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_status_str.argtypes = [ctypes.c_int]
    sigs = {
        "moe_size_hint": [ctypes.POINTER(moe_config), i32, ctypes.POINTER(ctypes.c_size_t)],
        "moe_ctx_create": [ctypes.POINTER(moe_config), ctypes.POINTER(vp)],
        "moe_ctx_destroy": [vp],
        "moe_ctx_config": [vp, ctypes.POINTER(moe_config)],
        "moe_ctx_tune": [vp, i32, i32],
        "moe_dispatch_layout": [vp, vp, i32, vp, vp, vp, vp],
        "moe_dispatch_layout_prefetch": [vp, vp, i32, vp, vp, vp, vp, vp],
        "moe_dispatch": [vp, vp, vp, i32, i32, ctypes.POINTER(moe_dispatch_buffers),
                         ctypes.POINTER(moe_handle), vp],
        "moe_combine": [vp, vp, vp, ctypes.POINTER(moe_handle), vp, vp],
        "moe_dispatch_backward": [vp, vp, ctypes.POINTER(moe_handle), vp, vp],
        "moe_combine_backward": [vp, vp, vp, vp, ctypes.POINTER(moe_handle), vp, vp, vp],
        "moe_ctx_set_max_workgroups": [vp, i32],
        "moe_hook_create": [ctypes.POINTER(vp)],
        "moe_hook_destroy": [vp],
        "moe_hook_record": [vp, vp],
        "moe_hook_wait": [vp, vp],
        "moe_poll_error": [vp, vp, u32p],
        "moe_timing_begin": [vp, i32],
        "moe_timing_end": [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)],
        "moe_timing_launches": [vp, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_float), i32,
                                ctypes.POINTER(ctypes.c_int32)],
        "moe_dispatch_noalloc": [ctypes.POINTER(moe_config), vp, vp, i32, ctypes.POINTER(moe_dispatch_buffers),
                                 ctypes.POINTER(moe_handle), vp, vp],
        "moe_expert_gemm": [vp, vp, i32, vp, i32, i32, ctypes.POINTER(moe_handle), vp, i32, vp],
        "moe_expert_gemm_fp8": [vp, vp, vp, i32, vp, vp, i32, i32, ctypes.POINTER(moe_handle), vp, i32, vp],
        "moe_expert_gemm_backward_rows": [vp, vp, i32, vp, i32, i32, ctypes.POINTER(moe_handle), vp, i32, vp],
        "moe_expert_gemm_backward_weights": [vp, vp, i32, vp, i32, i32, i32, ctypes.POINTER(moe_handle), vp, i32,
                                             i32, vp],
        "moe_swiglu": [vp, vp, i32, i32, ctypes.POINTER(moe_handle), vp, vp],
        "moe_swiglu_fp8": [vp, vp, i32, i32, ctypes.POINTER(moe_handle), vp, vp, vp],
        "moe_swiglu_backward": [vp, vp, vp, i32, i32, ctypes.POINTER(moe_handle), vp, vp],
        "moe_route": [vp, vp, i32, ctypes.c_int64, i32, ctypes.POINTER(moe_router), vp, vp, vp, vp],
        "moe_route_backward": [vp, vp, vp, i32, ctypes.c_int64, vp, i32, ctypes.POINTER(moe_router), vp, vp],
        "moe_linear": [vp, vp, i32, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp],
        "moe_linear_workspace": [i32, i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)],
        "moe_linear_backward": [vp, vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp],
        "moe_linear_backward_workspace": [i32, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)],
        "moe_layer": [vp, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, vp],
        "moe_layer_fp8": [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    _lib = lib
    return lib


def status_str(status):
    return load_library().moe_status_str(status).decode()


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


# Pointers and stream handles go to the C calls as plain ints (or None for
# NULL): ctypes converts them for c_void_p parameters, which costs less host
# time per call than building c_void_p objects.
def _ptr(t):
    return t.data_ptr() if t is not None else None


# torch's raw current-stream and device queries: ~0.1 us against ~2.7 us for
# building a torch.cuda.Stream object per call (half of an eager decode step's
# host time otherwise); the public API is the fallback where they are missing
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream=None):
    """HIP stream handle (an int; 0 = the null stream) of a torch stream
    (default: the current stream)."""
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(_raw_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def make_config(max_tokens, hidden, num_experts, num_ranks, topk, src_rank=0,
                quant=MOE_QUANT_BF16, layout=MOE_LAYOUT_CONTIGUOUS):
    return moe_config(max_tokens, hidden, num_experts, num_ranks, topk, src_rank, quant, layout)


def moe_size_hint(cfg, kind):
    n = ctypes.c_size_t(0)
    _check(load_library().moe_size_hint(ctypes.byref(cfg), kind, ctypes.byref(n)), "moe_size_hint")
    return n.value


# ---------------------------------------------------------------- context
class Context:
    """A moe_ctx on the current device, plus the configuration it was made with."""

    def __init__(self, cfg):
        lib = load_library()
        self.cfg = cfg
        h = ctypes.c_void_p(0)
        _check(lib.moe_ctx_create(ctypes.byref(cfg), ctypes.byref(h)), "moe_ctx_create")
        self._h = h
        self.device = torch.cuda.current_device()
        # identifies this context (and so its configuration) to the buffer
        # checks of the calls; a fresh object per context
        self._fit_token = object()

    @property
    def handle(self):
        if self._h is None or not self._h.value:
            raise RuntimeError("context already destroyed")
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _check(load_library().moe_ctx_destroy(self._h), "moe_ctx_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def hint(self, kind):
        """moe_size_hint for this context's configuration (fixed, so cached)."""
        cache = self.__dict__.setdefault("_hints", {})
        if kind not in cache:
            cache[kind] = moe_size_hint(self.cfg, kind)
        return cache[kind]

    def tune(self, dispatch_chunks=0, combine_chunks=0):
        _check(load_library().moe_ctx_tune(self.handle, dispatch_chunks, combine_chunks), "moe_ctx_tune")

    def set_max_workgroups(self, n):
        """Cap the workgroups of the dispatch, combine and backward kernels (0 = none)."""
        _check(load_library().moe_ctx_set_max_workgroups(self.handle, int(n)), "moe_ctx_set_max_workgroups")

    def timing_begin(self, max_launches):
        _check(load_library().moe_timing_begin(self.handle, max_launches), "moe_timing_begin")

    def timing_launches(self):
        """[(kernel name, ms)] of every launch timed so far, in launch order
        (before timing_end)."""
        lib = load_library()
        n = ctypes.c_int32(0)
        _check(lib.moe_timing_launches(self.handle, None, None, 0, ctypes.byref(n)), "moe_timing_launches")
        ids = (ctypes.c_int32 * max(n.value, 1))()
        ms = (ctypes.c_float * max(n.value, 1))()
        _check(lib.moe_timing_launches(self.handle, ids, ms, n.value, ctypes.byref(n)), "moe_timing_launches")
        return [(KERNEL_NAMES[ids[i]], ms[i]) for i in range(n.value)]

    def timing_end(self):
        n = len(KERNEL_NAMES)
        tot = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        _check(load_library().moe_timing_end(self.handle, tot, cnt), "moe_timing_end")
        return {KERNEL_NAMES[i]: {"total_ms": tot[i], "launches": cnt[i]} for i in range(n)}


class Hook:
    """Issue/complete split: record() after enqueuing dispatch or combine on a
    side stream, wait() on the stream that needs the results."""

    def __init__(self):
        self.h = ctypes.c_void_p()
        _check(load_library().moe_hook_create(ctypes.byref(self.h)), "moe_hook_create")

    def record(self, stream=None):
        _check(load_library().moe_hook_record(self.h, _stream(stream)), "moe_hook_record")

    def wait(self, stream=None):
        _check(load_library().moe_hook_wait(self.h, _stream(stream)), "moe_hook_wait")

    def close(self):
        if self.h:
            _check(load_library().moe_hook_destroy(self.h), "moe_hook_destroy")
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Handle:
    """Caller-owned device arrays of one dispatch (moe_handle), as torch tensors."""

    def __init__(self, ctx):
        c = ctx.cfg
        dev = torch.device("cuda", ctx.device)
        ksend = min(c.topk, c.num_ranks)
        i32 = torch.int32
        self.pos = torch.empty((c.max_tokens, c.topk), dtype=i32, device=dev)
        self.expert_offsets = torch.empty(c.num_experts + 1, dtype=i32, device=dev)
        self.rank_offsets = torch.empty(c.num_ranks + 1, dtype=i32, device=dev)
        self.send_src_idx = torch.empty(c.max_tokens * ksend, dtype=i32, device=dev)
        self.recv_src_idx = torch.empty(c.max_tokens * c.topk, dtype=i32, device=dev)
        self.recv_counts = torch.empty(c.num_experts, dtype=i32, device=dev)
        self.c = moe_handle(self.pos.data_ptr(), self.expert_offsets.data_ptr(),
                            self.rank_offsets.data_ptr(), self.send_src_idx.data_ptr(),
                            self.recv_src_idx.data_ptr(), self.recv_counts.data_ptr(), 0, 0)

    @property
    def num_tokens(self):
        return self.c.num_tokens


class DispatchBuffers:
    """Caller-owned dispatch outputs sized by moe_size_hint (full capacity)."""

    def __init__(self, ctx):
        c = ctx.cfg
        dev = torch.device("cuda", ctx.device)
        fp8 = c.quant == MOE_QUANT_FP8_E4M3
        ll = c.layout == MOE_LAYOUT_PADDED_LL
        H = c.hidden
        row_dt, row_w = (torch.uint8, H) if fp8 else (torch.bfloat16, H)
        row_bytes = H if fp8 else 2 * H
        n_send = ctx.hint(MOE_BUF_SEND_ROWS) // row_bytes
        n_recv = ctx.hint(MOE_BUF_RECV_ROWS) // row_bytes
        self.send_rows = None if ll else torch.empty((n_send, row_w), dtype=row_dt, device=dev)
        self.send_scales = (torch.empty((n_send, H // 128), dtype=torch.float32, device=dev)
                            if fp8 and not ll else None)
        self.recv_rows = torch.empty((n_recv, row_w), dtype=row_dt, device=dev)
        self.recv_scales = torch.empty((n_recv, H // 128), dtype=torch.float32, device=dev) if fp8 else None
        self.c = moe_dispatch_buffers(_ptr(self.send_rows), _ptr(self.send_scales),
                                      _ptr(self.recv_rows), _ptr(self.recv_scales))


# ---------------------------------------------------------------- the calls
def _as_dev(t, dtype, name):
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    return t


def _out(t, dtype, numel, name):
    """A caller-supplied output: contiguous, of the right dtype, at least numel elements."""
    _as_dev(t, dtype, name)
    if t.numel() < numel:
        raise ValueError("%s holds %d elements, needs %d" % (name, t.numel(), numel))
    return t


def _fits(ctx, obj, parts, what):
    """The kernels write a handle's arrays and the dispatch buffers through raw
    pointers, up to the sizes moe_size_hint gives for the context's
    configuration: check that every part is at least that large (and that the
    C struct still points at it), once per (object, context)."""
    key = ctx._fit_token
    if getattr(obj, "_fits_key", None) is key:
        return
    for t, kind, ptr in parts:
        need = ctx.hint(kind)
        if t is None:
            if need:
                raise ValueError("%s lacks a buffer this configuration needs (kind %d)" % (what, kind))
            continue
        if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < need:
            raise ValueError("%s was not made for this context's configuration (kind %d: %d bytes, needs %d)"
                             % (what, kind, t.numel() * t.element_size(), need))
        if ptr != t.data_ptr():
            raise ValueError("%s: the C struct no longer points at its tensors" % what)
    obj._fits_key = key


def _check_handle(ctx, h):
    if getattr(h, "_fits_key", None) is ctx._fit_token:   # checked before, as _fits does
        return
    c = h.c
    _fits(ctx, h, ((h.pos, MOE_BUF_HANDLE_POS, c.pos), (h.expert_offsets, MOE_BUF_HANDLE_EXPERT_OFFSETS,
                                                       c.expert_offsets),
                   (h.rank_offsets, MOE_BUF_HANDLE_RANK_OFFSETS, c.rank_offsets),
                   (h.send_src_idx, MOE_BUF_HANDLE_SEND_SRC, c.send_src_idx),
                   (h.recv_src_idx, MOE_BUF_HANDLE_RECV_SRC, c.recv_src_idx),
                   (h.recv_counts, MOE_BUF_HANDLE_RECV_COUNTS, c.recv_counts)), "handle")


def _check_bufs(ctx, b):
    c = b.c
    _fits(ctx, b, ((b.send_rows, MOE_BUF_SEND_ROWS, c.send_rows or 0),
                   (b.send_scales, MOE_BUF_SEND_SCALES, c.send_scales or 0),
                   (b.recv_rows, MOE_BUF_RECV_ROWS, c.recv_rows or 0),
                   (b.recv_scales, MOE_BUF_RECV_SCALES, c.recv_scales or 0)), "dispatch buffers")


def moe_dispatch_layout(ctx, topk_idx, num_tokens_per_expert=None, num_tokens_per_rank=None,
                        is_token_in_rank=None, x=None):
    """Returns (num_tokens_per_expert int32[E], num_tokens_per_rank int32[R],
    is_token_in_rank uint8[T, R]).  x: the bf16 token rows [T, H] of the
    dispatch that will reuse this layout; given, the same launch reads them
    into the Infinity Cache (moe_dispatch_layout_prefetch)."""
    c = ctx.cfg
    _as_dev(topk_idx, torch.int64, "topk_idx")
    T = _tokens(topk_idx.shape[0])
    if topk_idx.dim() != 2 or topk_idx.shape[1] != c.topk:
        raise ValueError("topk_idx must be [T, %d]" % c.topk)
    dev = topk_idx.device
    if num_tokens_per_expert is None:
        num_tokens_per_expert = torch.empty(c.num_experts, dtype=torch.int32, device=dev)
    if num_tokens_per_rank is None:
        num_tokens_per_rank = torch.empty(c.num_ranks, dtype=torch.int32, device=dev)
    if is_token_in_rank is None:
        is_token_in_rank = torch.empty((T, c.num_ranks), dtype=torch.uint8, device=dev)
    _out(num_tokens_per_expert, torch.int32, c.num_experts, "num_tokens_per_expert")
    _out(num_tokens_per_rank, torch.int32, c.num_ranks, "num_tokens_per_rank")
    _out(is_token_in_rank, torch.uint8, T * c.num_ranks, "is_token_in_rank")
    if x is None:
        _check(load_library().moe_dispatch_layout(
            ctx.handle, _ptr(topk_idx), T, _ptr(num_tokens_per_expert), _ptr(num_tokens_per_rank),
            _ptr(is_token_in_rank), _stream()), "moe_dispatch_layout")
    else:
        _as_dev(x, torch.bfloat16, "x")
        if x.dim() != 2 or tuple(x.shape) != (T, c.hidden):
            raise ValueError("x must be [T, %d]" % c.hidden)
        _check(load_library().moe_dispatch_layout_prefetch(
            ctx.handle, _ptr(topk_idx), T, _ptr(x), _ptr(num_tokens_per_expert), _ptr(num_tokens_per_rank),
            _ptr(is_token_in_rank), _stream()), "moe_dispatch_layout_prefetch")
    return num_tokens_per_expert, num_tokens_per_rank, is_token_in_rank


def moe_dispatch(ctx, x, topk_idx, reuse_layout=False, bufs=None, handle=None):
    """Returns (DispatchBuffers, Handle).  Pass preallocated bufs/handle to
    avoid any allocation (e.g. inside timed loops)."""
    c = ctx.cfg
    _as_dev(x, torch.bfloat16, "x")
    _as_dev(topk_idx, torch.int64, "topk_idx")
    xs = x.shape
    T = _tokens(xs[0])
    if len(xs) != 2 or xs[1] != c.hidden or topk_idx.shape != (T, c.topk):
        raise ValueError("x must be [T, %d] and topk_idx [T, %d]" % (c.hidden, c.topk))
    if bufs is None:
        bufs = DispatchBuffers(ctx)
    if handle is None:
        handle = Handle(ctx)
    _check_bufs(ctx, bufs)
    _check_handle(ctx, handle)
    _check(load_library().moe_dispatch(ctx.handle, _ptr(x), _ptr(topk_idx), T, int(bool(reuse_layout)),
                                       ctypes.byref(bufs.c), ctypes.byref(handle.c), _stream()),
           "moe_dispatch")
    return bufs, handle


def moe_combine(ctx, expert_out, topk_weights, handle, out=None):
    """Returns out, bf16 [T, H]."""
    c = ctx.cfg
    _as_dev(expert_out, torch.bfloat16, "expert_out")
    _as_dev(topk_weights, torch.float32, "topk_weights")
    T = handle.num_tokens
    if topk_weights.shape != (T, c.topk):
        raise ValueError("topk_weights must be [T, %d]" % c.topk)
    if expert_out.numel() * 2 < ctx.hint(MOE_BUF_EXPERT_OUT):
        raise ValueError("expert_out smaller than MOE_BUF_EXPERT_OUT")
    if out is None:
        out = torch.empty((T, c.hidden), dtype=torch.bfloat16, device=expert_out.device)
    _out(out, torch.bfloat16, T * c.hidden, "out")
    _check(load_library().moe_combine(ctx.handle, _ptr(expert_out), _ptr(topk_weights),
                                      ctypes.byref(handle.c), _ptr(out), _stream()), "moe_combine")
    return out


def moe_dispatch_backward(ctx, grad_recv, handle, grad_x=None):
    """Gradient of dispatch: grad_x bf16 [T, H] from the receive-layout
    gradient rows (bf16, at least MOE_BUF_EXPERT_OUT bytes)."""
    c = ctx.cfg
    _as_dev(grad_recv, torch.bfloat16, "grad_recv")
    if grad_recv.numel() * 2 < ctx.hint(MOE_BUF_EXPERT_OUT):
        raise ValueError("grad_recv smaller than MOE_BUF_EXPERT_OUT")
    T = handle.num_tokens
    if grad_x is None:
        grad_x = torch.empty((T, c.hidden), dtype=torch.bfloat16, device=grad_recv.device)
    _as_dev(grad_x, torch.bfloat16, "grad_x")
    if grad_x.numel() < T * c.hidden:
        raise ValueError("grad_x must hold [T, %d]" % c.hidden)
    _check(load_library().moe_dispatch_backward(ctx.handle, _ptr(grad_recv), ctypes.byref(handle.c),
                                                _ptr(grad_x), _stream()), "moe_dispatch_backward")
    return grad_x


def moe_combine_backward(ctx, grad_out, topk_weights, expert_out, handle, grad_expert_out=None,
                         grad_weights=None):
    """Gradients of combine: returns (grad_expert_out bf16 in the receive layout,
    grad_weights fp32 [T, k])."""
    c = ctx.cfg
    T = handle.num_tokens
    _as_dev(grad_out, torch.bfloat16, "grad_out")
    _as_dev(topk_weights, torch.float32, "topk_weights")
    _as_dev(expert_out, torch.bfloat16, "expert_out")
    if tuple(topk_weights.shape) != (T, c.topk) or grad_out.numel() < T * c.hidden:
        raise ValueError("topk_weights must be [T, %d] and grad_out [T, %d]" % (c.topk, c.hidden))
    if expert_out.numel() * 2 < ctx.hint(MOE_BUF_EXPERT_OUT):
        raise ValueError("expert_out smaller than MOE_BUF_EXPERT_OUT")
    if grad_expert_out is None:
        grad_expert_out = torch.empty_like(expert_out)
    _as_dev(grad_expert_out, torch.bfloat16, "grad_expert_out")
    if grad_expert_out.numel() * 2 < ctx.hint(MOE_BUF_EXPERT_OUT):
        raise ValueError("grad_expert_out smaller than MOE_BUF_EXPERT_OUT")
    if grad_weights is None:
        grad_weights = torch.empty((T, c.topk), dtype=torch.float32, device=grad_out.device)
    _as_dev(grad_weights, torch.float32, "grad_weights")
    if grad_weights.numel() < T * c.topk:
        raise ValueError("grad_weights must hold [T, %d]" % c.topk)
    _check(load_library().moe_combine_backward(ctx.handle, _ptr(grad_out), _ptr(topk_weights),
                                               _ptr(expert_out), ctypes.byref(handle.c),
                                               _ptr(grad_expert_out), _ptr(grad_weights), _stream()),
           "moe_combine_backward")
    return grad_expert_out, grad_weights


# ---------------------------------------------------------------- expert products
def _rows_capacity(ctx):
    """Rows of a buffer in each order: [MOE_ROWS_RECV, MOE_ROWS_PACKED] (fixed per context, so cached)."""
    cap = ctx.__dict__.get("_rows_cap")
    if cap is None:
        c = ctx.cfg
        packed = c.max_tokens * c.topk
        recv = c.num_experts * c.max_tokens * c.num_ranks if c.layout == MOE_LAYOUT_PADDED_LL else packed
        cap = ctx.__dict__["_rows_cap"] = (recv, packed)
    return cap


def _expert_rows(ctx, t, dtype, width, order, name):
    """Pointer of a row buffer of an expert product: [rows, width] of the dtype on
    the context's device, with every row that its order can address."""
    # what is right passes one test (these calls are made per product and layer); the rest says what is wrong
    if t.dtype is dtype and t.is_contiguous() and t.get_device() == ctx.device and 0 <= order <= 1:
        shape = t.shape
        if len(shape) == 2 and shape[1] == width and shape[0] >= (ctx.__dict__.get("_rows_cap") or _rows_capacity(ctx))[order]:
            return t.data_ptr()
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    if t.get_device() != ctx.device:
        raise ValueError("%s is on %s, the context on cuda:%d" % (name, t.device, ctx.device))
    if order != MOE_ROWS_RECV and order != MOE_ROWS_PACKED:
        raise ValueError("row order must be MOE_ROWS_RECV or MOE_ROWS_PACKED")
    raise ValueError("%s must be [%d, %d], is %s" % (name, _rows_capacity(ctx)[order], width, tuple(t.shape)))


def _expert_out(ctx, width, dtype, order):
    if order != MOE_ROWS_RECV and order != MOE_ROWS_PACKED:
        raise ValueError("row order must be MOE_ROWS_RECV or MOE_ROWS_PACKED")
    return torch.empty((_rows_capacity(ctx)[order], width), dtype=dtype, device=torch.device("cuda", ctx.device))


def _expert_mats(ctx, t, dtype, shape, name):
    """Pointer of the experts' matrices or their scales."""
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    if t.get_device() != ctx.device:
        raise ValueError("%s is on %s, the context on cuda:%d" % (name, t.device, ctx.device))
    if t.shape != shape:
        raise ValueError("%s must be %s, is %s" % (name, shape, tuple(t.shape)))
    return t.data_ptr()


def _mats_shape(ctx, weights):
    shape = weights.shape
    if len(shape) != 3 or shape[0] != ctx.cfg.num_experts:
        raise ValueError("weights must be [%d, out_features, in_features]" % ctx.cfg.num_experts)
    N, K = shape[1], shape[2]
    if N > _INT_MAX or K > _INT_MAX:
        _int32(N, K)
    return N, K


def moe_expert_gemm(ctx, rows, weights, handle, out=None, rows_order=MOE_ROWS_RECV, out_order=MOE_ROWS_RECV):
    """Each expert's rows times its matrix: rows bf16 [rows, K], weights bf16
    [E, N, K] -> out bf16 [rows, N].  The orders say how the row buffers are
    laid out (the receive layout, or packed by expert)."""
    N, K = _mats_shape(ctx, weights)
    _check_handle(ctx, handle)
    pw = _expert_mats(ctx, weights, torch.bfloat16, (ctx.cfg.num_experts, N, K), "weights")
    pr = _expert_rows(ctx, rows, torch.bfloat16, K, rows_order, "rows")
    if out is None:
        out = _expert_out(ctx, N, torch.bfloat16, out_order)
    po = _expert_rows(ctx, out, torch.bfloat16, N, out_order, "out")
    _check(load_library().moe_expert_gemm(ctx.handle, pr, rows_order, pw, K, N, ctypes.byref(handle.c), po, out_order,
                                          _stream()), "moe_expert_gemm")
    return out


def moe_expert_gemm_fp8(ctx, rows, row_scales, weights, weight_scales, handle, out=None, rows_order=MOE_ROWS_RECV,
                        out_order=MOE_ROWS_RECV):
    """moe_expert_gemm of E4M3 codes (uint8): rows [rows, K] with fp32 row_scales
    [rows, K/128], weights [E, N, K] with fp32 weight_scales [E, ceil(N/128), K/128]
    -> out bf16 [rows, N]."""
    N, K = _mats_shape(ctx, weights)
    _check_handle(ctx, handle)
    pw = _expert_mats(ctx, weights, torch.uint8, (ctx.cfg.num_experts, N, K), "weights")
    pr = _expert_rows(ctx, rows, torch.uint8, K, rows_order, "rows")
    prs = _expert_rows(ctx, row_scales, torch.float32, K // 128, rows_order, "row_scales")
    pws = _expert_mats(ctx, weight_scales, torch.float32, (ctx.cfg.num_experts, -(-N // 128), K // 128), "weight_scales")
    if out is None:
        out = _expert_out(ctx, N, torch.bfloat16, out_order)
    po = _expert_rows(ctx, out, torch.bfloat16, N, out_order, "out")
    _check(load_library().moe_expert_gemm_fp8(ctx.handle, pr, prs, rows_order, pw, pws, K, N, ctypes.byref(handle.c), po,
                                              out_order, _stream()), "moe_expert_gemm_fp8")
    return out


def moe_expert_gemm_backward_rows(ctx, grad_out, weights, handle, grad_rows=None, out_order=MOE_ROWS_RECV,
                                  rows_order=MOE_ROWS_RECV):
    """Gradient of moe_expert_gemm for its rows: bf16 [rows, K]."""
    N, K = _mats_shape(ctx, weights)
    _check_handle(ctx, handle)
    pw = _expert_mats(ctx, weights, torch.bfloat16, (ctx.cfg.num_experts, N, K), "weights")
    pg = _expert_rows(ctx, grad_out, torch.bfloat16, N, out_order, "grad_out")
    if grad_rows is None:
        grad_rows = _expert_out(ctx, K, torch.bfloat16, rows_order)
    po = _expert_rows(ctx, grad_rows, torch.bfloat16, K, rows_order, "grad_rows")
    _check(load_library().moe_expert_gemm_backward_rows(ctx.handle, pg, out_order, pw, K, N, ctypes.byref(handle.c), po,
                                                        rows_order, _stream()), "moe_expert_gemm_backward_rows")
    return grad_rows


def moe_expert_gemm_backward_weights(ctx, grad_out, rows, handle, grad_weights=None, out_order=MOE_ROWS_RECV,
                                     rows_order=MOE_ROWS_RECV, accumulate=False):
    """Gradient of moe_expert_gemm for its matrices: [E, N, K], bf16 (the
    default) or fp32 as grad_weights is.  accumulate: add to grad_weights."""
    c = ctx.cfg
    if grad_out.dim() != 2 or rows.dim() != 2:
        raise ValueError("grad_out and rows must have two dimensions")
    N, K = grad_out.shape[1], rows.shape[1]
    _int32(N, K)
    _check_handle(ctx, handle)
    pg = _expert_rows(ctx, grad_out, torch.bfloat16, N, out_order, "grad_out")
    pr = _expert_rows(ctx, rows, torch.bfloat16, K, rows_order, "rows")
    if grad_weights is None:
        if accumulate:
            raise ValueError("accumulate needs grad_weights")
        grad_weights = torch.empty((c.num_experts, N, K), dtype=torch.bfloat16, device=rows.device)
    dtype = grad_weights.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("grad_weights must be bfloat16 or float32")
    pw = _expert_mats(ctx, grad_weights, dtype, (c.num_experts, N, K), "grad_weights")
    kind = MOE_GRAD_F32 if dtype is torch.float32 else MOE_GRAD_BF16
    _check(load_library().moe_expert_gemm_backward_weights(ctx.handle, pg, out_order, pr, rows_order, K, N,
                                                           ctypes.byref(handle.c), pw, kind, int(bool(accumulate)),
                                                           _stream()), "moe_expert_gemm_backward_weights")
    return grad_weights


def _gate_up_features(gate_up):
    shape = gate_up.shape
    if len(shape) != 2 or shape[1] % 2:
        raise ValueError("gate_up must be [rows, 2 * features]")
    _int32(shape[1] // 2)
    return shape[1] // 2


def moe_swiglu(ctx, gate_up, handle, out=None, order=MOE_ROWS_RECV):
    """silu(gate) * up of rows bf16 [rows, 2I] (gate first) -> bf16 [rows, I]."""
    features = _gate_up_features(gate_up)
    _check_handle(ctx, handle)
    pg = _expert_rows(ctx, gate_up, torch.bfloat16, 2 * features, order, "gate_up")
    if out is None:
        out = _expert_out(ctx, features, torch.bfloat16, order)
    po = _expert_rows(ctx, out, torch.bfloat16, features, order, "out")
    _check(load_library().moe_swiglu(ctx.handle, pg, features, order, ctypes.byref(handle.c), po, _stream()), "moe_swiglu")
    return out


def moe_swiglu_fp8(ctx, gate_up, handle, out=None, scales=None, order=MOE_ROWS_RECV):
    """moe_swiglu as E4M3 codes (uint8 [rows, I]) and fp32 scales [rows, I/128]."""
    features = _gate_up_features(gate_up)
    _check_handle(ctx, handle)
    pg = _expert_rows(ctx, gate_up, torch.bfloat16, 2 * features, order, "gate_up")
    if out is None:
        out = _expert_out(ctx, features, torch.uint8, order)
    if scales is None:
        scales = _expert_out(ctx, features // 128, torch.float32, order)
    po = _expert_rows(ctx, out, torch.uint8, features, order, "out")
    ps = _expert_rows(ctx, scales, torch.float32, features // 128, order, "scales")
    _check(load_library().moe_swiglu_fp8(ctx.handle, pg, features, order, ctypes.byref(handle.c), po, ps, _stream()),
           "moe_swiglu_fp8")
    return out, scales


def moe_swiglu_backward(ctx, grad_out, gate_up, handle, grad_gate_up=None, order=MOE_ROWS_RECV):
    """Gradient of moe_swiglu: bf16 [rows, 2I] (grad_gate_up may be gate_up)."""
    features = _gate_up_features(gate_up)
    _check_handle(ctx, handle)
    pg = _expert_rows(ctx, gate_up, torch.bfloat16, 2 * features, order, "gate_up")
    pd = _expert_rows(ctx, grad_out, torch.bfloat16, features, order, "grad_out")
    if grad_gate_up is None:
        grad_gate_up = _expert_out(ctx, 2 * features, torch.bfloat16, order)
    po = _expert_rows(ctx, grad_gate_up, torch.bfloat16, 2 * features, order, "grad_gate_up")
    _check(load_library().moe_swiglu_backward(ctx.handle, pd, pg, features, order, ctypes.byref(handle.c), po, _stream()),
           "moe_swiglu_backward")
    return grad_gate_up


# ---------------------------------------------------------------- around the experts
# These calls are made per layer and token, and some of their kernels take a few microseconds: what is right passes one
# test per tensor, sizes are read once, and outputs that a call makes itself are not looked at again.
_BF16, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64


def _bad(ctx, t, dtype, shape, name):
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    if t.get_device() != ctx.device:
        raise ValueError("%s is on %s, the context on cuda:%d" % (name, t.device, ctx.device))
    raise ValueError("%s must be %s, is %s" % (name, tuple(shape), tuple(t.shape)))


def _arg(ctx, t, dtype, shape, name):
    """Pointer of a contiguous tensor of this dtype and shape on the context's device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == ctx.device:
        return t.data_ptr()
    _bad(ctx, t, dtype, shape, name)


def _opt(ctx, t, dtype, shape, name):
    """The same of a tensor that may be left out."""
    return None if t is None else _arg(ctx, t, dtype, shape, name)


def _layer_sizes(ctx):
    """Experts, hidden, slots and the device, as Python has them (fixed per context, so cached)."""
    sizes = ctx.__dict__.get("_sizes")
    if sizes is None:
        c = ctx.cfg
        sizes = ctx.__dict__["_sizes"] = (c.num_experts, c.hidden, c.topk, torch.device("cuda", ctx.device))
    return sizes


def _workspace(ctx, like, t, nbytes):
    """Pointer of at least nbytes bytes, and the tensor that holds them (one that a call made for itself may go when the call
    returns: its memory is used again in the order of the stream)."""
    if nbytes == 0:
        return None, None
    if t is None:
        t = like.new_empty((nbytes + 1) // 2)   # `like` is bf16
    elif not (t.is_cuda and t.is_contiguous() and t.get_device() == ctx.device):
        raise TypeError("workspace must be a contiguous CUDA tensor on cuda:%d" % ctx.device)
    elif t.numel() * t.element_size() < nbytes:
        raise ValueError("workspace holds %d bytes, needs %d" % (t.numel() * t.element_size(), nbytes))
    return t.data_ptr(), t


_LOGIT_TYPES = {torch.float32: MOE_LOGIT_F32, torch.bfloat16: MOE_LOGIT_BF16}


def _logits(ctx, t, E):
    """Tokens, pointer, type and row stride of a router's logits [T, E]."""
    kind = _LOGIT_TYPES.get(t.dtype)
    if kind is None or not t.is_cuda:
        raise TypeError("logits must be a float32 or bfloat16 CUDA tensor")
    if t.get_device() != ctx.device:
        raise ValueError("logits is on %s, the context on cuda:%d" % (t.device, ctx.device))
    shape = t.shape
    if len(shape) == 2 and shape[1] == E:
        _tokens(shape[0])
        if t.is_contiguous():
            return shape[0], t.data_ptr(), kind, E
        stride, columns = t.stride()
        if E == 1 or columns == 1:
            if shape[0] <= 1:
                stride = E
            if stride < E:
                raise ValueError("rows of logits overlap")
            return shape[0], t.data_ptr(), kind, stride
    raise ValueError("logits must be [T, %d], its rows contiguous" % E)


# What these caches keep is found by its sizes and settings.  They take plain numbers alone: a tensor of one element is a number to
# ctypes, but as a key it is itself, whatever it holds by then.
@functools.lru_cache(maxsize=256)
def _router_struct(score, groups, topk_groups, group_top, normalize, scale):
    _int32(score, groups, topk_groups, group_top)
    r = moe_router(score, groups, topk_groups, group_top, normalize, scale)
    return r, ctypes.byref(r)


def _router(score, groups, topk_groups, group_top, normalize, scale):
    return _router_struct(_index(score), _index(groups), _index(topk_groups), _index(group_top), bool(normalize), float(scale))[1]


def moe_route(ctx, logits, score=MOE_SCORE_SOFTMAX, bias=None, groups=1, topk_groups=1, group_top=1, normalize=True, scale=1.0,
              topk_idx=None, topk_weights=None):
    """The k experts of each token and their weights, from logits fp32 or bf16 [T, E] (any row stride): returns
    (topk_idx int64 [T, k], topk_weights fp32 [T, k]).  bias (fp32 [E]) is added to the scores for the choice alone; of
    `groups` groups of neighbouring experts the topk_groups with the largest sums of their group_top best scores stay.  Settings
    are numbers; what a tensor in their place holds is read on the host at each call."""
    E, _, k, device = _layer_sizes(ctx)
    T, p, kind, stride = _logits(ctx, logits, E)
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=_I64, device=device)
        pi = topk_idx.data_ptr()
    else:
        pi = _arg(ctx, topk_idx, _I64, (T, k), "topk_idx")
    if topk_weights is None:
        topk_weights = torch.empty((T, k), dtype=_F32, device=device)
        pw = topk_weights.data_ptr()
    else:
        pw = _arg(ctx, topk_weights, _F32, (T, k), "topk_weights")
    st = load_library().moe_route(ctx.handle, p, kind, stride, T, _router(score, groups, topk_groups, group_top, normalize, scale),
                                  _opt(ctx, bias, _F32, (E,), "bias"), pi, pw, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_route")
    return topk_idx, topk_weights


def moe_route_backward(ctx, grad_weights, logits, topk_idx, score=MOE_SCORE_SOFTMAX, normalize=True, scale=1.0, grad_logits=None):
    """Gradient of moe_route's weights for the logits: fp32 [T, E].  score, normalize and scale as they were there."""
    E, _, k, device = _layer_sizes(ctx)
    T, p, kind, stride = _logits(ctx, logits, E)
    if grad_logits is None:
        grad_logits = torch.empty((T, E), dtype=_F32, device=device)
        pg = grad_logits.data_ptr()
    else:
        pg = _arg(ctx, grad_logits, _F32, (T, E), "grad_logits")
    st = load_library().moe_route_backward(ctx.handle, _arg(ctx, grad_weights, _F32, (T, k), "grad_weights"), p, kind, stride,
                                           _arg(ctx, topk_idx, _I64, (T, k), "topk_idx"), T,
                                           _router(score, 1, 1, 1, normalize, scale), pg, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_route_backward")
    return grad_logits


_OUT_TYPES = {torch.bfloat16: MOE_OUT_BF16, torch.float32: MOE_OUT_F32}


def _linear_sizes(x, weights, act):
    """Rows, in_features, features and the matrix's rows."""
    xs, ws = x.shape, weights.shape
    if len(xs) != 2 or len(ws) != 2:
        raise ValueError("x must be [T, in_features] and weights [M, in_features]")
    M, K = ws
    if act != MOE_ACT_SWIGLU:
        return xs[0], K, M, M
    if M % 2:
        raise ValueError("weights of a gated product have 2 * features rows")
    return xs[0], K, M // 2, M


@functools.lru_cache(maxsize=4096)
def _linear_bytes(T, in_features, features, act):
    _int32(T, in_features, features, act)
    n = ctypes.c_size_t(0)
    _check(load_library().moe_linear_workspace(T, in_features, features, act, ctypes.byref(n)), "moe_linear_workspace")
    return n.value


def moe_linear_workspace(T, in_features, features, act=MOE_ACT_NONE):
    """Bytes that moe_linear works in (by sizes alone, so kept)."""
    return _linear_bytes(_index(T), _index(in_features), _index(features), _index(act))


def moe_linear(ctx, x, weights, bias=None, act=MOE_ACT_NONE, residual=None, out=None, out_dtype=torch.bfloat16, pre=None,
               workspace=None):
    """act(x weights^T + bias) + residual: x bf16 [T, K], weights bf16 [M, K], bias bf16 [M], residual bf16 [T, F] ->
    [T, F], bf16 or fp32 (out's dtype, or out_dtype), F = M, or M / 2 for MOE_ACT_SWIGLU.  pre: bf16 [T, M], receives
    what moe_linear_backward needs.  workspace: moe_linear_workspace bytes."""
    T, K, F, M = _linear_sizes(x, weights, act)
    nbytes = _linear_bytes(T, K, F, _index(act))
    px, pw = _arg(ctx, x, _BF16, (T, K), "x"), _arg(ctx, weights, _BF16, (M, K), "weights")
    if out is None:
        kind = _OUT_TYPES.get(out_dtype)
        if kind is None:
            raise TypeError("out must be bfloat16 or float32")
        out = x.new_empty((T, F)) if kind == MOE_OUT_BF16 else x.new_empty((T, F), dtype=_F32)
        po = out.data_ptr()
    else:
        kind = _OUT_TYPES.get(out.dtype)
        if kind is None:
            raise TypeError("out must be bfloat16 or float32")
        po = _arg(ctx, out, out.dtype, (T, F), "out")
    ps, workspace = _workspace(ctx, x, workspace, nbytes)
    st = load_library().moe_linear(ctx.handle, px, T, pw, K, F, _opt(ctx, bias, _BF16, (M,), "bias"), act,
                                   _opt(ctx, residual, _BF16, (T, F), "residual"), po, kind, _opt(ctx, pre, _BF16, (T, M), "pre"),
                                   ps, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_linear")
    return out


@functools.lru_cache(maxsize=4096)
def _linear_backward_bytes(T, in_features, features, act, out_type, bias):
    _int32(T, in_features, features, act)
    n = ctypes.c_size_t(0)
    _check(load_library().moe_linear_backward_workspace(T, in_features, features, act, out_type, bias, ctypes.byref(n)),
           "moe_linear_backward_workspace")
    return n.value


def moe_linear_backward_workspace(T, in_features, features, act=MOE_ACT_NONE, out_dtype=torch.bfloat16, bias=False):
    """Bytes that moe_linear_backward works in (by sizes and types alone, so kept)."""
    return _linear_backward_bytes(_index(T), _index(in_features), _index(features), _index(act), _OUT_TYPES[out_dtype], bool(bias))


def moe_linear_backward(ctx, grad_out, x, weights, act=MOE_ACT_NONE, pre=None, bias=False, need_x=True, need_weights=True,
                        grad_x=None, grad_weights=None, grad_bias=None, accumulate=False, workspace=None):
    """Gradients of moe_linear: returns (grad_x bf16 [T, K], grad_weights [M, K] bf16 or fp32 as given, grad_bias fp32
    [M]).  grad_out: bf16 or fp32 [T, F]; pre: as moe_linear left it.  grad_bias is None unless bias is true or it is
    given; need_x and need_weights leave out the others.  accumulate: add to grad_weights and grad_bias.  workspace:
    moe_linear_backward_workspace bytes."""
    T, K, F, M = _linear_sizes(x, weights, act)
    dtype = grad_out.dtype
    kind = _OUT_TYPES.get(dtype)
    if kind is None:
        raise TypeError("grad_out must be bfloat16 or float32")
    if accumulate and ((need_weights and grad_weights is None) or (bias and grad_bias is None)):
        raise ValueError("accumulate needs grad_weights and grad_bias")
    nbytes = _linear_backward_bytes(T, K, F, _index(act), kind, bool(bias) or grad_bias is not None)
    pd, px, pw = _arg(ctx, grad_out, dtype, (T, F), "grad_out"), _arg(ctx, x, _BF16, (T, K), "x"), _arg(ctx, weights, _BF16, (M, K), "weights")
    pp = _opt(ctx, pre, _BF16, (T, M), "pre")
    if grad_x is not None:
        pgx = _arg(ctx, grad_x, _BF16, (T, K), "grad_x")
    elif need_x:
        grad_x = torch.empty_like(x)
        pgx = grad_x.data_ptr()
    else:
        pgx = None
    grad_type = MOE_GRAD_BF16
    if grad_weights is not None:
        if grad_weights.dtype is _F32:
            grad_type = MOE_GRAD_F32
        elif grad_weights.dtype is not _BF16:
            raise TypeError("grad_weights must be bfloat16 or float32")
        pgw = _arg(ctx, grad_weights, grad_weights.dtype, (M, K), "grad_weights")
    elif need_weights:
        grad_weights = torch.empty_like(weights)
        pgw = grad_weights.data_ptr()
    else:
        pgw = None
    if grad_bias is not None:
        pgb = _arg(ctx, grad_bias, _F32, (M,), "grad_bias")
    elif bias:
        grad_bias = x.new_empty(M, dtype=_F32)
        pgb = grad_bias.data_ptr()
    else:
        pgb = None
    ps, workspace = _workspace(ctx, x, workspace, nbytes)
    st = load_library().moe_linear_backward(ctx.handle, pd, kind, T, px, pw, K, F, act, pp, pgx, pgw, grad_type, int(bool(accumulate)),
                                            pgb, ps, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_linear_backward")
    return grad_x, grad_weights, grad_bias


def _layer_args(ctx, x, topk_idx, topk_weights, w1, w2, dtype, residual, out, workspace):
    E, H, k, _ = _layer_sizes(ctx)
    xs, ws = x.shape, w2.shape
    if len(xs) != 2 or len(ws) != 3:
        raise ValueError("x must be [T, %d] and w2 [%d, %d, features]" % (H, E, H))
    T, I = _tokens(xs[0]), ws[2]
    if I > _INT_MAX:
        _int32(I)
    px = _arg(ctx, x, _BF16, (T, H), "x")
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    else:
        po = _arg(ctx, out, _BF16, (T, H), "out")
    ps, workspace = _workspace(ctx, x, workspace, T * k * I * 2)
    return (T, I, out, workspace, px, _arg(ctx, topk_idx, _I64, (T, k), "topk_idx"), _arg(ctx, topk_weights, _F32, (T, k), "topk_weights"),
            _arg(ctx, w1, dtype, (E, 2 * I, H), "w1"), _arg(ctx, w2, dtype, (E, H, I), "w2"), _opt(ctx, residual, _BF16, (T, H), "residual"),
            po, ps)


def moe_layer(ctx, x, topk_idx, topk_weights, w1, w2, residual=None, out=None, workspace=None):
    """The experts of a few tokens (T * k at most MOE_LAYER_MAX_ROWS; the faster way up to about 16 tokens, from about 32 on
    moe_dispatch, the expert products and moe_combine are) in one call: x bf16 [T, H], topk_idx int64 and
    topk_weights fp32 [T, k], w1 bf16 [E, 2I, H] (gates first), w2 bf16 [E, H, I], residual bf16 [T, H] -> bf16 [T, H].
    workspace: at least T * k * I * 2 bytes."""
    T, I, out, workspace, px, pi, pw, p1, p2, pr, po, ps = _layer_args(ctx, x, topk_idx, topk_weights, w1, w2, _BF16, residual, out, workspace)
    st = load_library().moe_layer(ctx.handle, px, pi, pw, T, p1, p2, I, pr, po, ps, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_layer")
    return out


def moe_layer_fp8(ctx, x, topk_idx, topk_weights, w1, w1_scales, w2, w2_scales, residual=None, out=None, workspace=None):
    """moe_layer with matrices of E4M3 codes (uint8) and fp32 scales of 128 x 128 blocks, w1_scales [E, 2I/128, H/128]
    and w2_scales [E, H/128, I/128]."""
    T, I, out, workspace, px, pi, pw, p1, p2, pr, po, ps = _layer_args(ctx, x, topk_idx, topk_weights, w1, w2, torch.uint8, residual, out,
                                                                       workspace)
    E, H, _, _ = _layer_sizes(ctx)
    s1 = _arg(ctx, w1_scales, _F32, (E, 2 * I // 128, H // 128), "w1_scales")
    s2 = _arg(ctx, w2_scales, _F32, (E, H // 128, I // 128), "w2_scales")
    st = load_library().moe_layer_fp8(ctx.handle, px, pi, pw, T, p1, s1, p2, s2, I, pr, po, ps, _stream())
    if st != MOE_OK:
        raise MoeError(st, "moe_layer_fp8")
    return out


# ---------------------------------------------------------------- prepared calls
# For tight host loops (decode steps): the arguments of a call are checked and
# marshalled once, and the returned callable only makes the C call, on the
# stream that was current when it was prepared.  The tensors must stay alive
# and keep their storage while the callable is used.
def prepare_dispatch(ctx, x, topk_idx, reuse_layout, bufs, handle, stream=None):
    c = ctx.cfg
    _as_dev(x, torch.bfloat16, "x")
    _as_dev(topk_idx, torch.int64, "topk_idx")
    T = _tokens(x.shape[0])
    if x.dim() != 2 or x.shape[1] != c.hidden or tuple(topk_idx.shape) != (T, c.topk):
        raise ValueError("x must be [T, %d] and topk_idx [T, %d]" % (c.hidden, c.topk))
    _check_bufs(ctx, bufs)
    _check_handle(ctx, handle)
    f = load_library().moe_dispatch
    args = (ctx.handle, _ptr(x), _ptr(topk_idx), ctypes.c_int32(T), ctypes.c_int32(int(bool(reuse_layout))),
            ctypes.byref(bufs.c), ctypes.byref(handle.c), _stream(stream))

    def call():
        st = f(*args)
        if st != MOE_OK:
            raise MoeError(st, "moe_dispatch")
    return call


def prepare_combine(ctx, expert_out, topk_weights, handle, out, num_tokens, stream=None):
    """num_tokens: the token count of the dispatch whose handle is combined
    (checked against the handle at every call)."""
    c = ctx.cfg
    _as_dev(expert_out, torch.bfloat16, "expert_out")
    _as_dev(topk_weights, torch.float32, "topk_weights")
    _as_dev(out, torch.bfloat16, "out")
    if tuple(topk_weights.shape) != (num_tokens, c.topk) or out.numel() < num_tokens * c.hidden:
        raise ValueError("topk_weights must be [%d, %d] and out hold [%d, %d]" % (num_tokens, c.topk, num_tokens,
                                                                                 c.hidden))
    if expert_out.numel() * 2 < ctx.hint(MOE_BUF_EXPERT_OUT):
        raise ValueError("expert_out smaller than MOE_BUF_EXPERT_OUT")
    f = load_library().moe_combine
    hc = handle.c
    args = (ctx.handle, _ptr(expert_out), _ptr(topk_weights), ctypes.byref(hc), _ptr(out), _stream(stream))

    def call():
        if hc.num_tokens != num_tokens:
            raise ValueError("handle holds %d tokens, prepared for %d" % (hc.num_tokens, num_tokens))
        st = f(*args)
        if st != MOE_OK:
            raise MoeError(st, "moe_combine")
    return call


class StaticConfig:
    """A configuration without a context (for moe_dispatch_noalloc): sizes
    for Handle and DispatchBuffers on the current device, nothing allocated by
    the library."""

    def __init__(self, cfg):
        self.cfg = cfg
        self.device = torch.cuda.current_device()
        self._fit_token = object()

    def hint(self, kind):
        cache = self.__dict__.setdefault("_hints", {})
        if kind not in cache:
            cache[kind] = moe_size_hint(self.cfg, kind)
        return cache[kind]


def moe_dispatch_noalloc(scfg, x, topk_idx, bufs, handle, error_word=None):
    """moe_dispatch without a context or any allocation: the library's static
    per-GPU scratch holds the layout.  scfg: a StaticConfig (or a Context, for
    its configuration); bufs and handle sized for it.  error_word: optional
    int32/uint32 device tensor of one element that collects moe_poll_error's
    bits.  Returns (bufs, handle)."""
    c = scfg.cfg
    _as_dev(x, torch.bfloat16, "x")
    _as_dev(topk_idx, torch.int64, "topk_idx")
    T = _tokens(x.shape[0])
    if x.dim() != 2 or x.shape[1] != c.hidden or tuple(topk_idx.shape) != (T, c.topk):
        raise ValueError("x must be [T, %d] and topk_idx [T, %d]" % (c.hidden, c.topk))
    _check_bufs(scfg, bufs)
    _check_handle(scfg, handle)
    if error_word is not None and not (error_word.is_cuda and error_word.element_size() == 4):
        raise TypeError("error_word must be a 4-byte CUDA tensor")
    _check(load_library().moe_dispatch_noalloc(ctypes.byref(c), _ptr(x), _ptr(topk_idx), T, ctypes.byref(bufs.c),
                                               ctypes.byref(handle.c), _ptr(error_word), _stream()),
           "moe_dispatch_noalloc")
    return bufs, handle


def moe_poll_error(ctx):
    """Synchronizes the current stream; returns (status, raw flags) and clears them."""
    flags = ctypes.c_uint32(0)
    st = load_library().moe_poll_error(ctx.handle, _stream(), ctypes.byref(flags))
    if st not in _POLL_STATUSES:
        raise MoeError(st, "moe_poll_error")
    return st, flags.value
