"""ctypes binding of libmoe.so (C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  The functions keep the C names (moe_init, moe_route,
moe_forward, moe_forward_host, moe_check, moe_set_wait_limit, moe_free,
moe_status_string, moe_selftest_wait_timeout) and take torch tensors where
the C functions take pointers; a non-zero status raises MoeError.
``MoeLayer`` bundles a handle with the weight tensors it borrows.

The library must have been built (``__graft_entry__.build()`` or
``python -m expert_routed_ffn_gemm_gb300.build``); loading raises otherwise.
There is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_TOO_MANY_TOKENS = 2
MOE_ERR_UNSUPPORTED = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE = 5
MOE_ERR_NO_DEVICE = 6

EXPORTED = ("moe_init", "moe_route", "moe_forward", "moe_forward_host", "moe_check", "moe_set_wait_limit",
            "moe_profile_enable", "moe_profile_read", "moe_free", "moe_status_string",
            "moe_selftest_wait_timeout", "moe_dispatch_noalloc", "moe_route_ex", "moe_forward_ex",
            "moe_route_stats", "moe_last_kernel_count", "moe_init_fp8", "moe_quantize_fp8", "moe_ep_init",
            "moe_ep_dispatch", "moe_ep_experts", "moe_ep_combine", "moe_mx4_quantize", "moe_mx4_gather", "moe_mx4_init",
            "moe_mx4_matmul", "moe_mx4_check", "moe_mx4_set_wait_limit", "moe_mx4_free", "moe_norm_residual",
            "moe_norm_residual_workspace", "moe_norm_residual_backward")
PROFILE_STAGES = ("routing", "dispatch", "gather", "gate_up_gemm", "down_gemm", "combine")


# data types and gate kinds of include/moe.h (moe_dtype, moe_gate_kind)
MOE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MOE_GATE_NONE, MOE_GATE_FEATURE, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {moe_status_string(status)} (status {status})")


class moe_config(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("ffn_width", ctypes.c_int), ("has_shared", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("out_fp32", ctypes.c_int)]


class moe_weights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p)]


class moe_weights_fp8(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("s_gate_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


class moe_ep_config(ctypes.Structure):
    _fields_ = [("layer", moe_config), ("ep_size", ctypes.c_int), ("ep_rank", ctypes.c_int),
                ("max_recv_rows", ctypes.c_int)]


class moe_call_options(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int), ("renormalize", ctypes.c_int)]


class moe_mx4_config(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int), ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("gated", ctypes.c_int)]


class moe_norm_config(ctypes.Structure):
    _fields_ = [("stream_dtype", ctypes.c_int), ("block_dtype", ctypes.c_int), ("gate_kind", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("sigmoid", ctypes.c_int), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float)]


def _opts(top_k, renormalize):
    if top_k is None and not renormalize:
        return None
    return ctypes.byref(moe_call_options(int(top_k or 0), int(bool(renormalize))))


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    """libmoe.so, or libmoe_debug.so (the build with the kernels' bounds
    checks) when MOE_LIBRARY=debug is set in the environment."""
    return _build.DEBUG_LIB_PATH if os.environ.get("MOE_LIBRARY") == "debug" else _build.LIB_PATH


def load():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first (__graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, i, ull = ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong
        lib.moe_init.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights), ctypes.POINTER(vp)]
        lib.moe_init_fp8.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights_fp8),
                                     ctypes.POINTER(vp)]
        lib.moe_quantize_fp8.argtypes = [vp, ctypes.c_longlong, i, vp, vp, vp]
        lib.moe_ep_init.argtypes = [ctypes.POINTER(moe_ep_config), ctypes.POINTER(moe_weights), ctypes.POINTER(vp)]
        lib.moe_ep_dispatch.argtypes = [vp, vp, i, vp, vp, vp, ctypes.POINTER(ctypes.c_int), vp]
        lib.moe_ep_experts.argtypes = [vp, vp, vp, vp, i, vp, vp, ctypes.POINTER(ctypes.c_int), vp]
        lib.moe_ep_combine.argtypes = [vp, vp, vp, vp, vp]
        lib.moe_route.argtypes = [vp, vp, i, vp, vp, vp, vp, vp, vp]
        lib.moe_forward.argtypes = [vp, vp, i, vp, vp]
        lib.moe_forward_host.argtypes = [vp, vp, i, vp, vp]
        lib.moe_check.argtypes = [vp, vp]
        lib.moe_last_kernel_count.argtypes = [vp]
        lib.moe_set_wait_limit.argtypes = [vp, ull]
        lib.moe_profile_enable.argtypes = [vp, i]
        lib.moe_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)]
        lib.moe_free.argtypes = [vp]
        lib.moe_status_string.argtypes = [i]
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_selftest_wait_timeout.argtypes = [ull, vp]
        lib.moe_dispatch_noalloc.argtypes = [vp, i, i, i, i, vp, vp, vp]
        lib.moe_route_ex.argtypes = [vp, vp, i, vp, vp, vp, vp, vp, vp, vp]
        lib.moe_forward_ex.argtypes = [vp, vp, i, vp, vp, vp]
        lib.moe_route_stats.argtypes = [vp, vp, i, i, vp, vp, vp, vp, vp]
        ll, norm = ctypes.c_longlong, ctypes.POINTER(moe_norm_config)
        lib.moe_mx4_quantize.argtypes = [vp, i, ll, i, vp, i, ll, vp, vp, vp, vp]
        lib.moe_mx4_gather.argtypes = [vp, vp, ll, i, vp, i, ll, vp, vp, vp]
        lib.moe_mx4_init.argtypes = [ctypes.POINTER(moe_mx4_config), vp, vp, ctypes.POINTER(vp)]
        lib.moe_mx4_matmul.argtypes = [vp, vp, vp, ll, vp, vp, vp, vp, i, ll, vp]
        lib.moe_mx4_check.argtypes = [vp, vp]
        lib.moe_mx4_set_wait_limit.argtypes = [vp, ull]
        lib.moe_mx4_free.argtypes = [vp]
        lib.moe_norm_residual.argtypes = [norm, i, i, vp, vp, i, vp, vp, vp, vp, vp, vp]
        lib.moe_norm_residual_workspace.argtypes = [i, i]
        lib.moe_norm_residual_backward.argtypes = [norm, i, i] + [vp] * 4 + [i] + [vp] * 9 + [ll, vp]
        for name in EXPORTED:
            if name != "moe_status_string":
                getattr(lib, name).restype = ctypes.c_int
        lib.moe_norm_residual_workspace.restype = ll
        _lib = lib
        return lib


def moe_status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _call_stream(t: torch.Tensor, stream):
    """(raw stream, context to allocate in or None) of a call on t's device.
    What a call allocates belongs to its stream, so that the caching allocator
    reuses a freed block in that stream's order.  The common case, the current
    stream, is looked up without a stream object (3 us on a Grace core)."""
    if not t.is_cuda:
        raise ValueError("expected device tensors")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device()), None
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, t.device) if raw else torch.cuda.default_stream(t.device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _empty(shape, dtype, device, context=None):
    """torch.empty, on the stream of a context from _call_stream."""
    if context is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with context:
        return torch.empty(shape, dtype=dtype, device=device)


def moe_init(cfg: moe_config, w_router: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor) -> int:
    w = moe_weights(_ptr(w_router), _ptr(w_gate_up), _ptr(w_down))
    h = ctypes.c_void_p()
    _check(load().moe_init(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)), "moe_init")
    return h.value


def moe_init_fp8(cfg: moe_config, w_router, q_gate_up, s_gate_up, q_down, s_down) -> int:
    w = moe_weights_fp8(_ptr(w_router), _ptr(q_gate_up), _ptr(s_gate_up), _ptr(q_down), _ptr(s_down))
    h = ctypes.c_void_p()
    _check(load().moe_init_fp8(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)), "moe_init_fp8")
    return h.value


def moe_quantize_fp8(w: torch.Tensor, stream=None):
    """Per-row E4M3 codes (uint8, same shape) and fp32 scales (shape[:-1]) of a
    bf16 device tensor, computed on the device (see include/moe.h)."""
    if w.dtype != torch.bfloat16:
        raise TypeError("moe_quantize_fp8 takes bf16 weights")
    cols = w.shape[-1]
    rows = w.numel() // cols
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    _check(load().moe_quantize_fp8(_ptr(w), rows, cols, _ptr(q), _ptr(s), _stream(stream)), "moe_quantize_fp8")
    return q, s


def moe_ep_init(cfg: moe_ep_config, w_router, w_gate_up_local, w_down_local) -> int:
    """Expert-parallel handle (moe_weights layout: the router over all experts,
    this rank's experts then the shared expert)."""
    w = moe_weights(_ptr(w_router), _ptr(w_gate_up_local), _ptr(w_down_local))
    h = ctypes.c_void_p()
    _check(load().moe_ep_init(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)), "moe_ep_init")
    return h.value


def moe_ep_dispatch(h: int, x, T: int, send_rows, send_w, send_counts, ep_size: int, stream=None) -> list[int]:
    rows = (ctypes.c_int * ep_size)()
    _check(load().moe_ep_dispatch(h, _ptr(x), int(T), _ptr(send_rows), _ptr(send_w), _ptr(send_counts), rows,
                                  _stream(stream)), "moe_ep_dispatch")
    return list(rows)


def moe_ep_experts(h: int, recv_rows, recv_counts, recv_w, n_recv: int, out_rows, out_exp, ep_size: int,
                   stream=None) -> list[int]:
    chunks = (ctypes.c_int * ep_size)()
    _check(load().moe_ep_experts(h, _ptr(recv_rows), _ptr(recv_counts), _ptr(recv_w), int(n_recv), _ptr(out_rows),
                                 _ptr(out_exp), chunks, _stream(stream)), "moe_ep_experts")
    return list(chunks)


def moe_ep_combine(h: int, ret_rows, ret_exp, y, stream=None) -> None:
    _check(load().moe_ep_combine(h, _ptr(ret_rows), _ptr(ret_exp), _ptr(y), _stream(stream)), "moe_ep_combine")


def moe_route(h: int, x, T: int, idx, prob, perm, offsets, gap=None, stream=None) -> None:
    _check(load().moe_route(h, _ptr(x), int(T), _ptr(idx), _ptr(prob), _ptr(perm), _ptr(offsets), _ptr(gap),
                            _stream(stream)), "moe_route")


def moe_forward(h: int, x, T: int, y, stream=None) -> None:
    _check(load().moe_forward(h, _ptr(x), int(T), _ptr(y), _stream(stream)), "moe_forward")


def moe_route_ex(h: int, x, T: int, top_k, renormalize, idx, prob, perm, offsets, gap=None, stream=None) -> None:
    _check(load().moe_route_ex(h, _ptr(x), int(T), _opts(top_k, renormalize), _ptr(idx), _ptr(prob), _ptr(perm),
                               _ptr(offsets), _ptr(gap), _stream(stream)), "moe_route_ex")


def moe_forward_ex(h: int, x, T: int, top_k, renormalize, y, stream=None) -> None:
    _check(load().moe_forward_ex(h, _ptr(x), int(T), _opts(top_k, renormalize), _ptr(y), _stream(stream)),
           "moe_forward_ex")


def moe_route_stats(h: int, x, T: int, n_groups: int, counts, group_f, group_p, summary, stream=None) -> None:
    _check(load().moe_route_stats(h, _ptr(x), int(T), int(n_groups), _ptr(counts), _ptr(group_f), _ptr(group_p),
                                  _ptr(summary), _stream(stream)), "moe_route_stats")


def moe_forward_host(h: int, x_host: torch.Tensor, T: int, y_host: torch.Tensor, stream=None) -> None:
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("moe_forward_host takes host tensors")
    _check(load().moe_forward_host(h, _ptr(x_host), int(T), _ptr(y_host), _stream(stream)), "moe_forward_host")


def moe_last_kernel_count(h: int) -> int:
    """Kernels the last forward call on the handle enqueued (-1: bad handle)."""
    return int(load().moe_last_kernel_count(h))


def moe_check(h: int, stream=None) -> int:
    """Returns the status (does not raise): MOE_OK or MOE_ERR_DEVICE/CUDA."""
    return int(load().moe_check(h, _stream(stream)))


def moe_set_wait_limit(h: int, ns: int) -> None:
    _check(load().moe_set_wait_limit(h, int(ns)), "moe_set_wait_limit")


def moe_profile_enable(h: int, enable: bool) -> None:
    _check(load().moe_profile_enable(h, int(bool(enable))), "moe_profile_enable")


def moe_profile_read(h: int):
    """Returns ({stage: total ms}, number of recorded calls) and clears the record."""
    ms = (ctypes.c_float * len(PROFILE_STAGES))()
    n = ctypes.c_int()
    _check(load().moe_profile_read(h, ms, ctypes.byref(n)), "moe_profile_read")
    return dict(zip(PROFILE_STAGES, [float(v) for v in ms])), int(n.value)


def moe_free(h: int) -> None:
    _check(load().moe_free(h), "moe_free")


def moe_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(load().moe_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def moe_dispatch_noalloc(idx, T: int, n_experts: int, top_k: int, has_shared: bool, offsets, perm,
                         stream=None) -> None:
    """Dispatch order from existing routing without any device allocation
    (for callers that must not call cudaMalloc); see include/moe.h."""
    _check(load().moe_dispatch_noalloc(_ptr(idx), int(T), int(n_experts), int(top_k), int(bool(has_shared)),
                                       _ptr(offsets), _ptr(perm), _stream(stream)), "moe_dispatch_noalloc")


def mx4_code_bytes(cols: int) -> int:
    """Bytes of E2M1 codes of a matrix row of `cols` columns."""
    return (cols + 31) // 32 * 16


def mx4_scale_bytes(cols: int) -> int:
    """Scale bytes of a matrix row of `cols` columns, padding included."""
    return (cols + 127) // 128 * 4


def _mx4_source(x, src, src_div):
    """(rows, source rows, columns, type code) of a quantiser call, its arguments checked."""
    if x.dim() != 2:
        raise ValueError("expected a matrix [rows, cols]")
    dtype = MOE_DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError("expected bf16, fp16 or fp32 elements")
    n_src, cols = x.shape
    if src is None:
        return n_src, n_src, cols, dtype
    if src.dtype != torch.int32 or src.dim() != 1:
        raise TypeError("src must be int32 [rows]")
    if src_div < 1:
        raise ValueError("src_div must be at least 1")
    return src.shape[0], n_src, cols, dtype


# Rows gathered several times from at least this many elements are quantised
# once and copied (8192 tokens of 4096 columns to 9 rows each: 141 us by
# quantising every copy, 44 us so); below, one launch is quicker than two.
_MX4_GATHER_ELEMENTS = 1 << 20


def moe_mx4_quantize(x: torch.Tensor, src: torch.Tensor | None = None, src_div: int = 1, stream=None):
    """MX 4-bit codes and scale bytes (uint8 [rows, ...]) of a device matrix;
    with src int32 [rows], of the rows x[src // src_div] (see include/moe.h)."""
    rows, n_src, cols, dtype = _mx4_source(x, src, src_div)
    raw, context = _call_stream(x, stream)
    lib, dev = load(), x.device
    codes = _empty((rows, (cols + 31) // 32 * 16), torch.uint8, dev, context)
    scales = _empty((rows, (cols + 127) // 128 * 4), torch.uint8, dev, context)
    if src is not None and rows >= 2 * n_src and n_src * cols >= _MX4_GATHER_ELEMENTS:
        once, once_scales = moe_mx4_quantize(x, stream=stream)
        _check(lib.moe_mx4_gather(once.data_ptr(), once_scales.data_ptr(), n_src, cols, _ptr(src), src_div, rows,
                                  codes.data_ptr(), scales.data_ptr(), raw), "moe_mx4_gather")
        return codes, scales
    status = lib.moe_mx4_quantize(_ptr(x), dtype, n_src, cols, _ptr(src), src_div, rows, codes.data_ptr(),
                                  scales.data_ptr(), None, raw)
    if status:
        raise MoeError(status, "moe_mx4_quantize")
    return codes, scales


def moe_mx4_gather(codes: torch.Tensor, scales: torch.Tensor, cols: int, src: torch.Tensor, src_div: int = 1,
                   stream=None):
    """Rows src // src_div of a quantised matrix with cols columns."""
    n_src = codes.shape[0]
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or src.dtype != torch.int32 or src.dim() != 1:
        raise TypeError("codes and scales must be uint8, src int32 [rows]")
    if codes.shape != (n_src, mx4_code_bytes(cols)) or scales.shape != (n_src, mx4_scale_bytes(cols)):
        raise ValueError("codes and scales must be [rows, bytes] of rows with cols columns")
    raw, context = _call_stream(codes, stream)
    rows = src.shape[0]
    out = _empty((rows, codes.shape[1]), torch.uint8, codes.device, context)
    out_scales = _empty((rows, scales.shape[1]), torch.uint8, codes.device, context)
    _check(load().moe_mx4_gather(_ptr(codes), _ptr(scales), n_src, cols, _ptr(src), src_div, rows, _ptr(out),
                                 _ptr(out_scales), raw), "moe_mx4_gather")
    return out, out_scales


def moe_mx4_round(x: torch.Tensor, src: torch.Tensor | None = None, src_div: int = 1, stream=None) -> torch.Tensor:
    """The values that moe_mx4_quantize's codes stand for, in x's type."""
    rows, n_src, cols, dtype = _mx4_source(x, src, src_div)
    raw, context = _call_stream(x, stream)
    values = _empty((rows, cols), x.dtype, x.device, context)
    _check(load().moe_mx4_quantize(_ptr(x), dtype, n_src, cols, _ptr(src), src_div, rows, None, None,
                                   values.data_ptr(), raw), "moe_mx4_quantize")
    return values


class Mx4Experts:
    """4-bit weights of a set of experts and the handle that borrows them.

    codes uint8 [groups, rows, mx4_code_bytes(cols)], scales uint8 [groups,
    rows, mx4_scale_bytes(cols)], as moe_mx4_quantize writes them for the
    matrix [groups * rows, cols].  gated: rows 0..F-1 are the gate projection,
    rows F..2F-1 the up projection.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, gated: bool = False):
        self.handle = None
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.dim() != 3 or tuple(scales.shape) != (*codes.shape[:2], mx4_scale_bytes(cols)) or \
                codes.shape[2] != mx4_code_bytes(cols):
            raise ValueError("codes and scales must be [groups, rows, bytes] of matrices with cols columns")
        self.groups, self.rows = codes.shape[0], codes.shape[1]
        self.cols, self.gated = cols, bool(gated)
        self.out_cols = self.rows // 2 if gated else self.rows
        self.code_bytes, self.scale_bytes = codes.shape[2], scales.shape[2]
        self.codes = codes  # borrowed by the handle
        cfg = moe_mx4_config(self.groups, self.rows, cols, int(self.gated))
        h = ctypes.c_void_p()
        with torch.cuda.device(codes.device):
            _check(load().moe_mx4_init(ctypes.byref(cfg), _ptr(codes), _ptr(scales), ctypes.byref(h)), "moe_mx4_init")
        self.handle = h.value

    @classmethod
    def quantize(cls, w: torch.Tensor, gated: bool = False, stream=None) -> "Mx4Experts":
        """From weights [groups, rows, cols] in bf16, fp16 or fp32."""
        groups, rows, cols = w.shape
        codes, scales = moe_mx4_quantize(w.reshape(groups * rows, cols), stream=stream)
        return cls(codes.view(groups, rows, -1), scales.view(groups, rows, -1), cols, gated)

    def matmul(self, codes: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
               out_rows: torch.Tensor | None = None, row_scale: torch.Tensor | None = None, n_out: int | None = None,
               dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Products of quantised token rows, grouped by offsets int32 [groups + 1];
        with out_rows int32 [rows], row r goes to row out_rows[r] of the n_out
        (default: as many as token rows) rows of the result, times row_scale
        fp32 [n_out] of that row.  Rows that no product reaches stay as `out`
        has them; without `out` they hold whatever that memory held before."""
        rows = codes.shape[0]
        n_out = rows if n_out is None else int(n_out)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.shape != (rows, self.code_bytes) or scales.shape != (rows, self.scale_bytes):
            raise ValueError("codes and scales must be [rows, bytes] of rows with the weights' columns")
        if offsets.dtype != torch.int32 or offsets.numel() != self.groups + 1:
            raise ValueError("offsets must be int32 [groups + 1]")
        if out_rows is not None and (out_rows.dtype != torch.int32 or out_rows.numel() != rows):
            raise ValueError("out_rows must be int32 [rows]")
        if row_scale is not None and (row_scale.dtype != torch.float32 or row_scale.numel() != n_out):
            raise ValueError("row_scale must be fp32 [n_out]")
        raw, context = _call_stream(codes, stream)
        if out is None:
            if dtype not in MOE_DTYPES:
                raise TypeError("results are bf16, fp16 or fp32")
            out = _empty((n_out, self.out_cols), dtype, codes.device, context)
        elif out.dtype not in MOE_DTYPES or out.shape != (n_out, self.out_cols):
            raise ValueError("out must be [n_out, out_cols] in bf16, fp16 or fp32")
        status = load().moe_mx4_matmul(self.handle, _ptr(codes), _ptr(scales), rows, _ptr(offsets), _ptr(out_rows),
                                       _ptr(row_scale), _ptr(out), MOE_DTYPES[out.dtype], n_out, raw)
        if status:
            raise MoeError(status, "moe_mx4_matmul")
        return out

    def check(self, stream=None) -> int:
        """Returns the status (does not raise): MOE_OK or MOE_ERR_DEVICE/CUDA."""
        return int(load().moe_mx4_check(self.handle, _stream(stream)))

    def set_wait_limit(self, ns: int) -> None:
        _check(load().moe_mx4_set_wait_limit(self.handle, int(ns)), "moe_mx4_set_wait_limit")

    def close(self) -> None:
        if getattr(self, "handle", None):
            load().moe_mx4_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


@functools.lru_cache(maxsize=64)
def _norm_config(stream_dtype, block_dtype, kind, gate_dtype, sigmoid, alpha, eps):
    return moe_norm_config(MOE_DTYPES[stream_dtype], MOE_DTYPES[block_dtype], kind, MOE_DTYPES.get(gate_dtype, 0),
                           int(sigmoid), alpha, eps)


def _norm_parts(x, y, block_dtype, w_post, gate, w_pre, alpha, eps, sigmoid):
    """(config, T, d, terms, gate kind) of a norm call on stream rows x, its shapes and types checked."""
    if x.dim() != 2:
        raise ValueError("expected token rows [T, d]")
    T, d = x.shape
    if x.dtype not in MOE_DTYPES or block_dtype not in MOE_DTYPES:
        raise TypeError("expected bf16, fp16 or fp32 elements")
    terms = 0
    if y is not None:
        shape = y.shape
        if len(shape) not in (2, 3) or shape[0] != T or shape[-1] != d:
            raise ValueError("y must be [T, d] or [T, terms, d]")
        terms = shape[1] if len(shape) == 3 else 1
    for w in (w_post, w_pre):
        if w is not None and (w.dtype != torch.float32 or w.shape != (d,)):
            raise ValueError("norm weights must be fp32 [d]")
    kind, gate_dtype = MOE_GATE_NONE, None
    if gate is not None:
        gate_dtype, shape = gate.dtype, gate.shape
        if gate_dtype not in MOE_DTYPES:
            raise TypeError("the gate must be bf16, fp16 or fp32")
        if shape == (d,):
            kind = MOE_GATE_FEATURE
        elif shape == (T, 1):  # with one column the same as a gate for each element
            kind = MOE_GATE_TOKEN
        elif shape == (T, d):
            kind = MOE_GATE_FULL
        else:
            raise ValueError("the gate must be [d], [T, 1] or [T, d]")
    cfg = _norm_config(x.dtype, block_dtype, kind, gate_dtype, bool(sigmoid), float(alpha), float(eps))
    return cfg, T, d, terms, kind


def moe_norm_residual(x: torch.Tensor, y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                      gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None, alpha: float = 1.0,
                      eps: float = 1e-6, sigmoid: bool = False, block_dtype: torch.dtype | None = None, stream=None):
    """(out, n): out = x + alpha * gate * norm(sum of y's terms; w_post) and
    n = norm(out; w_pre) (see include/moe.h).  x [T, d]; y [T, d] or [T, terms,
    d]; gate [d], [T, 1] or [T, d].  Without y, out is x itself; without
    w_pre, n is None.  block_dtype: the type of n where there is no y to take
    it from (default: x's)."""
    bt = y.dtype if y is not None else (block_dtype or x.dtype)
    cfg, T, d, terms, _ = _norm_parts(x, y, bt, w_post, gate, w_pre, alpha, eps, sigmoid)
    raw, context = _call_stream(x, stream)
    out = _empty((T, d), x.dtype, x.device, context) if y is not None else None
    n = _empty((T, d), bt, x.device, context) if w_pre is not None else None
    status = load().moe_norm_residual(cfg, T, d, _ptr(x), _ptr(y), terms, _ptr(w_post), _ptr(gate), _ptr(w_pre),
                                      None if out is None else out.data_ptr(), None if n is None else n.data_ptr(), raw)
    if status:
        raise MoeError(status, "moe_norm_residual")
    return (x if out is None else out), n


def moe_norm_residual_backward(d_out: torch.Tensor | None, d_n: torch.Tensor | None, out: torch.Tensor,
                               y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                               gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                               alpha: float = 1.0, eps: float = 1e-6, sigmoid: bool = False, stream=None) -> dict:
    """Gradients of moe_norm_residual's results: {"x", "y", "w_post", "gate",
    "w_pre"}, those of the inputs given.  "y" [T, d] is the gradient of each
    term; the weights' and a [d] or [T, 1] gate's are fp32."""
    bt = y.dtype if y is not None else (d_n.dtype if d_n is not None else out.dtype)
    cfg, T, d, terms, kind = _norm_parts(out, y, bt, w_post, gate, w_pre, alpha, eps, sigmoid)
    for g, dtype in ((d_out, out.dtype), (d_n, bt)):
        if g is not None and (g.dtype != dtype or g.shape != (T, d)):
            raise ValueError("gradients must have the shape and type of what they belong to")
    raw, context = _call_stream(out, stream)
    dev, lib = out.device, load()
    need = _norm_workspace(T, d, out.get_device())
    ws = _empty((need,), torch.uint8, dev, context)
    grads = {"x": _empty((T, d), out.dtype, dev, context)}
    if y is not None:
        grads["y"] = _empty((T, d), bt, dev, context)
    if w_post is not None:
        grads["w_post"] = _empty((d,), torch.float32, dev, context)
    if gate is not None:
        grads["gate"] = _empty(gate.shape, gate.dtype if kind == MOE_GATE_FULL else torch.float32, dev, context)
    if w_pre is not None:
        grads["w_pre"] = _empty((d,), torch.float32, dev, context)
    g = grads.get
    status = lib.moe_norm_residual_backward(cfg, T, d, _ptr(d_out), _ptr(d_n), _ptr(out), _ptr(y), terms, _ptr(w_post),
                                            _ptr(gate), _ptr(w_pre), _ptr(g("x")), _ptr(g("y")), _ptr(g("w_post")),
                                            _ptr(g("gate")), _ptr(g("w_pre")), ws.data_ptr(), need, raw)
    if status:
        raise MoeError(status, "moe_norm_residual_backward")
    return grads


@functools.lru_cache(maxsize=1024)
def _norm_workspace(T: int, d: int, device: int) -> int:
    """Bytes of workspace of a backward call on a device (by its SM count)."""
    with torch.cuda.device(device):
        need = load().moe_norm_residual_workspace(T, d)
    if need < 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_norm_residual_workspace")
    return max(16, need)


class MoeLayer:
    """A handle plus the device weight tensors it borrows.

    w_router fp32 [E, d]; w_gate_up bf16 [E+1, 2F, d] (gate rows, then up
    rows; group E is the shared expert); w_down bf16 [E+1, d, F].
    """

    def __init__(self, w_router, w_gate_up, w_down, top_k: int, max_tokens: int, has_shared: bool = True,
                 out_fp32: bool = False, scales=None):
        E, d = w_router.shape
        G, twoF, d2 = w_gate_up.shape
        F = twoF // 2
        if d2 != d or G != E + int(has_shared) or tuple(w_down.shape) != (G, d, F):
            raise ValueError("weight shapes do not match [E,d], [G,2F,d], [G,d,F]")
        wdt = torch.uint8 if scales is not None else torch.bfloat16
        if w_router.dtype != torch.float32 or w_gate_up.dtype != wdt or w_down.dtype != wdt:
            raise TypeError("w_router must be fp32 and the expert weights bf16 (or uint8 E4M3 codes with scales)")
        self.weights = (w_router, w_gate_up, w_down) + tuple(scales or ())  # borrowed by the handle
        self.d, self.E, self.k, self.F = d, E, top_k, F
        self.has_shared, self.out_fp32, self.max_tokens = has_shared, out_fp32, max_tokens
        self.device = w_gate_up.device
        cfg = moe_config(d, E, top_k, F, int(has_shared), max_tokens, int(out_fp32))
        if scales is None:
            self.handle = moe_init(cfg, w_router, w_gate_up, w_down)
        else:
            s_gu, s_d = scales
            if tuple(s_gu.shape) != (G, 2 * F) or tuple(s_d.shape) != (G, d):
                raise ValueError("scales must be [G, 2F] and [G, d]")
            self.handle = moe_init_fp8(cfg, w_router, w_gate_up, s_gu, w_down, s_d)

    @classmethod
    def fp8(cls, w_router, q_gate_up, s_gate_up, q_down, s_down, top_k: int, max_tokens: int,
            has_shared: bool = True, out_fp32: bool = False) -> "MoeLayer":
        """A layer with E4M3 expert weights (uint8 codes) and fp32 row scales."""
        return cls(w_router, q_gate_up, q_down, top_k, max_tokens, has_shared, out_fp32,
                   scales=(s_gate_up, s_down))

    def route(self, x: torch.Tensor, stream=None, with_gap: bool = True, top_k: int | None = None,
              renormalize: bool = False):
        T = x.shape[0]
        dev = x.device
        k = top_k or self.k
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        prob = torch.empty((T, k), dtype=torch.float32, device=dev)
        perm = torch.empty((T * k,), dtype=torch.int32, device=dev)
        offsets = torch.empty((self.E + 2,), dtype=torch.int32, device=dev)
        gap = torch.empty((T,), dtype=torch.float32, device=dev) if with_gap else None
        if top_k is None and not renormalize:
            moe_route(self.handle, x, T, idx, prob, perm, offsets, gap, stream)
        else:
            moe_route_ex(self.handle, x, T, top_k, renormalize, idx, prob, perm, offsets, gap, stream)
        return idx, prob, perm, offsets, gap

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None, top_k: int | None = None,
                renormalize: bool = False) -> torch.Tensor:
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.d), dtype=torch.float32 if self.out_fp32 else torch.bfloat16,
                            device=x.device)
        if top_k is None and not renormalize:
            moe_forward(self.handle, x, T, y, stream)
        else:
            moe_forward_ex(self.handle, x, T, top_k, renormalize, y, stream)
        return y

    def route_stats(self, x: torch.Tensor, n_groups: int, stream=None):
        """(counts [E] int32, group_f [G], group_p [G], summary [4]) on the device."""
        T = x.shape[0]
        dev = x.device
        counts = torch.empty((self.E,), dtype=torch.int32, device=dev)
        group_f = torch.empty((n_groups,), dtype=torch.float32, device=dev)
        group_p = torch.empty((n_groups,), dtype=torch.float32, device=dev)
        summary = torch.empty((4,), dtype=torch.float32, device=dev)
        moe_route_stats(self.handle, x, T, n_groups, counts, group_f, group_p, summary, stream)
        return counts, group_f, group_p, summary

    __call__ = forward

    def forward_host(self, x_host: torch.Tensor, y_host: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        T = x_host.shape[0]
        if y_host is None:
            y_host = torch.empty((T, self.d), dtype=torch.float32 if self.out_fp32 else torch.bfloat16,
                                 pin_memory=True)
        moe_forward_host(self.handle, x_host, T, y_host, stream)
        return y_host

    def check(self, stream=None) -> int:
        return moe_check(self.handle, stream)

    def last_kernel_count(self) -> int:
        return moe_last_kernel_count(self.handle)

    def set_wait_limit(self, ns: int) -> None:
        moe_set_wait_limit(self.handle, ns)

    def profile_enable(self, enable: bool = True) -> None:
        moe_profile_enable(self.handle, enable)

    def profile_read(self):
        return moe_profile_read(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            moe_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
