"""Python binding of libmoe.so, the GB300 routed-MoE expert FFN (MXFP4 weights,
online FP8 activations).

Argument marshalling only: every step runs in the library's CUDA kernels.  PyTorch
provides device memory and the current stream.  The functions carry the C names
(see include/moe.h for argument meaning, layouts and errors); each raises
MoeError when the C call returns a non-zero status.  Importing this package does
not need a GPU; calling into the library does, and fails loudly if libmoe.so has
not been built (python -m moe_expert_ffn_scan_gb300.build).
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
STATUS_WAIT_TIMEOUT = 1
STATUS_BAD_INDEX = 2
STATUS_BAD_PLAN = 4


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        msg = lib().moe_error_string(code).decode() if _LIB is not None else str(code)
        super().__init__(f"{fn}: status {code} ({msg})")
        self.code = code


class moe_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "E", "k", "has_shared")]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w13", "w13_s", "w2", "w2_s")]


class moe_options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("fuse_combine", "fuse_swiglu", "pair_tiles",
                                              "large_chunk_rows")]


class moe_weights_nvfp4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w13", "w13_s", "w13_gs", "w2", "w2_s", "w2_gs")]


class moe_linear_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("M", "N", "K", "act", "bias_dtype", "y_dtype")] +
                [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldr", "ldy", "ldz")])


class moe_swiglu_backward_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "R", "I")]


ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}  # MOE_ACT_*


DEBUG_FIELDS = ("idx", "w", "counts", "offsets", "perm_src", "inv", "xq", "xs", "y13", "hq",
                "hs", "y2")


class moe_debug_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in DEBUG_FIELDS]


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_DP = ctypes.POINTER(moe_dims)


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m moe_expert_ffn_scan_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_error_string.argtypes = [ctypes.c_int]
        L.moe_error_string.restype = ctypes.c_char_p
        for fn in ("moe_workspace_size", "moe_route_workspace_size", "moe_gemm_workspace_size",
                   "moe_host_workspace_size", "moe_workspace_size_nvfp4",
                   "moe_gemm_workspace_size_nvfp4"):
            getattr(L, fn).argtypes = [_DP]
            getattr(L, fn).restype = _SZ
        L.moe_route.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_quant_act.argtypes = [_I, _I, _P, _P, _P, _P]
        L.moe_router_split_bytes.argtypes = [_I, _I]
        L.moe_router_split_bytes.restype = _SZ
        L.moe_router_split.argtypes = [_I, _I, _P, _P, _P]
        L.moe_router_split.restype = ctypes.c_int
        L.moe_router_logits_split.argtypes = [_I, _I, _I, _P, _P, _P, _P]
        L.moe_router_logits_split.restype = ctypes.c_int
        L.moe_router_logits.argtypes = [_I, _I, _I, _P, _P, _P, _P]
        L.moe_grouped_gemm_w13.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_swiglu_quant.argtypes = [_I, _I, _P, _P, _P, _P]
        L.moe_grouped_gemm_w2.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_combine.argtypes = [_DP, _P, _P, _P, _P, _P]
        L.moe_forward.argtypes = [_DP, _P, _P, ctypes.POINTER(moe_weights), _P,
                                  ctypes.POINTER(moe_debug_out), _P, _SZ, _P]
        L.moe_forward_host.argtypes = [_DP, _P, _P, ctypes.POINTER(moe_weights), _P, _P, _SZ,
                                       _P]
        L.moe_forward_timed.argtypes = [_DP, _P, _P, ctypes.POINTER(moe_weights), _P,
                                        ctypes.POINTER(moe_debug_out), ctypes.POINTER(_P), _P,
                                        _SZ, _P]
        _WN = ctypes.POINTER(moe_weights_nvfp4)
        L.moe_forward_nvfp4.argtypes = [_DP, _P, _P, _WN, _P, ctypes.POINTER(moe_debug_out), _P,
                                        _SZ, _P]
        L.moe_forward_nvfp4_timed.argtypes = [_DP, _P, _P, _WN, _P,
                                              ctypes.POINTER(moe_debug_out), ctypes.POINTER(_P),
                                              _P, _SZ, _P]
        L.moe_grouped_gemm_w13_nvfp4.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                                 _P]
        L.moe_grouped_gemm_w2_nvfp4.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward_ex.argtypes = [_DP, _P, _P, ctypes.POINTER(moe_weights),
                                     ctypes.POINTER(moe_options), _P,
                                     ctypes.POINTER(moe_debug_out), ctypes.POINTER(_P), _P, _SZ,
                                     _P]
        L.moe_route_static.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_route_static_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_check_status.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_join_status.argtypes = [_P, ctypes.POINTER(_P), _I, _P]
        L.moe_join_status.restype = ctypes.c_int
        L.moe_selftest_wait_timeout.argtypes = [_P, _P]
        L.moe_host_pipeline_workspace_size.argtypes = [_DP, _I]
        L.moe_host_pipeline_workspace_size.restype = _SZ
        L.moe_host_pipeline_create.argtypes = [_DP, ctypes.POINTER(moe_weights), _I, _P, _SZ,
                                               ctypes.POINTER(_P)]
        L.moe_host_pipeline_submit.argtypes = [_P, _P, _P, _P]
        L.moe_host_pipeline_sync.argtypes = [_P]
        L.moe_host_pipeline_destroy.argtypes = [_P]
        for fn in ("moe_host_pipeline_create", "moe_host_pipeline_submit",
                   "moe_host_pipeline_sync", "moe_host_pipeline_destroy"):
            getattr(L, fn).restype = ctypes.c_int
        _F = ctypes.c_float
        L.moe_add_rmsnorm.argtypes = [_I, _I, _P, _P, _I, _P, _I, _F, _P, _P, _P, _P, _P, _P]
        L.moe_add_rmsnorm_backward_workspace_size.argtypes = [_I, _I]
        L.moe_add_rmsnorm_backward.argtypes = [_I, _I, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P,
                                               _P, _SZ, _P]
        L.moe_balance_loss_workspace_size.argtypes = [_I] * 4
        L.moe_balance_loss.argtypes = [_I] * 4 + [_P] * 10 + [_SZ, _P]
        L.moe_balance_loss_backward.argtypes = [_I] * 4 + [_P] * 11
        _LD = ctypes.POINTER(moe_linear_desc)
        L.moe_linear_workspace_size.argtypes = [_LD]
        L.moe_linear.argtypes = [_LD] + [_P] * 7 + [_SZ, _P]
        L.moe_linear_backward_workspace_size.argtypes = [_LD]
        L.moe_linear_backward.argtypes = [_LD] + [_P] * 8 + [_SZ, _P]
        for fn in ("moe_add_rmsnorm_backward_workspace_size", "moe_balance_loss_workspace_size",
                   "moe_linear_workspace_size", "moe_linear_backward_workspace_size"):
            getattr(L, fn).restype = _SZ
        for fn in ("moe_add_rmsnorm", "moe_add_rmsnorm_backward", "moe_balance_loss",
                   "moe_balance_loss_backward", "moe_linear", "moe_linear_backward"):
            getattr(L, fn).restype = ctypes.c_int
        L.moe_dispatch.argtypes = [_DP] + [_P] * 4
        L.moe_dispatch_backward.argtypes = [_DP, _P, _P, _P, _I, _P, _P]
        L.moe_combine_backward.argtypes = [_DP] + [_P] * 7
        L.moe_swiglu_quant_save.argtypes = [_I, _I] + [_P] * 6
        L.moe_swiglu_backward.argtypes = ([ctypes.POINTER(moe_swiglu_backward_desc)] + [_P] * 11)
        L.moe_gemm_backward_workspace_size.argtypes = [_DP]
        L.moe_gemm_backward_workspace_size.restype = _SZ
        for fn in ("moe_grouped_gemm_w2_backward", "moe_grouped_gemm_w13_backward"):
            getattr(L, fn).argtypes = [_DP] + [_P] * 6 + [_SZ, _P]
            getattr(L, fn + "_nvfp4").argtypes = [_DP] + [_P] * 7 + [_SZ, _P]
            getattr(L, fn + "_nvfp4").restype = ctypes.c_int
        L.moe_gemm_backward_ctas.argtypes = [_DP, _I]
        L.moe_gemm_backward_ctas.restype = ctypes.c_int
        L.moe_gemm_backward_form.argtypes = [_DP, _I, _I, _I] + [_P] * 7 + [_SZ, _P]
        L.moe_gemm_backward_form.restype = ctypes.c_int
        for fn in ("moe_dispatch", "moe_dispatch_backward", "moe_combine_backward",
                   "moe_swiglu_quant_save", "moe_swiglu_backward",
                   "moe_grouped_gemm_w2_backward", "moe_grouped_gemm_w13_backward"):
            getattr(L, fn).restype = ctypes.c_int
        for fn in ("moe_route", "moe_quant_act", "moe_grouped_gemm_w13", "moe_swiglu_quant",
                   "moe_grouped_gemm_w2", "moe_combine", "moe_forward", "moe_forward_timed",
                   "moe_check_status", "moe_forward_nvfp4", "moe_forward_nvfp4_timed",
                   "moe_grouped_gemm_w13_nvfp4", "moe_grouped_gemm_w2_nvfp4",
                   "moe_route_static", "moe_route_static_status", "moe_forward_ex"):
            getattr(L, fn).restype = ctypes.c_int
        _LIB = L
    return _LIB


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _raw_stream(stream):
    """_stream for calls short enough for its cost to show (tensors exist: CUDA is up)."""
    if stream is not None:
        return stream.cuda_stream
    return _current_raw_stream(_current_device())


_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _t(t, dtype, shape, name):
    """_p of a tensor whose type and shape are checked first (None stays None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return _p(t)  # raises


_DTYPE_CODE = {torch.bfloat16: 0, torch.float32: 1}  # MOE_DTYPE_*


def _dtype_code(t, name):
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return code


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def dims(T, H, I, E, k, has_shared):
    return moe_dims(int(T), int(H), int(I), int(E), int(k), int(has_shared))


def _d(d):
    if not isinstance(d, moe_dims):
        d = dims(d.T, d.H, d.I, d.E, d.k, d.has_shared)
    return ctypes.byref(d)


def workspace_size(d) -> int:
    return lib().moe_workspace_size(_d(d))


def host_workspace_size(d) -> int:
    return lib().moe_host_workspace_size(_d(d))


def host_pipeline_workspace_size(d, depth) -> int:
    return lib().moe_host_pipeline_workspace_size(_d(d), depth)


def workspace_size_nvfp4(d) -> int:
    return lib().moe_workspace_size_nvfp4(_d(d))


def gemm_workspace_size_nvfp4(d) -> int:
    return lib().moe_gemm_workspace_size_nvfp4(_d(d))


def route_workspace_size(d) -> int:
    return lib().moe_route_workspace_size(_d(d))


def gemm_workspace_size(d) -> int:
    return lib().moe_gemm_workspace_size(_d(d))


def alloc_workspace(nbytes, device="cuda", stream=None):
    """A workspace tensor (torch allocations are 256-byte aligned or better), its status
    word zeroed.  It belongs to `stream` (None: the current one), which does the zeroing:
    calls that use it on another stream have to be ordered behind that."""
    with torch.cuda.stream(stream):
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        ws[:256].zero_()
    return ws


def moe_route(d, logits, idx, w, counts, offsets, perm_src, inv, ws, stream=None):
    _check("moe_route", lib().moe_route(_d(d), _p(logits), _p(idx), _p(w), _p(counts),
                                        _p(offsets), _p(perm_src), _p(inv), _p(ws),
                                        ws.numel(), _stream(stream)))


def moe_router_logits(x, wg, logits, stream=None):
    """logits [T, E] fp32 = x [T, H] bf16 . wg [E, H] fp32 ^T (router gate projection)."""
    T, H = x.shape
    E = wg.shape[0]
    _check("moe_router_logits", lib().moe_router_logits(T, H, E, _p(x), _p(wg), _p(logits),
                                                        _stream(stream)))


def moe_router_split(wg, wg3=None, stream=None):
    """Splits the fp32 gate weight [E, H] into the three bf16 pieces [3, E, H] the
    tensor-core router projection reads (hi + mid + lo == wg).  Returns wg3."""
    E, H = wg.shape
    if wg3 is None:
        wg3 = torch.empty(3, E, H, dtype=torch.bfloat16, device=wg.device)
    _check("moe_router_split", lib().moe_router_split(E, H, _p(wg), _p(wg3), _stream(stream)))
    return wg3


def moe_router_logits_split(x, wg3, logits, stream=None):
    """logits [T, E] fp32 = x [T, H] bf16 . wg^T on the tensor cores, from the pieces of
    moe_router_split."""
    T, H = x.shape
    E = wg3.shape[1]
    _check("moe_router_logits_split", lib().moe_router_logits_split(
        T, H, E, _p(x), _p(wg3), _p(logits), _stream(stream)))


def moe_quant_act(x, q, s, stream=None):
    rows, cols = x.shape
    _check("moe_quant_act", lib().moe_quant_act(rows, cols, _p(x), _p(q), _p(s),
                                                _stream(stream)))


def moe_grouped_gemm_w13(d, xq, xs, perm_src, group_offsets, w13, w13_s, y13, ws, stream=None):
    _check("moe_grouped_gemm_w13", lib().moe_grouped_gemm_w13(
        _d(d), _p(xq), _p(xs), _p(perm_src), _p(group_offsets), _p(w13), _p(w13_s), _p(y13),
        _p(ws), ws.numel(), _stream(stream)))


def moe_swiglu_quant(y13, hq, hs, stream=None):
    rows, two_i = y13.shape
    _check("moe_swiglu_quant", lib().moe_swiglu_quant(rows, two_i // 2, _p(y13), _p(hq), _p(hs),
                                                      _stream(stream)))


def moe_grouped_gemm_w2(d, hq, hs, group_offsets, w2, w2_s, y2, ws, stream=None):
    _check("moe_grouped_gemm_w2", lib().moe_grouped_gemm_w2(
        _d(d), _p(hq), _p(hs), _p(group_offsets), _p(w2), _p(w2_s), _p(y2), _p(ws),
        ws.numel(), _stream(stream)))


def moe_combine(d, y2, inv, w, out, stream=None):
    _check("moe_combine", lib().moe_combine(_d(d), _p(y2), _p(inv), _p(w), _p(out),
                                            _stream(stream)))


def moe_forward(d, x, logits, w13, w13_s, w2, w2_s, out, ws, debug=None, stream=None):
    W = moe_weights(_p(w13), _p(w13_s), _p(w2), _p(w2_s))
    dbg = None
    if debug:
        dbg = moe_debug_out(*[_p(debug.get(n)) for n in DEBUG_FIELDS])
    _check("moe_forward", lib().moe_forward(
        _d(d), _p(x), _p(logits), ctypes.byref(W), _p(out),
        ctypes.byref(dbg) if dbg is not None else None, _p(ws), ws.numel(), _stream(stream)))


def _nv_weights(w13, w13_s, w13_gs, w2, w2_s, w2_gs):
    return moe_weights_nvfp4(_p(w13), _p(w13_s), _p(w13_gs), _p(w2), _p(w2_s), _p(w2_gs))


def moe_forward_nvfp4(d, x, logits, w13, w13_s, w13_gs, w2, w2_s, w2_gs, out, ws, debug=None,
                      stream=None):
    """moe_forward with NVFP4 expert weights (codes, E4M3 scales per 16, fp32 tensor
    scales [G, 2] / [G] or None); ws: workspace_size_nvfp4(d) bytes."""
    W = _nv_weights(w13, w13_s, w13_gs, w2, w2_s, w2_gs)
    dbg = None
    if debug:
        dbg = moe_debug_out(*[_p(debug.get(n)) for n in DEBUG_FIELDS])
    _check("moe_forward_nvfp4", lib().moe_forward_nvfp4(
        _d(d), _p(x), _p(logits), ctypes.byref(W), _p(out),
        ctypes.byref(dbg) if dbg is not None else None, _p(ws), ws.numel(), _stream(stream)))


def moe_forward_nvfp4_timed(d, x, logits, w13, w13_s, w13_gs, w2, w2_s, w2_gs, out, ws, events,
                            stream=None):
    W = _nv_weights(w13, w13_s, w13_gs, w2, w2_s, w2_gs)
    ev = (_P * 8)(*[e.cuda_event for e in events])
    _check("moe_forward_nvfp4_timed", lib().moe_forward_nvfp4_timed(
        _d(d), _p(x), _p(logits), ctypes.byref(W), _p(out), None, ev, _p(ws), ws.numel(),
        _stream(stream)))


def moe_grouped_gemm_w13_nvfp4(d, xq, xs, perm_src, group_offsets, w13, w13_s, w13_gs, y13, ws,
                               stream=None):
    _check("moe_grouped_gemm_w13_nvfp4", lib().moe_grouped_gemm_w13_nvfp4(
        _d(d), _p(xq), _p(xs), _p(perm_src), _p(group_offsets), _p(w13), _p(w13_s), _p(w13_gs),
        _p(y13), _p(ws), ws.numel(), _stream(stream)))


def moe_grouped_gemm_w2_nvfp4(d, hq, hs, group_offsets, w2, w2_s, w2_gs, y2, ws, stream=None):
    _check("moe_grouped_gemm_w2_nvfp4", lib().moe_grouped_gemm_w2_nvfp4(
        _d(d), _p(hq), _p(hs), _p(group_offsets), _p(w2), _p(w2_s), _p(w2_gs), _p(y2), _p(ws),
        ws.numel(), _stream(stream)))


def moe_route_static(d, logits, idx, w, counts, offsets, perm_src, inv, stream=None):
    """moe_route without a workspace: its scratch is a fixed array inside the library
    (calls must not overlap on the GPU)."""
    _check("moe_route_static", lib().moe_route_static(
        _d(d), _p(logits), _p(idx), _p(w), _p(counts), _p(offsets), _p(perm_src), _p(inv),
        _stream(stream)))


def moe_route_static_status(stream=None) -> int:
    """Synchronises the stream and returns the device status bits of moe_route_static's
    fixed array (those of its last call)."""
    bits = ctypes.c_uint32(0)
    rc = lib().moe_route_static_status(_stream(stream), ctypes.byref(bits))
    if rc not in (MOE_OK, 5):
        raise MoeError("moe_route_static_status", rc)
    return bits.value


def moe_forward_ex(d, x, logits, w13, w13_s, w2, w2_s, out, ws, fuse_combine=False,
                   fuse_swiglu=False, pair_tiles=False, large_chunk_rows=0, debug=None,
                   events=None, stream=None):
    """moe_forward with options (fuse_combine: the W2 GEMM's epilogue performs the
    weighted top-k combine + shared add; fuse_swiglu: the W13 GEMM's epilogue performs
    SwiGLU + FP8 quantisation; pair_tiles: groups above 64 rows on SM pairs;
    large_chunk_rows: the tile plan's chunk size for groups above 64 rows, 0 = 224) and
    optional stage events."""
    W = moe_weights(_p(w13), _p(w13_s), _p(w2), _p(w2_s))
    opt = moe_options(int(bool(fuse_combine)), int(bool(fuse_swiglu)), int(bool(pair_tiles)),
                      int(large_chunk_rows))
    dbg = None
    if debug:
        dbg = moe_debug_out(*[_p(debug.get(n)) for n in DEBUG_FIELDS])
    ev = (_P * 8)(*[e.cuda_event for e in events]) if events else None
    _check("moe_forward_ex", lib().moe_forward_ex(
        _d(d), _p(x), _p(logits), ctypes.byref(W), ctypes.byref(opt), _p(out),
        ctypes.byref(dbg) if dbg is not None else None, ev, _p(ws), ws.numel(),
        _stream(stream)))


def _host_p(t):
    if t.device.type != "cpu":
        raise ValueError("tensor must live in host memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def moe_forward_host(d, x_host, logits_host, w13, w13_s, w2, w2_s, out_host, ws, stream=None):
    """The layer from host buffers to a host buffer (two copies in, one out, on the
    stream; pinned buffers keep them asynchronous).  ws: host_workspace_size(d)."""
    W = moe_weights(_p(w13), _p(w13_s), _p(w2), _p(w2_s))
    _check("moe_forward_host", lib().moe_forward_host(
        _d(d), _host_p(x_host), _host_p(logits_host), ctypes.byref(W), _host_p(out_host),
        _p(ws), ws.numel(), _stream(stream)))


STAGES = ("route", "quant", "plan_gather", "gemm_w13", "swiglu_quant", "gemm_w2", "combine")


def moe_forward_timed(d, x, logits, w13, w13_s, w2, w2_s, out, ws, events, debug=None,
                      stream=None):
    """moe_forward recording 8 torch.cuda.Event objects at the stage boundaries (see
    STAGES); the events must already exist (recorded once)."""
    W = moe_weights(_p(w13), _p(w13_s), _p(w2), _p(w2_s))
    dbg = None
    if debug:
        dbg = moe_debug_out(*[_p(debug.get(n)) for n in DEBUG_FIELDS])
    ev = (_P * 8)(*[e.cuda_event for e in events])
    _check("moe_forward_timed", lib().moe_forward_timed(
        _d(d), _p(x), _p(logits), ctypes.byref(W), _p(out),
        ctypes.byref(dbg) if dbg is not None else None, ev, _p(ws), ws.numel(),
        _stream(stream)))


# ---------------------------------------------------------------- around the expert FFN

def add_rmsnorm_backward_workspace_size(rows, cols) -> int:
    return lib().moe_add_rmsnorm_backward_workspace_size(rows, cols)


def moe_add_rmsnorm(x, residual, gain, eps, h=None, y=None, q=None, s=None, rstd=None,
                    stream=None):
    """a = x + residual (or x), RMS norm of a times gain.  x [rows, cols] bf16, residual and h
    bf16 or fp32 (the residual stream), gain bf16 or fp32 [cols].  Writes what is given of h
    (a), y (bf16), q / s (uint8 E4M3 codes [rows, cols] and scale bytes [rows, cols / 128] of
    y) and rstd [rows] fp32."""
    rows, cols = shape = x.shape
    st = residual if residual is not None else h
    sd = st.dtype if st is not None else torch.bfloat16
    sc = _dtype_code(st, "residual / h") if st is not None else 0
    rc = lib().moe_add_rmsnorm(
        rows, cols, _t(x, torch.bfloat16, shape, "x"), _t(residual, sd, shape, "residual"), sc,
        _t(gain, gain.dtype, (cols,), "gain"), _dtype_code(gain, "gain"), eps,
        _t(h, sd, shape, "h"), _t(y, torch.bfloat16, shape, "y"), _t(q, torch.uint8, shape, "q"),
        _t(s, torch.uint8, (rows, cols // 128), "s"), _t(rstd, torch.float32, (rows,), "rstd"),
        _raw_stream(stream))
    if rc:
        raise MoeError("moe_add_rmsnorm", rc)


def moe_add_rmsnorm_backward(dy, h, gain, rstd, ws, dh_in=None, dh=None, dx=None, dgain=None,
                             stream=None):
    """Gradient of moe_add_rmsnorm from dy [rows, cols] bf16, the forward's h and rstd, and
    dh_in (the gradient that reaches h by other ways, or None).  Writes what is given of dh
    (h's type), dx (dh in bf16) and dgain [cols] fp32.  ws:
    add_rmsnorm_backward_workspace_size(rows, cols) bytes (None without dgain)."""
    rows, cols = shape = dy.shape
    hd = h.dtype
    rc = lib().moe_add_rmsnorm_backward(
        rows, cols, _t(dy, torch.bfloat16, shape, "dy"), _t(h, hd, shape, "h"),
        _dtype_code(h, "h"), _t(gain, gain.dtype, (cols,), "gain"), _dtype_code(gain, "gain"),
        _t(rstd, torch.float32, (rows,), "rstd"), _t(dh_in, hd, shape, "dh_in"),
        _t(dh, hd, shape, "dh"), _t(dx, torch.bfloat16, shape, "dx"),
        _t(dgain, torch.float32, (cols,), "dgain"), _p(ws), ws.numel() if ws is not None else 0,
        _raw_stream(stream))
    if rc:
        raise MoeError("moe_add_rmsnorm_backward", rc)


def balance_loss_workspace_size(T, E, k, S=1) -> int:
    return lib().moe_balance_loss_workspace_size(T, E, k, S)


def _balance_args(logits, idx, seq_offsets, token_mask):
    """(T, E, k, S) and the pointers of the four inputs, checked."""
    T, E = logits.shape
    k = idx.shape[1]
    S = seq_offsets.shape[0] - 1 if seq_offsets is not None else 1
    if token_mask is not None and token_mask.dtype is torch.bool:
        token_mask = token_mask.view(torch.uint8)
    return (T, E, k, S), (
        _t(logits, torch.float32, (T, E), "logits"), _t(idx, torch.int32, (T, k), "idx"),
        _t(seq_offsets, torch.int32, (S + 1,), "seq_offsets"),
        _t(token_mask, torch.uint8, (T,), "token_mask"))


def moe_balance_loss(logits, idx, counts, n_tokens, prob, loss, z_loss, ws, seq_offsets=None,
                     token_mask=None, stream=None):
    """Balance loss of logits [T, E] fp32 and the chosen experts idx [T, k] int32, for each of
    the S sequences of seq_offsets [S + 1] int32 (None: one sequence of all tokens), without
    the tokens whose token_mask [T] (uint8 or bool) is 0.  Writes counts [S, E] and n_tokens
    [S] int32, prob [S, E], loss [S] and, if given, z_loss [S] fp32.  ws:
    balance_loss_workspace_size(T, E, k, S) bytes; moe_check_status(ws) reads its checks."""
    (T, E, k, S), inputs = _balance_args(logits, idx, seq_offsets, token_mask)
    rc = lib().moe_balance_loss(
        T, E, k, S, *inputs, _t(counts, torch.int32, (S, E), "counts"),
        _t(n_tokens, torch.int32, (S,), "n_tokens"), _t(prob, torch.float32, (S, E), "prob"),
        _t(loss, torch.float32, (S,), "loss"), _t(z_loss, torch.float32, (S,), "z_loss"),
        _p(ws), ws.numel(), _raw_stream(stream))
    if rc:
        raise MoeError("moe_balance_loss", rc)


def moe_balance_loss_backward(logits, idx, counts, n_tokens, dlogits, dloss=None, dz_loss=None,
                              dw=None, seq_offsets=None, token_mask=None, stream=None):
    """Gradient of the logits [T, E] from dloss [S], dz_loss [S] (moe_balance_loss's outputs)
    and dw [T, k] (moe_route's combine weights), each None for none; counts and n_tokens as
    the forward wrote them.  Writes dlogits [T, E] fp32."""
    (T, E, k, S), inputs = _balance_args(logits, idx, seq_offsets, token_mask)
    rc = lib().moe_balance_loss_backward(
        T, E, k, S, *inputs, _t(counts, torch.int32, (S, E), "counts"),
        _t(n_tokens, torch.int32, (S,), "n_tokens"), _t(dloss, torch.float32, (S,), "dloss"),
        _t(dz_loss, torch.float32, (S,), "dz_loss"), _t(dw, torch.float32, (T, k), "dw"),
        _t(dlogits, torch.float32, (T, E), "dlogits"), _raw_stream(stream))
    if rc:
        raise MoeError("moe_balance_loss_backward", rc)


def _linear_desc(M, N, K, act="none", ldx=0, ldw=0, ldr=0, ldy=0, ldz=0):
    return moe_linear_desc(M, N, K, ACTS[act], 0, 0, ldx, ldw, ldr, ldy, ldz)


def linear_workspace_size(M, N, K, ldx=0, ldw=0) -> int:
    """ldx, ldw: row strides of x and w in elements (0: contiguous)."""
    return lib().moe_linear_workspace_size(ctypes.byref(_linear_desc(M, N, K, ldx=ldx, ldw=ldw)))


def linear_backward_workspace_size(M, N, K, ldx=0, ldw=0, lddy=0, act="silu") -> int:
    """The default act gives the size that does for all of them."""
    return lib().moe_linear_backward_workspace_size(
        ctypes.byref(_linear_desc(M, N, K, act, ldx, ldw, ldy=lddy)))


def _m(t, dtype, shape, name):
    """Pointer and row stride of a matrix whose columns are contiguous (None: null)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    rows, cols = shape
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return t.data_ptr(), ld if rows > 1 else 0


def moe_linear(x, w, y, ws, bias=None, residual=None, z=None, act="none", stream=None):
    """y [M, N] = act(x [M, K] . w [N, K]^T + bias [N]) + residual [M, N].  x, w bf16; y and
    residual bf16 or fp32; bias bf16 or fp32; z [M, N] bf16 takes the value in front of the
    activation.  Matrices may have any row stride.  act: one of ACTS.  ws:
    linear_workspace_size(M, N, K[, ldx, ldw]) bytes."""
    (M, K), N = x.shape, w.shape[0]
    yd, out = y.dtype, (M, N)
    xp, ldx = _m(x, torch.bfloat16, (M, K), "x")
    wp, ldw = _m(w, torch.bfloat16, (N, K), "w")
    rp, ldr = _m(residual, yd, out, "residual")
    yp, ldy = _m(y, yd, out, "y")
    zp, ldz = _m(z, torch.bfloat16, out, "z")
    bp, bd = None, 0
    if bias is not None:
        bd = _dtype_code(bias, "bias")
        bp = _t(bias, bias.dtype, (N,), "bias")
    d = moe_linear_desc(M, N, K, ACTS[act], bd, _dtype_code(y, "y"), ldx, ldw, ldr, ldy, ldz)
    rc = lib().moe_linear(ctypes.byref(d), xp, wp, bp, rp, yp, zp, _p(ws), ws.numel(),
                          _raw_stream(stream))
    if rc:
        raise MoeError("moe_linear", rc)


def moe_linear_backward(x, w, dy, ws, z=None, act="none", dx=None, dw=None, dbias=None,
                        stream=None):
    """Gradient of moe_linear from dy [M, N] bf16 and, with an activation, its z.  Writes
    what is given of dx [M, K], dw [N, K] bf16 and dbias [N] fp32 (contiguous).  ws:
    linear_backward_workspace_size(M, N, K[, ldx, ldw, lddy]) bytes."""
    (M, K), N = x.shape, w.shape[0]
    out = (M, N)
    xp, ldx = _m(x, torch.bfloat16, (M, K), "x")
    wp, ldw = _m(w, torch.bfloat16, (N, K), "w")
    gp, ldg = _m(dy, torch.bfloat16, out, "dy")
    zp, ldz = _m(z, torch.bfloat16, out, "z")
    d = moe_linear_desc(M, N, K, ACTS[act], 0, 0, ldx, ldw, 0, ldg, ldz)
    rc = lib().moe_linear_backward(
        ctypes.byref(d), xp, wp, zp, gp, _t(dx, torch.bfloat16, (M, K), "dx"),
        _t(dw, torch.bfloat16, (N, K), "dw"), _t(dbias, torch.float32, (N,), "dbias"), _p(ws),
        ws.numel(), _raw_stream(stream))
    if rc:
        raise MoeError("moe_linear_backward", rc)


# ---------------------------------------------------------------- the layer's gradient

def _packed_rows(d):
    return d.T * (d.k + d.has_shared)


# (each call's first tensor says on which device it is, here `dev`: the others have to be there,
# and it has to be the current one, on whose streams the call runs)

def _on(dev, t, dtype, shape, name):
    """_t of a tensor on that device."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0 and t.is_contiguous():
        return t.data_ptr()
    _t(t, dtype, shape, name)  # raises, but for another device
    raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _flat(dev, t, dtype, n, name):
    """_on of n contiguous values of any shape."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.get_device() == dev >= 0 and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.numel() != n:
        raise ValueError(f"{name}: expected {n} values of {dtype}, got {t.numel()} of {t.dtype}")
    return _on(dev, t, dtype, t.shape, name)  # raises


def _stream_on(dev, stream):
    """_raw_stream of a call on that device."""
    now = _current_device()
    if now != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{now}")
    return stream.cuda_stream if stream is not None else _current_raw_stream(now)


def moe_dispatch(d, x, inv, xp, stream=None):
    """x [T, H] bf16 to the packed rows of its experts, xp [Rs, H]: row inv[t*k+j] (moe_route's
    inv, [T*k] int32; an entry outside [0, T*k): no row) and, with a shared expert, row
    T*k + t."""
    dev = x.get_device()
    rc = lib().moe_dispatch(
        _d(d), _on(dev, x, _BF16, (d.T, d.H), "x"), _flat(dev, inv, _I32, d.T * d.k, "inv"),
        _on(dev, xp, _BF16, (_packed_rows(d), d.H), "xp"), _stream_on(dev, stream))
    if rc:
        raise MoeError("moe_dispatch", rc)


def moe_dispatch_backward(d, dxp, inv, dx, dx_in=None, stream=None):
    """Gradient of moe_dispatch: dx [T, H] (bf16 or fp32) = dx_in (dx's type, or None) + the sum
    of each token's rows of dxp [Rs, H] bf16."""
    dev = dx.get_device()
    shape, dt, code = (d.T, d.H), dx.dtype, _dtype_code(dx, "dx")
    rc = lib().moe_dispatch_backward(
        _d(d), _on(dev, dxp, _BF16, (_packed_rows(d), d.H), "dxp"),
        _flat(dev, inv, _I32, d.T * d.k, "inv"), _on(dev, dx_in, dt, shape, "dx_in"),
        code, _on(dev, dx, dt, shape, "dx"), _stream_on(dev, stream))
    if rc:
        raise MoeError("moe_dispatch_backward", rc)


def moe_combine_backward(d, dout, y2, inv, w, dy2=None, dw=None, stream=None):
    """Gradient of moe_combine from dout [T, H] bf16: writes what is given of dy2 [Rs, H] bf16
    (w [T, k] fp32 times the token's dout) and dw [T, k] fp32 (from y2 [Rs, H] bf16, else
    None)."""
    dev = dout.get_device()
    rows = (_packed_rows(d), d.H)
    rc = lib().moe_combine_backward(
        _d(d), _on(dev, dout, _BF16, (d.T, d.H), "dout"), _on(dev, y2, _BF16, rows, "y2"),
        _flat(dev, inv, _I32, d.T * d.k, "inv"), _on(dev, w, _F32, (d.T, d.k), "w"),
        _on(dev, dy2, _BF16, rows, "dy2"), _on(dev, dw, _F32, (d.T, d.k), "dw"),
        _stream_on(dev, stream))
    if rc:
        raise MoeError("moe_combine_backward", rc)


def moe_swiglu_quant_save(y13, hq, hs, yq, ys, stream=None):
    """moe_swiglu_quant of y13 [rows, 2I] bf16 (hq [rows, I], hs [rows, I/128]) that also saves
    y13 in 8 bits, yq [rows, 2I] and ys [rows, 2I/128], for moe_swiglu_backward (all uint8)."""
    dev = y13.get_device()
    rows, two_i = y13.shape
    I = two_i // 2
    rc = lib().moe_swiglu_quant_save(
        rows, I, _on(dev, y13, _BF16, (rows, 2 * I), "y13"), _on(dev, hq, _U8, (rows, I), "hq"),
        _on(dev, hs, _U8, (rows, I // 128), "hs"), _on(dev, yq, _U8, (rows, 2 * I), "yq"),
        _on(dev, ys, _U8, (rows, 2 * I // 128), "ys"), _stream_on(dev, stream))
    if rc:
        raise MoeError("moe_swiglu_quant_save", rc)


def moe_swiglu_backward(dh, dy13, y13=None, yq=None, ys=None, hq=None, hs=None, perm_src=None,
                        w=None, dw=None, stream=None):
    """Gradient of SwiGLU from dh [rows, I] bf16 and its input, either in 8 bits (yq, ys as
    moe_swiglu_quant_save wrote them) or y13 [rows, 2I] bf16.  Writes dy13 [rows, 2I] bf16, each
    routed row's (the first perm_src.numel() of them) times its weight of w [T, k] fp32 (None:
    1), and, if given, dw [T, k] fp32: the weights' gradient, from the values of hq, hs if given,
    else from silu(g) u."""
    dev = dh.get_device()
    rows, I = dh.shape
    R = perm_src.numel() if perm_src is not None else 0
    wp, dwp = _flat(dev, w, _F32, R, "w"), _flat(dev, dw, _F32, R, "dw")
    desc = moe_swiglu_backward_desc(rows, R, I)
    two, blocks = (rows, 2 * I), I // 128
    rc = lib().moe_swiglu_backward(
        ctypes.byref(desc), _on(dev, dh, _BF16, (rows, I), "dh"), _on(dev, y13, _BF16, two, "y13"),
        _on(dev, yq, _U8, two, "yq"), _on(dev, ys, _U8, (rows, 2 * blocks), "ys"),
        _on(dev, hq, _U8, (rows, I), "hq"), _on(dev, hs, _U8, (rows, blocks), "hs"),
        _flat(dev, perm_src, _I32, R, "perm_src"), wp, _on(dev, dy13, _BF16, two, "dy13"), dwp,
        _stream_on(dev, stream))
    if rc:
        raise MoeError("moe_swiglu_backward", rc)


def gemm_backward_workspace_size(d) -> int:
    return lib().moe_gemm_backward_workspace_size(_d(d))


def _gemm_backward(name, d, dy, cols_in, group_offsets, w, w_s, dx, cols_out, ws, stream,
                   block=32, scales=(), form=()):
    dev = dy.get_device()
    rows, G = _packed_rows(d), d.E + d.has_shared
    rc = getattr(lib(), name)(
        _d(d), *form, _on(dev, dy, _BF16, (rows, cols_in), "dy"),
        _on(dev, group_offsets, _I32, (G + 1,), "group_offsets"),
        _on(dev, w, _U8, (G, cols_in, cols_out // 2), "w"),
        _on(dev, w_s, _U8, (G, cols_in, cols_out // block), "w_s"),
        *[_on(dev, t, _F32, shape, n) for t, shape, n in scales],
        _on(dev, dx, _BF16, (rows, cols_out), "dx"), _on(dev, ws, ws.dtype, ws.shape, "ws"),
        ws.numel(), _stream_on(dev, stream))
    if rc:
        raise MoeError(name, rc)


def moe_grouped_gemm_w2_backward(d, dy2, group_offsets, w2, w2_s, dh, ws, stream=None):
    """dh [Rs, I] = dy2 [Rs, H] . deq(w2[g]) [H, I] for the packed rows of each group (bf16, MXFP4
    weights).  ws: gemm_backward_workspace_size(d) bytes, kept to the gradient products."""
    _gemm_backward("moe_grouped_gemm_w2_backward", d, dy2, d.H, group_offsets, w2, w2_s, dh, d.I,
                   ws, stream)


def moe_grouped_gemm_w13_backward(d, dy13, group_offsets, w13, w13_s, dxp, ws, stream=None):
    """dxp [Rs, H] = dy13 [Rs, 2I] . deq(w13[g]) [2I, H], as moe_grouped_gemm_w2_backward."""
    _gemm_backward("moe_grouped_gemm_w13_backward", d, dy13, 2 * d.I, group_offsets, w13, w13_s,
                   dxp, d.H, ws, stream)


def moe_grouped_gemm_w2_backward_nvfp4(d, dy2, group_offsets, w2, w2_s, w2_gs, dh, ws,
                                       stream=None):
    """moe_grouped_gemm_w2_backward with NVFP4 weights: w2_s [G, H, I/16] E4M3 scales, w2_gs [G]
    fp32 (None: 1)."""
    _gemm_backward("moe_grouped_gemm_w2_backward_nvfp4", d, dy2, d.H, group_offsets, w2, w2_s, dh,
                   d.I, ws, stream, 16, [(w2_gs, (d.E + d.has_shared,), "w2_gs")])


def moe_grouped_gemm_w13_backward_nvfp4(d, dy13, group_offsets, w13, w13_s, w13_gs, dxp, ws,
                                        stream=None):
    """moe_grouped_gemm_w13_backward with NVFP4 weights: w13_s [G, 2I, H/16] E4M3 scales, w13_gs
    [G, 2] fp32 of the gate and up rows (None: 1)."""
    _gemm_backward("moe_grouped_gemm_w13_backward_nvfp4", d, dy13, 2 * d.I, group_offsets, w13,
                   w13_s, dxp, d.H, ws, stream, 16,
                   [(w13_gs, (d.E + d.has_shared, 2), "w13_gs")])


def gemm_backward_ctas(d, product) -> int:
    """CTAs a tile that the gradient product (2 or 13) of these dims runs with: 1, or 2 (SM pairs)."""
    return lib().moe_gemm_backward_ctas(_d(d), product)


def moe_gemm_backward_form(d, product, ctas, dy, group_offsets, w, w_s, dx, ws, gs=None,
                           nvfp4=False, stream=None):
    """The gradient product 2 or 13 with `ctas` CTAs a tile, whatever the dims' cost (for tests)."""
    cols = (d.H, d.I) if product == 2 else (2 * d.I, d.H)
    G = d.E + d.has_shared
    _gemm_backward("moe_gemm_backward_form", d, dy, cols[0], group_offsets, w, w_s, dx, cols[1], ws,
                   stream, 16 if nvfp4 else 32, [(gs, (G,) if product == 2 else (G, 2), "gs")],
                   (product, int(nvfp4), ctas))


def moe_check_status(ws, stream=None) -> int:
    """Synchronises the stream and returns the device status bits of a workspace."""
    bits = ctypes.c_uint32(0)
    rc = lib().moe_check_status(_p(ws), _stream(stream), ctypes.byref(bits))
    if rc not in (MOE_OK, 5):
        raise MoeError("moe_check_status", rc)
    return bits.value


def stage_workspaces(ws, n):
    """n workspaces in one buffer, for calls one behind another on a stream: a status word each,
    256 bytes apart, the scratch behind them shared (the buffer: 256 (n - 1) bytes and the largest
    call's).  moe_join_status makes their words one."""
    return [ws[256 * i:] for i in range(n)]


def moe_join_status(ws, others, stream=None):
    """ORs the status words of the workspaces `others` (up to 8) into that of ws, on the stream."""
    n = len(others)
    rc = lib().moe_join_status(_p(ws), (_P * n)(*[_p(w) for w in others]), n, _raw_stream(stream))
    if rc:
        raise MoeError("moe_join_status", rc)


def moe_selftest_wait_timeout(ws, stream=None):
    """Runs the failure-path self-test (a wait that must time out) on ws's status word."""
    _check("moe_selftest_wait_timeout", lib().moe_selftest_wait_timeout(_p(ws), _stream(stream)))


def debug_buffers(d, device="cuda"):
    """Device buffers for every intermediate moe_forward can expose."""
    T, H, I, E, k, sh = d.T, d.H, d.I, d.E, d.k, d.has_shared
    R = T * k
    Rs = R + (T if sh else 0)
    G = E + sh
    z = lambda *s, dt: torch.empty(*s, dtype=dt, device=device)
    return dict(idx=z(T, k, dt=torch.int32), w=z(T, k, dt=torch.float32),
                counts=z(E, dt=torch.int32), offsets=z(G + 1, dt=torch.int32),
                perm_src=z(max(R, 1), dt=torch.int32), inv=z(max(R, 1), dt=torch.int32),
                xq=z(T, H, dt=torch.uint8), xs=z(T, H // 128, dt=torch.uint8),
                y13=z(Rs, 2 * I, dt=torch.bfloat16), hq=z(Rs, I, dt=torch.uint8),
                hs=z(Rs, I // 128, dt=torch.uint8), y2=z(Rs, H, dt=torch.bfloat16))


class HostGraph:
    """forward_host captured once as a CUDA graph over pinned buffers x_host [T, H]
    bf16, logits_host [T, E] fp32 and out_host [T, H] bf16.  Write a step's inputs
    into x_host / logits_host, call replay(), synchronise, read out_host."""

    def __init__(self, layer, T):
        self.layer, self.T = layer, T
        self.x_host = torch.zeros(T, layer.H, dtype=torch.bfloat16).pin_memory()
        self.logits_host = torch.zeros(T, layer.E, dtype=torch.float32).pin_memory()
        self.out_host = torch.zeros(T, layer.H, dtype=torch.bfloat16).pin_memory()
        layer.host_workspace(T)  # allocated before capture
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer.forward_host(self.x_host, self.logits_host, self.out_host)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            layer.forward_host(self.x_host, self.logits_host, self.out_host)
        torch.cuda.synchronize()

    def replay(self):
        self.graph.replay()
        return self.out_host


class HostPipeline:
    """The native host-buffer pipeline (moe_host_pipeline_*): submit() enqueues one
    layer step from pinned host buffers to a pinned host buffer and returns; step i's
    copies overlap steps i-1 and i+1 on the pipeline's own streams; sync() waits for
    every submitted step.  Buffers passed to submit() stay in use until sync()."""

    def __init__(self, layer, T, depth=2):
        self.T, self.H, self.E, self.depth = T, layer.H, layer.E, depth
        d = layer.dims(T)
        size = host_pipeline_workspace_size(d, depth)
        if size == 0:
            raise ValueError(f"unsupported dims or depth {depth} (1..8)")
        self.ws = alloc_workspace(size, layer.w13.device)
        # the pipeline's own streams wait for no other: what is queued for this memory (its
        # zeroing, its last owner's kernels) and for the weights ends first
        torch.cuda.current_stream(layer.w13.device).synchronize()
        self._weights = (layer.w13, layer.w13_s, layer.w2, layer.w2_s)  # kept alive
        W = moe_weights(*[_p(t) for t in self._weights])
        h = _P()
        _check("moe_host_pipeline_create", lib().moe_host_pipeline_create(
            _d(d), ctypes.byref(W), depth, _p(self.ws), self.ws.numel(), ctypes.byref(h)))
        self._h = h

    def _host(self, t, shape, dtype):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
        return _host_p(t)

    def submit(self, x_host, logits_host, out_host):
        if self._h is None:
            raise RuntimeError("pipeline closed")
        _check("moe_host_pipeline_submit", lib().moe_host_pipeline_submit(
            self._h, self._host(x_host, (self.T, self.H), torch.bfloat16),
            self._host(logits_host, (self.T, self.E), torch.float32),
            self._host(out_host, (self.T, self.H), torch.bfloat16)))

    def sync(self):
        _check("moe_host_pipeline_sync", lib().moe_host_pipeline_sync(self._h))

    def close(self):
        if getattr(self, "_h", None) is not None:
            h, self._h = self._h, None
            _check("moe_host_pipeline_destroy", lib().moe_host_pipeline_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _LayerWorkspace:
    """A layer's workspace for the longest step so far (size: T -> bytes), made anew for a longer
    one.  A graph goes on using the one it was captured with, which therefore stays as long as
    the layer; any other is given back once the streams that used it are through."""

    def __init__(self, size):
        self.size, self.ws, self.T, self.stream = size, None, -1, None
        self.in_graph, self.of_graphs = False, []

    def get(self, T, weight, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.get(T, weight)
        if T > self.T:
            n = self.size(T)
            if self.ws is None or n > self.ws.numel():
                if self.in_graph:
                    self.of_graphs.append(self.ws)
                self.ws, self.stream = alloc_workspace(n, weight.device), _raw_stream(None)
                self.in_graph = False
            self.T = T
        if torch.cuda.is_current_stream_capturing():
            self.in_graph = True
        elif _raw_stream(None) != self.stream:
            self.ws.record_stream(torch.cuda.current_stream())
        return self.ws


class MoELayer:
    """The user-facing layer: resident MXFP4 weights plus a reusable workspace.

    `forward(x, logits)` runs moe_forward on the current stream and returns the
    bf16 output [T, H].  Graphs captured with a layer keep its workspaces of that time: they may
    be replayed after longer steps."""

    def __init__(self, H, I, E, k, has_shared, w13, w13_s, w2, w2_s, fmt="mxfp4", w13_gs=None,
                 w2_gs=None, fuse_combine=False, fuse_swiglu=False, pair_tiles=False,
                 large_chunk_rows=0):
        if fmt not in ("mxfp4", "nvfp4"):
            raise ValueError(f"unknown weight format {fmt!r}")
        if (fuse_combine or fuse_swiglu or pair_tiles or large_chunk_rows) and fmt != "mxfp4":
            raise ValueError("the fusion and tile options take MXFP4 weights")
        self.fuse_combine = bool(fuse_combine)
        self.fuse_swiglu = bool(fuse_swiglu)
        self.pair_tiles = bool(pair_tiles)
        self.large_chunk_rows = int(large_chunk_rows)
        self.H, self.I, self.E, self.k, self.has_shared = H, I, E, k, has_shared
        self.w13, self.w13_s, self.w2, self.w2_s = w13, w13_s, w2, w2_s
        self.fmt, self.w13_gs, self.w2_gs = fmt, w13_gs, w2_gs
        self._ws = _LayerWorkspace(self._forward_size)
        self._hws = _LayerWorkspace(lambda T: host_workspace_size(self.dims(T)))
        self._tws, self._stages = _LayerWorkspace(self._forward_train_size), None
        self._bws = None

    def dims(self, T):
        return dims(T, self.H, self.I, self.E, self.k, self.has_shared)

    def _forward_size(self, T):
        size = (workspace_size if self.fmt == "mxfp4" else workspace_size_nvfp4)(self.dims(T))
        if size == 0:
            raise ValueError(f"unsupported dims for {self.fmt} weights")
        return size

    def workspace(self, T, stream=None):
        return self._ws.get(T, self.w13, stream)

    def _mxfp4_only(self, what):
        if self.fmt != "mxfp4":
            raise NotImplementedError(f"{what} takes MXFP4 weights")

    def host_workspace(self, T, stream=None):
        self._mxfp4_only("the host-buffer forward")
        return self._hws.get(T, self.w13, stream)

    def host_pipeline(self, T, depth=2):
        """A HostPipeline for T-token steps (its own workspace and streams)."""
        self._mxfp4_only("the host-buffer pipeline")
        return HostPipeline(self, T, depth)

    def forward_host(self, x_host, logits_host, out_host, stream=None):
        """End to end from host memory: x_host [T, H] bf16 and logits_host [T, E] fp32
        (pinned) in, out_host [T, H] bf16 (pinned) written when the stream reaches it."""
        T = x_host.shape[0]
        moe_forward_host(self.dims(T), x_host, logits_host, self.w13, self.w13_s, self.w2,
                         self.w2_s, out_host, self.host_workspace(T, stream), stream=stream)
        return out_host

    def host_graph(self, T):
        """A CUDA graph of forward_host on layer-owned pinned buffers (see HostGraph):
        one launch per step for the copies in, the layer's kernels and the copy out."""
        return HostGraph(self, T)

    def forward(self, x, logits, out=None, debug=None, stream=None):
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.H, dtype=torch.bfloat16, device=x.device)
        if self.fmt == "mxfp4":
            moe_forward_ex(self.dims(T), x, logits, self.w13, self.w13_s, self.w2, self.w2_s, out,
                           self.workspace(T, stream), fuse_combine=self.fuse_combine,
                           fuse_swiglu=self.fuse_swiglu, pair_tiles=self.pair_tiles,
                           large_chunk_rows=self.large_chunk_rows, debug=debug, stream=stream)
        else:
            moe_forward_nvfp4(self.dims(T), x, logits, self.w13, self.w13_s, self.w13_gs,
                              self.w2, self.w2_s, self.w2_gs, out, self.workspace(T, stream),
                              debug=debug, stream=stream)
        return out

    def _forward_train_size(self, T):
        d = self.dims(T)
        gemm = (gemm_workspace_size if self.fmt == "mxfp4" else gemm_workspace_size_nvfp4)(d)
        if gemm == 0:
            raise ValueError("unsupported dims")
        return max(route_workspace_size(d), 512 + gemm)  # (the stages': see forward_train)

    def _backward_workspace(self):
        """The gradient products' status word collects the bits of every step: made once, and
        zeroed before any other stream can have it (in a capture: by that graph's replays)."""
        if self._bws is None:
            self._bws = alloc_workspace(gemm_backward_workspace_size(self.dims(1)), self.w13.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(self.w13.device).synchronize()
        return self._bws

    def train_workspaces(self, T, stream=None):
        """The workspaces of forward_train and backward steps of up to T tokens (moe_check_status
        reads the checks of the last forward_train, and of every backward so far; where a capture
        was the first to ask for them, of every one since that graph's last replay began)."""
        with torch.cuda.stream(stream):
            return self._tws.get(T, self.w13), self._backward_workspace()

    def forward_train(self, x, logits, out=None, checkpoint="fp8", stream=None):
        """forward by its stages, keeping what backward needs.  Returns the output [T, H] and the
        step's state: routing (idx, w, inv, perm_src, offsets, counts) and the activations, in
        one of two forms:
          checkpoint="fp8"   the experts' inner activations in 8 bits (3 I bytes a row),
          checkpoint="bf16"  in bf16, with the experts' outputs (4 I + 2 H bytes a row).
        Steps of one layer share its workspaces: one at a time, as forward."""
        if checkpoint not in ("fp8", "bf16"):
            raise ValueError(f"unknown checkpoint form {checkpoint!r}")
        T, H, I, k, sh, E = x.shape[0], self.H, self.I, self.k, self.has_shared, self.E
        d, dev = self.dims(T), x.get_device()
        R, Rs = T * k, T * (k + sh)
        with torch.cuda.stream(stream):
            # (the stages take what they are given)
            _on(dev, x, _BF16, (T, H), "x"), _on(dev, logits, _F32, (T, E), "logits")
            _on(dev, out, _BF16, (T, H), "out"), _stream_on(dev, None)
            new = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=x.device)  # noqa: E731
            if out is None:
                out = new(T, H)
            # each stage clears its status word at its start: one each, joined at the end
            ws = self._tws.get(T, self.w13)
            if self._stages is None or self._stages[0].data_ptr() != ws.data_ptr():
                self._stages = stage_workspaces(ws, 3)
            stages = self._stages
            s = dict(T=T, idx=new(T, k, dt=_I32), w=new(T, k, dt=_F32), counts=new(E, dt=_I32),
                     offsets=new(E + sh + 1, dt=_I32), perm_src=new(R, dt=_I32),
                     inv=new(R, dt=_I32))
            moe_route(d, logits, s["idx"], s["w"], s["counts"], s["offsets"], s["perm_src"],
                      s["inv"], stages[0])
            xq, xs = new(T, H, dt=_U8), new(T, H // 128, dt=_U8)
            moe_quant_act(x, xq, xs)
            y13, y2 = new(Rs, 2 * I), new(Rs, H)
            nv = self.fmt != "mxfp4"
            if nv:
                moe_grouped_gemm_w13_nvfp4(d, xq, xs, s["perm_src"], s["offsets"], self.w13,
                                           self.w13_s, self.w13_gs, y13, stages[1])
            else:
                moe_grouped_gemm_w13(d, xq, xs, s["perm_src"], s["offsets"], self.w13, self.w13_s,
                                     y13, stages[1])
            hq, hs = new(Rs, I, dt=_U8), new(Rs, I // 128, dt=_U8)
            if checkpoint == "fp8":
                s |= dict(hq=hq, hs=hs, yq=new(Rs, 2 * I, dt=_U8),
                          ys=new(Rs, 2 * I // 128, dt=_U8))
                moe_swiglu_quant_save(y13, hq, hs, s["yq"], s["ys"])
            else:
                s |= dict(y13=y13, y2=y2)
                moe_swiglu_quant(y13, hq, hs)
            if nv:
                moe_grouped_gemm_w2_nvfp4(d, hq, hs, s["offsets"], self.w2, self.w2_s, self.w2_gs,
                                          y2, stages[2])
            else:
                moe_grouped_gemm_w2(d, hq, hs, s["offsets"], self.w2, self.w2_s, y2, stages[2])
            moe_combine(d, y2, s["inv"], s["w"], out)
            moe_join_status(stages[0], stages[1:])
        return out, s

    def backward(self, dout, saved, dx=None, dx_in=None, stream=None):
        """Gradient of forward_train from dout [T, H] bf16 and the state it returned (not
        changed).  Returns dx [T, H] (of dx's type where it is given, else bf16) = dx_in (the
        gradient that reaches x by other ways, or None) + the experts' part, and dw [T, k] fp32,
        the combine weights' gradient, which moe_balance_loss_backward takes to the logits.
        The experts' weights have none."""
        T, H, I = saved["T"], self.H, self.I
        d = self.dims(T)
        Rs = T * (self.k + self.has_shared)
        with torch.cuda.stream(stream):
            new = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dout.device)  # noqa: E731
            ws = self._backward_workspace()
            if dx is None:
                dx = new(T, H)
            rows, dh, dy13, dw = new(Rs, H), new(Rs, I), new(Rs, 2 * I), new(T, self.k, dt=_F32)
            if "yq" in saved:
                moe_dispatch(d, dout, saved["inv"], rows)
                act = dict(yq=saved["yq"], ys=saved["ys"], hq=saved["hq"], hs=saved["hs"],
                           perm_src=saved["perm_src"], w=saved["w"], dw=dw)
            else:
                moe_combine_backward(d, dout, saved["y2"], saved["inv"], saved["w"], dy2=rows,
                                     dw=dw)
                act = dict(y13=saved["y13"])
            off, nv = saved["offsets"], self.fmt != "mxfp4"
            if nv:
                moe_grouped_gemm_w2_backward_nvfp4(d, rows, off, self.w2, self.w2_s, self.w2_gs, dh,
                                                   ws)
            else:
                moe_grouped_gemm_w2_backward(d, rows, off, self.w2, self.w2_s, dh, ws)
            moe_swiglu_backward(dh, dy13, **act)
            if nv:
                moe_grouped_gemm_w13_backward_nvfp4(d, dy13, off, self.w13, self.w13_s, self.w13_gs,
                                                    rows, ws)
            else:
                moe_grouped_gemm_w13_backward(d, dy13, off, self.w13, self.w13_s, rows, ws)
            moe_dispatch_backward(d, rows, saved["inv"], dx, dx_in=dx_in)
        return dx, dw

    CHUNK_CANDIDATES = (224, 208, 192, 176, 160, 144)

    def tune_chunk_rows(self, x, logits, candidates=CHUNK_CANDIDATES, steps=10, warmup=3):
        """Exact-shape tuning of the tile plan on a recorded batch (its routing histogram
        decides the group sizes): times the layer with each candidate chunk size for
        groups above 64 rows (CUDA events, median of `steps` forwards after `warmup`),
        keeps the fastest in self.large_chunk_rows and returns (best, {candidate: ms}).
        Every candidate gives the same output bit for bit; only the tiling changes."""
        self._mxfp4_only("chunk-size tuning")
        out = torch.empty(x.shape[0], self.H, dtype=torch.bfloat16, device=x.device)
        times = {}
        keep = self.large_chunk_rows
        try:
            for c in candidates:
                self.large_chunk_rows = int(c)
                for _ in range(warmup):
                    self.forward(x, logits, out=out)
                ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
                      for _ in range(steps)]
                for a, b in ev:
                    a.record()
                    self.forward(x, logits, out=out)
                    b.record()
                torch.cuda.synchronize()
                ts = sorted(a.elapsed_time(b) for a, b in ev)
                times[int(c)] = ts[len(ts) // 2]
        except Exception:
            self.large_chunk_rows = keep
            raise
        best = min(times, key=times.get)
        self.large_chunk_rows = best
        return best, times

    def forward_timed(self, x, logits, out, events, stream=None):
        """forward recording the 8 stage events of moe_forward_timed (see STAGES)."""
        T = x.shape[0]
        if self.fmt == "mxfp4":
            moe_forward_ex(self.dims(T), x, logits, self.w13, self.w13_s, self.w2, self.w2_s, out,
                           self.workspace(T, stream), fuse_combine=self.fuse_combine,
                           fuse_swiglu=self.fuse_swiglu, pair_tiles=self.pair_tiles,
                           large_chunk_rows=self.large_chunk_rows, events=events,
                           stream=stream)
        else:
            moe_forward_nvfp4_timed(self.dims(T), x, logits, self.w13, self.w13_s, self.w13_gs,
                                    self.w2, self.w2_s, self.w2_gs, out, self.workspace(T, stream),
                                    events, stream=stream)
        return out
