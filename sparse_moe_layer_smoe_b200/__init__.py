"""Python binding for libstepmoe: the C-ABI of include/stepmoe.h, same names, argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module only turns torch
tensors (or raw integers) into pointers and checks the returned status. PyTorch supplies
device memory and streams. If ``libstepmoe.so`` is missing the binding raises: there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import re
import warnings
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstepmoe.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "stepmoe.h")

STATUS = {0: "SMOE_OK", 1: "SMOE_ERR_INVALID_ARG", 2: "SMOE_ERR_UNSUPPORTED", 3: "SMOE_ERR_WORKSPACE",
          4: "SMOE_ERR_CUDA", 5: "SMOE_ERR_DEVICE", 6: "SMOE_ERR_TIMEOUT"}
SMOE_OK, SMOE_ERR_INVALID_ARG, SMOE_ERR_UNSUPPORTED, SMOE_ERR_WORKSPACE = 0, 1, 2, 3
SMOE_ERR_CUDA, SMOE_ERR_DEVICE, SMOE_ERR_TIMEOUT = 4, 5, 6
SMOE_NOALLOC_SCRATCH_BYTES = 16 << 20   # include/stepmoe.h: the allocation-free router's static scratch


class SmoeConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32), ("route_scale", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float), ("swiglu_limit_shared", ctypes.c_float)]


class SmoeError(RuntimeError):
    def __init__(self, fn: str, status: int, why: str = ""):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}" + (f": {why}" if why else ""))
        self.status = status


def config(hidden=4096, n_experts=288, top_k=8, inter=1280, shared_inter=1280, route_scale=3.0,
           swiglu_limit=0.0, swiglu_limit_shared=0.0) -> SmoeConfig:
    return SmoeConfig(hidden, n_experts, top_k, inter, shared_inter, route_scale, swiglu_limit, swiglu_limit_shared)


class SmoeKernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_float)]


class SmoeDiag(ctypes.Structure):
    """smoe_diag_t: device pointers of the monitoring outputs (see include/stepmoe.h)."""
    _fields_ = [("expert_count", ctypes.c_void_p), ("expert_norm_mean", ctypes.c_void_p),
                ("expert_norm_max", ctypes.c_void_p), ("token_confidence", ctypes.c_void_p),
                ("summary", ctypes.c_void_p)]


# indices into smoe_diag_t.summary
(SMOE_DIAG_ACTIVE_EXPERTS, SMOE_DIAG_NORM_MEDIAN, SMOE_DIAG_NORM_MAX_TO_MEDIAN, SMOE_DIAG_NORM_MIN_TO_MEDIAN,
 SMOE_DIAG_CONF_MEAN, SMOE_DIAG_CONF_MIN, SMOE_DIAG_LOAD_MAX_TO_MEAN, SMOE_DIAG_NORM_PEAK, SMOE_DIAG_SUMMARY) = range(9)
DIAG_FIELDS = ("expert_count", "expert_norm_mean", "expert_norm_max", "token_confidence", "summary")


_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_cfgp = ctypes.POINTER(SmoeConfig)
_SIGS = {
    "smoe_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "smoe_check_config": ([_cfgp], ctypes.c_int),
    "smoe_scratch_bytes": ([_cfgp, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_workspace_bytes": ([_cfgp, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_packed_weight_bytes": ([_cfgp, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_pack_weights": ([_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "smoe_route": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_permute": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_expert_ffn": ([_cfgp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_combine": ([_cfgp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_forward": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_forward_diag": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(SmoeDiag), _vp, _sz, _vp],
                          ctypes.c_int),
    "smoe_get_device_error": ([_vp, ctypes.POINTER(ctypes.c_int32), _vp], ctypes.c_int),
    "smoe_clear_device_error": ([_vp, _vp], ctypes.c_int),
    "smoe_last_launch_count": ([], ctypes.c_int32),
    "smoe_timing_begin": ([ctypes.c_int32], ctypes.c_int),
    "smoe_timing_end": ([ctypes.POINTER(SmoeKernelTime), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
                        ctypes.c_int),
    "smoe_route_noalloc": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "smoe_packed_weight_bytes_fp8": ([_cfgp, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_pack_weights_fp8": ([_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "smoe_workspace_bytes_fp8": ([_cfgp, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_forward_fp8": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_backward_bytes": ([_cfgp, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "smoe_expert_ffn_save": ([_cfgp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_checkpoint_values": ([_cfgp, _vp, _vp, _i64, _vp, _vp], ctypes.c_int),
    "smoe_combine_backward": ([_cfgp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_route_backward": ([_cfgp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
                            ctypes.c_int),
    "smoe_expert_ffn_backward": ([_cfgp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_permute_backward": ([_cfgp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
    "smoe_selftest_wait_timeout": ([ctypes.c_uint64, _vp, _vp, _vp], ctypes.c_int),
    "smoe_selftest_swiglu": ([_vp, _vp, _i64, _vp, _vp], ctypes.c_int),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libstepmoe.so (built in-tree). Raises if it is missing: the layer has no other path."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with sparse_moe_layer_smoe_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/stepmoe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^SMOE_API\s+[\w\s\*]*?\b(smoe_\w+)\s*\(", text, flags=re.M)


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_cuda = None   # torch's current device and, by device, the current stream as an integer (a torch.cuda.Stream
               # object costs 3 us a call)


def _current():
    global _cuda
    if _cuda is None:
        import torch
        _cuda = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream
    return _cuda


def _s(stream) -> int | None:
    if stream is None:
        device, raw_stream = _current()
        return raw_stream(device()) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _check(name: str, status: int) -> None:
    if status != SMOE_OK:
        raise SmoeError(name, status)


def _bytes(fn, cfg, *args) -> int:
    out = _sz(0)
    _check(fn.__name__, fn(ctypes.byref(cfg), *args, ctypes.byref(out)))
    return out.value


# ------------------------------------------------------------------------------ same-name wrappers
def smoe_status_string(status: int) -> str:
    return lib().smoe_status_string(status).decode()


def smoe_check_config(cfg: SmoeConfig) -> int:
    return lib().smoe_check_config(ctypes.byref(cfg))


def smoe_scratch_bytes(cfg: SmoeConfig, T: int) -> int:
    return _bytes(lib().smoe_scratch_bytes, cfg, T)


def smoe_workspace_bytes(cfg: SmoeConfig, T: int) -> int:
    return _bytes(lib().smoe_workspace_bytes, cfg, T)


def smoe_packed_weight_bytes(cfg: SmoeConfig) -> int:
    return _bytes(lib().smoe_packed_weight_bytes, cfg)


def smoe_pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed, stream=None) -> None:
    _check("smoe_pack_weights", lib().smoe_pack_weights(ctypes.byref(cfg), _p(w_gate), _p(w_up), _p(w_down),
                                                         _p(ws_gate), _p(ws_up), _p(ws_down), _p(packed), _s(stream)))


def smoe_route(cfg, x, T, w_router, bias, topk_idx, topk_w, logits=None, ws=None, ws_bytes=None, stream=None):
    _check("smoe_route", lib().smoe_route(ctypes.byref(cfg), _p(x), T, _p(w_router), _p(bias), _p(topk_idx),
                                          _p(topk_w), _p(logits), _p(ws), _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_route_noalloc(cfg, x, T, w_router, bias, topk_idx, topk_w, logits=None, stream=None):
    """smoe_route without a workspace (library-owned static scratch; see include/stepmoe.h)."""
    _check("smoe_route_noalloc", lib().smoe_route_noalloc(ctypes.byref(cfg), _p(x), T, _p(w_router), _p(bias),
                                                          _p(topk_idx), _p(topk_w), _p(logits), _s(stream)))


def smoe_permute(cfg, topk_idx, T, x, counts, offsets, perm_row, row_token, x_perm, ws=None, ws_bytes=None,
                 stream=None):
    _check("smoe_permute", lib().smoe_permute(ctypes.byref(cfg), _p(topk_idx), T, _p(x), _p(counts), _p(offsets),
                                              _p(perm_row), _p(row_token), _p(x_perm), _p(ws),
                                              _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_expert_ffn(cfg, x, x_perm, row_token, offsets, T, packed, y, ws=None, ws_bytes=None, stream=None):
    _check("smoe_expert_ffn", lib().smoe_expert_ffn(ctypes.byref(cfg), _p(x), _p(x_perm), _p(row_token),
                                                    _p(offsets), T, _p(packed), _p(y), _p(ws),
                                                    _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_combine(cfg, y, perm_row, topk_w, T, out, ws=None, ws_bytes=None, stream=None):
    _check("smoe_combine", lib().smoe_combine(ctypes.byref(cfg), _p(y), _p(perm_row), _p(topk_w), T, _p(out),
                                              _p(ws), _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_forward(cfg, x, T, w_router, bias, packed, out, ws=None, ws_bytes=None, stream=None):
    _check("smoe_forward", lib().smoe_forward(ctypes.byref(cfg), _p(x), T, _p(w_router), _p(bias), _p(packed),
                                              _p(out), _p(ws), _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_forward_diag(cfg, x, T, w_router, bias, packed, out, diag, ws=None, ws_bytes=None, stream=None):
    """diag: a mapping with the smoe_diag_t fields (device tensors), e.g. from diag_buffers()."""
    d = SmoeDiag(*[_p(diag[f]) for f in DIAG_FIELDS])
    _check("smoe_forward_diag", lib().smoe_forward_diag(ctypes.byref(cfg), _p(x), T, _p(w_router), _p(bias),
                                                        _p(packed), _p(out), ctypes.byref(d), _p(ws),
                                                        _ws_bytes(ws, ws_bytes), _s(stream)))


def smoe_packed_weight_bytes_fp8(cfg: SmoeConfig) -> int:
    return _bytes(lib().smoe_packed_weight_bytes_fp8, cfg)


def smoe_workspace_bytes_fp8(cfg: SmoeConfig, T: int) -> int:
    return _bytes(lib().smoe_workspace_bytes_fp8, cfg, T)


def smoe_pack_weights_fp8(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed, stream=None) -> None:
    _check("smoe_pack_weights_fp8", lib().smoe_pack_weights_fp8(ctypes.byref(cfg), _p(w_gate), _p(w_up), _p(w_down),
                                                                 _p(ws_gate), _p(ws_up), _p(ws_down), _p(packed),
                                                                 _s(stream)))


def smoe_forward_fp8(cfg, x, T, w_router, bias, packed_fp8, out, ws=None, ws_bytes=None, stream=None):
    _check("smoe_forward_fp8", lib().smoe_forward_fp8(ctypes.byref(cfg), _p(x), T, _p(w_router), _p(bias),
                                                      _p(packed_fp8), _p(out), _p(ws), _ws_bytes(ws, ws_bytes),
                                                      _s(stream)))


_dtypes = {}   # name -> torch dtype, filled on the first checked call


def _arguments(fn: str, T: int, ws, ws_bytes, stream, *args) -> list:
    """The pointers of (name, tensor, dtype, n) arguments, given flat, then the workspace's pointer and bytes and the
    stream. A torch tensor must hold at least n elements of that type, contiguous, on the current CUDA device
    (whose current stream the call goes to); the workspace too must be there. With dtype None the type does not
    matter and n is in bytes. Raw pointers and None are passed on as they are: the library checks them."""
    if not _dtypes:
        import torch
        _dtypes.update({n: getattr(torch, n) for n in ("bfloat16", "float32", "int32", "uint8")})
    here = _current()[0]() if T > 0 else None
    out = []
    for name, t, dtype, n in zip(*(iter((*args, "ws", ws, None, 0)),) * 4):
        if t is None or type(t) is int:
            out.append(t)
            continue
        why = None
        if dtype is not None and t.dtype is not _dtypes[dtype]:
            why = f"{name} is {t.dtype}, not torch.{dtype}"
        elif not t.is_contiguous():
            why = f"{name} is not contiguous"
        elif dtype is not None and t.numel() < n:
            why = f"{name} has {t.numel()} elements, {n} are needed"
        elif dtype is None and t.numel() * t.element_size() < n:
            why = f"{name} has {t.numel() * t.element_size()} bytes, {n} are needed"
        elif here is not None and t.get_device() != here:
            why = f"{name} is on {t.device}, the call runs on cuda:{here}"
        if why:
            raise SmoeError(fn, SMOE_ERR_INVALID_ARG, why)
        out.append(t.data_ptr())
    return [*out, _ws_bytes(ws, ws_bytes), _s(stream) if T > 0 or stream is not None else _stream_or_default()]


def _packed_bytes(cfg) -> int:
    """smoe_packed_weight_bytes, without its check of the config (which the calls make themselves)."""
    return (cfg.n_experts + 1) * 3 * cfg.inter * cfg.hidden * 2


def _stream_or_default():
    """The current stream, or the default one where there is no CUDA device (calls with T == 0)."""
    import torch
    return _s(None) if torch.cuda.is_available() else None


_native = None   # the _pyargs module, or what stands in for it


class _LeavesAll:
    """Stands in for the native module where it cannot be loaded: every call is left to Python."""
    def __getattr__(self, name):
        return lambda *args: None


def _load_native():
    """The training calls in C++ (csrc/pyargs.cpp). Each takes the arguments of the function below of the same
    name and returns the library's status, or None where it leaves the call to that function. The module is built
    for one Python and one torch; under others the functions below make the calls, a few us slower."""
    global _native
    functions = [ctypes.cast(getattr(lib(), f), _vp).value for f in (
        "smoe_expert_ffn_save", "smoe_checkpoint_values", "smoe_combine_backward", "smoe_route_backward",
        "smoe_expert_ffn_backward", "smoe_permute_backward")]
    try:
        import torch  # noqa: F401  (the module links against its libraries)
        from . import _pyargs
    except ImportError as e:
        warnings.warn(f"the native training calls cannot be loaded ({e}); calling through Python. Rebuild them with "
                      "sparse_moe_layer_smoe_b200.build.build_pyargs()", RuntimeWarning, stacklevel=3)
        _native = _LeavesAll()
        return _native
    _pyargs.use(*functions)
    _native = _pyargs
    return _pyargs


def smoe_backward_bytes(cfg: SmoeConfig, T: int) -> int:
    return _bytes(lib().smoe_backward_bytes, cfg, T)


def smoe_expert_ffn_save(cfg, x, x_perm, row_token, offsets, T, packed, y, gu_q, gu_scale, ws=None, ws_bytes=None,
                         stream=None):
    """smoe_expert_ffn with the 8-bit checkpoint of the gate and up products (see include/stepmoe.h)."""
    status = (_native or _load_native()).expert_ffn_save(
        cfg, x, x_perm, row_token, offsets, T, packed, y, gu_q, gu_scale, ws, ws_bytes, stream)
    if status is None:
        H, I, R = cfg.hidden, cfg.inter, T * cfg.top_k
        p = _arguments("smoe_expert_ffn_save", T, ws, ws_bytes, stream,
                       "x", x, "bfloat16", T * H, "x_perm", x_perm, "bfloat16", R * H,
                       "row_token", row_token, "int32", R, "offsets", offsets, "int32", cfg.n_experts + 1,
                       "packed", packed, None, _packed_bytes(cfg), "y", y, "bfloat16", (R + T) * H, "gu_q", gu_q, "uint8", (R + T) * 2 * I,
                       "gu_scale", gu_scale, "uint8", 2 * I // 32 * (R + T))
        status = lib().smoe_expert_ffn_save(ctypes.byref(cfg), *p[:4], T, *p[4:])
    _check("smoe_expert_ffn_save", status)


def smoe_checkpoint_values(cfg, gu_q, gu_scale, T, gu, stream=None):
    """The bf16 values a checkpoint stands for."""
    status = (_native or _load_native()).checkpoint_values(cfg, gu_q, gu_scale, T, gu, stream)
    if status is None:
        I, rows = cfg.inter, T * cfg.top_k + T
        p = _arguments("smoe_checkpoint_values", T, None, None, stream,
                       "gu_q", gu_q, "uint8", rows * 2 * I,
                       "gu_scale", gu_scale, "uint8", 2 * I // 32 * rows, "gu", gu, "bfloat16", rows * 2 * I)
        status = lib().smoe_checkpoint_values(ctypes.byref(cfg), p[0], p[1], T, p[2], p[5])
    _check("smoe_checkpoint_values", status)


def smoe_combine_backward(cfg, dout, y, perm_row, topk_w, T, dy, dtopk_w, ws=None, ws_bytes=None, stream=None):
    status = (_native or _load_native()).combine_backward(
        cfg, dout, y, perm_row, topk_w, T, dy, dtopk_w, ws, ws_bytes, stream)
    if status is None:
        H, R = cfg.hidden, T * cfg.top_k
        p = _arguments("smoe_combine_backward", T, ws, ws_bytes, stream,
                       "dout", dout, "bfloat16", T * H, "y", y, "bfloat16", (R + T) * H,
                       "perm_row", perm_row, "int32", R, "topk_w", topk_w, "float32", R, "dy", dy, "bfloat16", R * H,
                       "dtopk_w", dtopk_w, "float32", R)
        status = lib().smoe_combine_backward(ctypes.byref(cfg), *p[:4], T, *p[4:])
    _check("smoe_combine_backward", status)


def smoe_route_backward(cfg, x, T, logits, topk_idx, topk_w, dtopk_w, offsets, perm_row, row_token, dlogits, dw_router,
                        ws=None, ws_bytes=None, stream=None):
    status = (_native or _load_native()).route_backward(
        cfg, x, T, logits, topk_idx, topk_w, dtopk_w, offsets, perm_row, row_token, dlogits, dw_router, ws, ws_bytes,
        stream)
    if status is None:
        H, E, R = cfg.hidden, cfg.n_experts, T * cfg.top_k
        p = _arguments("smoe_route_backward", T, ws, ws_bytes, stream,
                       "x", x, "bfloat16", T * H, "logits", logits, "float32", T * E,
                       "topk_idx", topk_idx, "int32", R, "topk_w", topk_w, "float32", R,
                       "dtopk_w", dtopk_w, "float32", R, "offsets", offsets, "int32", E + 1,
                       "perm_row", perm_row, "int32", R, "row_token", row_token, "int32", R,
                       "dlogits", dlogits, "float32", R, "dw_router", dw_router, "float32", E * H)
        status = lib().smoe_route_backward(ctypes.byref(cfg), p[0], T, *p[1:])
    _check("smoe_route_backward", status)


def smoe_expert_ffn_backward(cfg, x, x_perm, offsets, T, packed, gu_q, gu_scale, dy, dout, dx_rows, dw_gate, dw_up,
                             dw_down, dws_gate, dws_up, dws_down, ws=None, ws_bytes=None, stream=None):
    status = (_native or _load_native()).expert_ffn_backward(
        cfg, x, x_perm, offsets, T, packed, gu_q, gu_scale, dy, dout, dx_rows, dw_gate, dw_up, dw_down, dws_gate,
        dws_up, dws_down, ws, ws_bytes, stream)
    if status is None:
        H, E, I, R = cfg.hidden, cfg.n_experts, cfg.inter, T * cfg.top_k
        w = H * I
        p = _arguments("smoe_expert_ffn_backward", T, ws, ws_bytes, stream,
                       "x", x, "bfloat16", T * H, "x_perm", x_perm, "bfloat16", R * H,
                       "offsets", offsets, "int32", E + 1, "packed", packed, None, _packed_bytes(cfg),
                       "gu_q", gu_q, "uint8", (R + T) * 2 * I,
                       "gu_scale", gu_scale, "uint8", 2 * I // 32 * (R + T), "dy", dy, "bfloat16", R * H,
                       "dout", dout, "bfloat16", T * H, "dx_rows", dx_rows, "bfloat16", (R + T) * H,
                       "dw_gate", dw_gate, "bfloat16", E * w, "dw_up", dw_up, "bfloat16", E * w,
                       "dw_down", dw_down, "bfloat16", E * w, "dws_gate", dws_gate, "bfloat16", w,
                       "dws_up", dws_up, "bfloat16", w, "dws_down", dws_down, "bfloat16", w)
        status = lib().smoe_expert_ffn_backward(ctypes.byref(cfg), *p[:3], T, *p[3:])
    _check("smoe_expert_ffn_backward", status)


def smoe_permute_backward(cfg, dx_rows, perm_row, topk_idx, dlogits, w_router, T, dx, ws=None, ws_bytes=None,
                          stream=None):
    status = (_native or _load_native()).permute_backward(
        cfg, dx_rows, perm_row, topk_idx, dlogits, w_router, T, dx, ws, ws_bytes, stream)
    if status is None:
        H, E, R = cfg.hidden, cfg.n_experts, T * cfg.top_k
        p = _arguments("smoe_permute_backward", T, ws, ws_bytes, stream,
                       "dx_rows", dx_rows, "bfloat16", (R + T) * H,
                       "perm_row", perm_row, "int32", R, "topk_idx", topk_idx, "int32", R,
                       "dlogits", dlogits, "float32", R, "w_router", w_router, "float32", E * H,
                       "dx", dx, "bfloat16", T * H)
        status = lib().smoe_permute_backward(ctypes.byref(cfg), *p[:5], T, *p[5:])
    _check("smoe_permute_backward", status)


def smoe_selftest_swiglu(g, u, n, out, stream=None) -> None:
    """The expert epilogue's SiLU(g) * u (see include/stepmoe.h)."""
    _check("smoe_selftest_swiglu", lib().smoe_selftest_swiglu(_p(g), _p(u), int(n), _p(out), _s(stream)))


def smoe_selftest_wait_timeout(limit_ns, elapsed_ns=None, ws=None, stream=None) -> None:
    _check("smoe_selftest_wait_timeout", lib().smoe_selftest_wait_timeout(int(limit_ns), _p(elapsed_ns), _p(ws),
                                                                          _s(stream)))


def smoe_get_device_error(ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check("smoe_get_device_error", lib().smoe_get_device_error(_p(ws), ctypes.byref(code), _s(stream)))
    return code.value


def smoe_clear_device_error(ws, stream=None) -> None:
    _check("smoe_clear_device_error", lib().smoe_clear_device_error(_p(ws), _s(stream)))


def smoe_last_launch_count() -> int:
    return int(lib().smoe_last_launch_count())


def smoe_timing_begin(max_launches: int) -> None:
    _check("smoe_timing_begin", lib().smoe_timing_begin(max_launches))


def smoe_timing_end() -> dict:
    """{kernel name: (launches, total_ms)} for the launches recorded since smoe_timing_begin."""
    buf = (SmoeKernelTime * 64)()
    n = ctypes.c_int32(0)
    _check("smoe_timing_end", lib().smoe_timing_end(buf, 64, ctypes.byref(n)))
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(n.value)}


def _ws_bytes(ws, ws_bytes) -> int:
    if ws_bytes is not None:
        return int(ws_bytes)
    if ws is None or isinstance(ws, int):
        return 0
    return ws.numel() * ws.element_size()


# ------------------------------------------------------------------------------ conveniences (torch memory)
def workspace(cfg: SmoeConfig, T: int, forward: bool = True, device="cuda", fp8: bool = False,
              backward: bool = False):
    """A zeroed uint8 CUDA tensor large enough for smoe_forward (smoe_forward_fp8 with fp8=True,
    or the per-call entry points with forward=False). With backward=True: for the per-call entry points
    of a training step, forward and backward."""
    import torch
    if backward:
        n = max(smoe_scratch_bytes(cfg, T), smoe_backward_bytes(cfg, T))
    elif fp8:
        n = smoe_workspace_bytes_fp8(cfg, T)
    else:
        n = smoe_workspace_bytes(cfg, T) if forward else smoe_scratch_bytes(cfg, T)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _stream_context(stream):
    """torch.cuda.stream(stream); stream may be None (the current one) or a raw handle."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def diag_buffers(cfg: SmoeConfig, T: int, device="cuda") -> dict:
    """Device arrays for smoe_forward_diag's outputs."""
    import torch
    E = cfg.n_experts
    return {"expert_count": torch.empty(E, dtype=torch.int32, device=device),
            "expert_norm_mean": torch.empty(E, dtype=torch.float32, device=device),
            "expert_norm_max": torch.empty(E, dtype=torch.float32, device=device),
            "token_confidence": torch.empty(max(T, 1), dtype=torch.float32, device=device),
            "summary": torch.empty(SMOE_DIAG_SUMMARY, dtype=torch.float32, device=device)}


def pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, stream=None):
    import torch
    packed = torch.empty(smoe_packed_weight_bytes(cfg), dtype=torch.uint8, device=w_gate.device)
    smoe_pack_weights(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed, stream)
    return packed


def pack_weights_fp8(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, stream=None):
    import torch
    packed = torch.empty(smoe_packed_weight_bytes_fp8(cfg), dtype=torch.uint8, device=w_gate.device)
    smoe_pack_weights_fp8(cfg, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, packed, stream)
    return packed


@dataclass
class MoELayer:
    """Parameters of one layer on the device: fp32 router weights and bias, packed bf16 experts."""
    cfg: SmoeConfig
    w_router: object
    bias: object
    packed: object

    def forward(self, x, out=None, ws=None, stream=None):
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.cfg.hidden, dtype=torch.bfloat16, device=x.device)
        if ws is None:
            ws = workspace(self.cfg, T, device=x.device)
        smoe_forward(self.cfg, x, T, self.w_router, self.bias, self.packed, out, ws, stream=stream)
        return out

    def forward_train(self, x, ws=None, stream=None):
        """The layer's output for x [T, hidden], and what backward() needs of this step (in 8 bits: the experts'
        gate and up products; x itself, which like the layer's weights must stay as it is until then). ws: workspace(cfg, T, backward=True), which steps may share one after another.
        stream: as under torch.cuda.stream(stream), so what is returned belongs to that stream."""
        with _stream_context(stream):
            return self._forward_train(x, ws)

    def _forward_train(self, x, ws):
        import torch
        cfg, T = self.cfg, x.shape[0]
        E, k, H, I = cfg.n_experts, cfg.top_k, cfg.hidden, cfg.inter
        R = T * k

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=x.device)

        if tuple(x.shape) != (T, H):
            raise SmoeError("forward_train", SMOE_ERR_INVALID_ARG, f"x is {tuple(x.shape)}, not (T, {H})")
        if ws is None:
            ws = workspace(cfg, T, device=x.device, backward=True)
        _arguments("forward_train", T, ws, None, None, "x", x, "bfloat16", T * H, "w_router", self.w_router, "float32",
                   E * H, "bias", self.bias, "float32", E, "packed", self.packed, None, _packed_bytes(cfg))
        s = {"x": x, "topk_idx": new(T, k, dtype=torch.int32), "topk_w": new(T, k, dtype=torch.float32),
             "logits": new(T, E, dtype=torch.float32),
             "offsets": torch.zeros(E + 1, dtype=torch.int32, device=x.device),
             "perm_row": new(R, dtype=torch.int32), "row_token": new(R, dtype=torch.int32), "x_perm": new(R, H),
             "y": new(R + T, H), "gu_q": new(R + T, 2 * I, dtype=torch.uint8),
             "gu_scale": new(2 * I // 32, R + T, dtype=torch.uint8)}
        out, counts = new(T, H), new(E, dtype=torch.int32)
        smoe_route(cfg, x, T, self.w_router, self.bias, s["topk_idx"], s["topk_w"], s["logits"], ws=ws)
        smoe_permute(cfg, s["topk_idx"], T, x, counts, s["offsets"], s["perm_row"], s["row_token"], s["x_perm"], ws=ws)
        smoe_expert_ffn_save(cfg, x, s["x_perm"], s["row_token"], s["offsets"], T, self.packed, s["y"], s["gu_q"],
                             s["gu_scale"], ws=ws)
        smoe_combine(cfg, s["y"], s["perm_row"], s["topk_w"], T, out, ws=ws)
        return out, s

    def backward(self, saved, dout, ws=None, stream=None) -> dict:
        """Gradients of <dout, output> of the step that forward_train saved: dx, dw_router, and the experts'
        dw_gate, dw_up, dw_down, dws_gate, dws_up, dws_down (layouts of pack_weights' inputs). stream: as in
        forward_train."""
        with _stream_context(stream):
            return self._backward(saved, dout, ws)

    def _backward(self, s, dout, ws):
        import torch
        cfg, T = self.cfg, dout.shape[0]
        E, k, H, I = cfg.n_experts, cfg.top_k, cfg.hidden, cfg.inter
        R = T * k

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dout.device)

        if dout.shape != s["x"].shape:
            raise SmoeError("backward", SMOE_ERR_INVALID_ARG,
                            f"dout is {tuple(dout.shape)}, the saved step's output {tuple(s['x'].shape)}")
        if ws is None:
            ws = workspace(cfg, T, device=dout.device, backward=True)
        dy, dtopk_w, dlogits = new(R, H), new(T, k, dtype=torch.float32), new(T, k, dtype=torch.float32)
        dx_rows = new(R + T, H)
        g = {"dx": new(T, H), "dw_router": new(E, H, dtype=torch.float32), "dw_gate": new(E, I, H),
             "dw_up": new(E, I, H), "dw_down": new(E, H, I), "dws_gate": new(I, H), "dws_up": new(I, H),
             "dws_down": new(H, I)}
        smoe_combine_backward(cfg, dout, s["y"], s["perm_row"], s["topk_w"], T, dy, dtopk_w, ws=ws)
        smoe_expert_ffn_backward(cfg, s["x"], s["x_perm"], s["offsets"], T, self.packed, s["gu_q"], s["gu_scale"], dy,
                                 dout, dx_rows, g["dw_gate"], g["dw_up"], g["dw_down"], g["dws_gate"], g["dws_up"],
                                 g["dws_down"], ws=ws)
        smoe_route_backward(cfg, s["x"], T, s["logits"], s["topk_idx"], s["topk_w"], dtopk_w, s["offsets"],
                            s["perm_row"], s["row_token"], dlogits, g["dw_router"], ws=ws)
        smoe_permute_backward(cfg, dx_rows, s["perm_row"], s["topk_idx"], dlogits, self.w_router, T, g["dx"], ws=ws)
        return g
