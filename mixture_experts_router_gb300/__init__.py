"""Python binding of libcbmoe.so, the GB300 MoE FFN layer (C ABI in include/cb_moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch is used by callers for device memory and streams; this module
takes raw pointers (ints) or torch tensors and forwards them.  There is no
fallback: if the shared library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcbmoe.so")

CB_OK, CB_ERR_INVALID_ARG, CB_ERR_UNSUPPORTED, CB_ERR_ALIGNMENT = 0, 1, 2, 3
CB_ERR_OOM, CB_ERR_CUDA, CB_ERR_TIMEOUT, CB_ERR_DEVICE = 4, 5, 6, 7
CB_W_BF16, CB_W_INT8, CB_W_INT4, CB_W_FP8 = 0, 1, 2, 3
WDTYPES = {"bf16": CB_W_BF16, "int8": CB_W_INT8, "int4": CB_W_INT4, "fp8": CB_W_FP8}
CB_FLAG_KEEP_LOGITS = 0x1
CB_FLAG_STAGE_TIMING = 0x2
CB_FLAG_TEST_STALL = 0x4
CB_FLAG_TEST_STALL_DISPATCH = 0x8
CB_FLAG_GUARDS = 0x10
CB_N_STAGES = 5
STAGE_NAMES = ("router", "dispatch", "gateup_gemm", "down_gemm", "combine")

# every symbol include/cb_moe.h declares
ABI_SYMBOLS = ("cb_moe_init", "cb_moe_forward", "cb_moe_forward_f32out", "cb_moe_forward_host",
               "cb_moe_routing", "cb_moe_stage_times", "cb_moe_last_error", "cb_moe_device_bytes",
               "cb_moe_free", "cb_status_string", "cb_moe_dispatch_noalloc", "cb_moe_kernels_per_forward",
               "cb_moe_set_stage_timing", "cb_moe_check_guards", "cb_moe_forward_few", "cb_moe_forward_few_f32out",
               "cb_moe_forward_routed", "cb_moe_forward_routed_f32out", "cb_moe_forward_few_routed",
               "cb_moe_forward_few_routed_f32out")


CB_MOE_MAX_FEW = 16
# every symbol include/cb_fp4.h declares
FP4_SYMBOLS = ("cb_fp4_scale_bytes", "cb_fp4_quantize", "cb_fp4_dequantize", "cb_fp4_matmul", "cb_fp4_last_error")
CB_FP4_MX, CB_FP4_NV = 0, 1
CB_T_BF16, CB_T_F32 = 0, 1
FP4_FORMATS = {"mx": CB_FP4_MX, "nv": CB_FP4_NV}
FP4_BLOCK = {"mx": 32, "nv": 16}
# every symbol include/cb_serve.h declares
SERVE_SYMBOLS = ("cb_rms_norm", "cb_route", "cb_int4_matmul_few")
CB_NORM_MAX_COLS, CB_FP8_COLS, CB_ROUTE_MAX_GROUPS = 32768, 128, 32
CB_INT4_MAX_ROWS, CB_INT4_MAX_K = CB_MOE_MAX_FEW, 49152
CB_SCORE_SIGMOID, CB_SCORE_SOFTMAX = 0, 1
CB_GROUP_TOP2, CB_GROUP_MAX = 0, 1
SCORES = {"sigmoid": CB_SCORE_SIGMOID, "softmax": CB_SCORE_SOFTMAX}
GROUP_SCORES = {"top2": CB_GROUP_TOP2, "max": CB_GROUP_MAX}
CB_ROUTER_SOFTMAX_TOPK, CB_ROUTER_RAW_LOGITS, CB_ROUTER_HASH = 0, 1, 2
CB_MAX_HASH_DIMS = 8
ROUTER_MODES = {"softmax": CB_ROUTER_SOFTMAX_TOPK, "raw": CB_ROUTER_RAW_LOGITS, "hash": CB_ROUTER_HASH}


class cb_moe_config_t(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("wdtype", ctypes.c_int32),
                ("device", ctypes.c_int32), ("flags", ctypes.c_uint32), ("router_mode", ctypes.c_int32),
                ("hash_dims", ctypes.c_int32)]


class cb_moe_weights_t(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("w_hash", ctypes.c_void_p),
                ("z_gate", ctypes.c_void_p), ("z_up", ctypes.c_void_p), ("z_down", ctypes.c_void_p)]


class cb_routing_view_t(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("tok", ctypes.c_void_p), ("inv", ctypes.c_void_p),
                ("logits", ctypes.c_void_p), ("tile_offsets", ctypes.c_void_p)]


class cb_fp4_matmul_t(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("a_codes", ctypes.c_void_p), ("a_scales", ctypes.c_void_p), ("a_tensor_scale", ctypes.c_void_p),
                ("b_codes", ctypes.c_void_p), ("b_scales", ctypes.c_void_p), ("b_tensor_scale", ctypes.c_void_p),
                ("n_groups", ctypes.c_int32), ("tile_offsets", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("status", ctypes.c_void_p)]


_FP4_MATMUL = struct.Struct("@2i3q6Pi4xPPqP")  # cb_fp4_matmul_t
assert _FP4_MATMUL.size == ctypes.sizeof(cb_fp4_matmul_t)


class cb_rms_norm_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("sum", ctypes.c_void_p), ("ld_sum", ctypes.c_int64), ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("x_type", ctypes.c_int32), ("weight_type", ctypes.c_int32), ("out_type", ctypes.c_int32)]


class cb_route_t(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("logits", ctypes.c_void_p), ("ld_logits", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("logits_type", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalise", ctypes.c_int32)]


class cb_int4_matmul_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("ld_x", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("n_tokens", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("group", ctypes.c_int32), ("x_per_slot", ctypes.c_int32), ("swiglu", ctypes.c_int32),
                ("out_type", ctypes.c_int32)]


# the same layouts for calls that are made every few microseconds
_RMS_NORM, _ROUTE, _INT4 = struct.Struct("@2qPqPqPPqPqPPf3i"), struct.Struct("@qPq3Pf8i4x"), struct.Struct("@9P4q7i4x")
for _s, _t in ((_RMS_NORM, cb_rms_norm_t), (_ROUTE, cb_route_t), (_INT4, cb_int4_matmul_t)):
    assert _s.size == ctypes.sizeof(_t), _t


class CbMoeError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {cb_status_string(status)} (status {status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libcbmoe.so (build it first with __graft_entry__.build() or build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libcbmoe.so is not built ({path}); run mixture_experts_router_gb300/build.py")
    lib = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.cb_moe_init.argtypes = [ctypes.POINTER(cb_moe_config_t), ctypes.POINTER(cb_moe_weights_t),
                                ctypes.POINTER(vp)]
    lib.cb_moe_forward.argtypes = [vp, vp, vp, vp]
    lib.cb_moe_forward_f32out.argtypes = [vp, vp, vp, vp]
    lib.cb_moe_forward_host.argtypes = [vp, vp, vp, vp]
    lib.cb_moe_forward_few.argtypes = [vp, vp, ctypes.c_int32, vp, vp]
    lib.cb_moe_forward_few_f32out.argtypes = [vp, vp, ctypes.c_int32, vp, vp]
    lib.cb_moe_forward_routed.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.cb_moe_forward_routed_f32out.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.cb_moe_forward_few_routed.argtypes = [vp, vp, ctypes.c_int32, vp, vp, vp, vp]
    lib.cb_moe_forward_few_routed_f32out.argtypes = [vp, vp, ctypes.c_int32, vp, vp, vp, vp]
    lib.cb_moe_routing.argtypes = [vp, ctypes.POINTER(cb_routing_view_t)]
    lib.cb_moe_stage_times.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.c_int32]
    lib.cb_moe_last_error.argtypes = [vp]
    lib.cb_moe_check_guards.argtypes = [vp]
    lib.cb_moe_device_bytes.argtypes = [ctypes.POINTER(cb_moe_config_t), ctypes.POINTER(ctypes.c_uint64)]
    lib.cb_moe_free.argtypes = [vp]
    lib.cb_moe_kernels_per_forward.argtypes = [vp, ctypes.POINTER(i32)]
    lib.cb_moe_set_stage_timing.argtypes = [vp, i32]
    lib.cb_moe_dispatch_noalloc.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp,
                                            vp, vp]
    lib.cb_moe_dispatch_noalloc.restype = i32
    for name in ("cb_moe_init", "cb_moe_forward", "cb_moe_forward_f32out", "cb_moe_forward_host",
                 "cb_moe_routing", "cb_moe_stage_times", "cb_moe_last_error", "cb_moe_device_bytes",
                 "cb_moe_free", "cb_moe_kernels_per_forward", "cb_moe_set_stage_timing", "cb_moe_check_guards",
                 "cb_moe_forward_few", "cb_moe_forward_few_f32out", "cb_moe_forward_routed", "cb_moe_forward_routed_f32out",
                 "cb_moe_forward_few_routed", "cb_moe_forward_few_routed_f32out"):
        getattr(lib, name).restype = i32
    i64 = ctypes.c_int64
    lib.cb_fp4_scale_bytes.argtypes = [ctypes.c_int32, i64, i64, ctypes.POINTER(ctypes.c_uint64)]
    lib.cb_fp4_quantize.argtypes = [ctypes.c_int32, vp, ctypes.c_int32, i64, i64, i64, vp, vp, vp, vp]
    lib.cb_fp4_dequantize.argtypes = [ctypes.c_int32, vp, vp, vp, i64, i64, vp, ctypes.c_int32, i64, vp]
    lib.cb_fp4_matmul.argtypes = [vp, vp]
    lib.cb_fp4_last_error.argtypes = []
    for name in FP4_SYMBOLS:
        getattr(lib, name).restype = i32
    for name in SERVE_SYMBOLS:
        getattr(lib, name).argtypes = [vp, vp]
        getattr(lib, name).restype = i32
    lib.cb_status_string.argtypes = [i32]
    lib.cb_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


# --------------------------------------------------------- same-name calls
def cb_status_string(status: int) -> str:
    return load_library().cb_status_string(int(status)).decode()


def cb_moe_init(cfg: cb_moe_config_t, weights: cb_moe_weights_t):
    """Returns (status, handle); handle is None unless status == CB_OK."""
    h = ctypes.c_void_p()
    st = load_library().cb_moe_init(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(h))
    return st, (h.value if st == CB_OK else None)


def cb_moe_forward(handle, x_ptr: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward(handle, x_ptr, out_ptr, stream)


def cb_moe_forward_f32out(handle, x_ptr: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_f32out(handle, x_ptr, out_ptr, stream)


def cb_moe_forward_few(handle, x_ptr: int, n_tokens: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_few(handle, x_ptr, n_tokens, out_ptr, stream)


def cb_moe_forward_few_f32out(handle, x_ptr: int, n_tokens: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_few_f32out(handle, x_ptr, n_tokens, out_ptr, stream)


def cb_moe_forward_routed(handle, x_ptr: int, ids_ptr: int, w_ptr: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_routed(handle, x_ptr, ids_ptr, w_ptr, out_ptr, stream)


def cb_moe_forward_routed_f32out(handle, x_ptr: int, ids_ptr: int, w_ptr: int, out_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_routed_f32out(handle, x_ptr, ids_ptr, w_ptr, out_ptr, stream)


def cb_moe_forward_few_routed(handle, x_ptr: int, n_tokens: int, ids_ptr: int, w_ptr: int, out_ptr: int,
                              stream: int = 0) -> int:
    return load_library().cb_moe_forward_few_routed(handle, x_ptr, n_tokens, ids_ptr, w_ptr, out_ptr, stream)


def cb_moe_forward_few_routed_f32out(handle, x_ptr: int, n_tokens: int, ids_ptr: int, w_ptr: int, out_ptr: int,
                                     stream: int = 0) -> int:
    return load_library().cb_moe_forward_few_routed_f32out(handle, x_ptr, n_tokens, ids_ptr, w_ptr, out_ptr, stream)


def cb_moe_forward_host(handle, x_host_ptr: int, out_host_ptr: int, stream: int = 0) -> int:
    return load_library().cb_moe_forward_host(handle, x_host_ptr, out_host_ptr, stream)


def cb_moe_routing(handle):
    v = cb_routing_view_t()
    st = load_library().cb_moe_routing(handle, ctypes.byref(v))
    return st, v


def cb_moe_stage_times(handle):
    """Returns (status, [router, dispatch, gate/up, down, combine] ms)."""
    ms = (ctypes.c_float * CB_N_STAGES)()
    st = load_library().cb_moe_stage_times(handle, ms, CB_N_STAGES)
    return st, list(ms)


def cb_moe_last_error(handle) -> int:
    return load_library().cb_moe_last_error(handle)


def cb_moe_check_guards(handle) -> int:
    return load_library().cb_moe_check_guards(handle)


def cb_moe_device_bytes(cfg: cb_moe_config_t):
    b = ctypes.c_uint64()
    st = load_library().cb_moe_device_bytes(ctypes.byref(cfg), ctypes.byref(b))
    return st, b.value


def cb_moe_kernels_per_forward(handle):
    n = ctypes.c_int32()
    st = load_library().cb_moe_kernels_per_forward(handle, ctypes.byref(n))
    return st, n.value


def cb_moe_free(handle) -> int:
    return load_library().cb_moe_free(handle)


def cb_moe_dispatch_noalloc(ids_ptr, n_tokens, top_k, n_experts, counts_ptr, offsets_ptr, tok_ptr, inv_ptr,
                            status_ptr=None, stream: int = 0) -> int:
    """Dispatch of routing ids with no device allocation (static scratch); see cb_moe.h."""
    return load_library().cb_moe_dispatch_noalloc(ids_ptr, n_tokens, top_k, n_experts, counts_ptr, offsets_ptr,
                                                  tok_ptr, inv_ptr, status_ptr, stream)


def cb_fp4_scale_bytes(fmt: int, rows: int, cols: int):
    b = ctypes.c_uint64()
    st = load_library().cb_fp4_scale_bytes(fmt, rows, cols, ctypes.byref(b))
    return st, b.value


def cb_fp4_quantize(fmt, x_ptr, x_type, rows, cols, ld, tensor_scale_ptr, codes_ptr, scales_ptr, stream: int = 0) -> int:
    return load_library().cb_fp4_quantize(fmt, x_ptr, x_type, rows, cols, ld, tensor_scale_ptr, codes_ptr, scales_ptr,
                                          stream)


def cb_fp4_dequantize(fmt, codes_ptr, scales_ptr, tensor_scale_ptr, rows, cols, out_ptr, out_type, ld,
                      stream: int = 0) -> int:
    return load_library().cb_fp4_dequantize(fmt, codes_ptr, scales_ptr, tensor_scale_ptr, rows, cols, out_ptr, out_type,
                                            ld, stream)


def cb_fp4_matmul(args: cb_fp4_matmul_t, stream: int = 0) -> int:
    return load_library().cb_fp4_matmul(ctypes.byref(args), stream)


def cb_fp4_last_error() -> int:
    return load_library().cb_fp4_last_error()


def cb_rms_norm(args: cb_rms_norm_t, stream: int = 0) -> int:
    return load_library().cb_rms_norm(ctypes.byref(args), stream)


def cb_route(args: cb_route_t, stream: int = 0) -> int:
    return load_library().cb_route(ctypes.byref(args), stream)


def cb_int4_matmul_few(args: cb_int4_matmul_t, stream: int = 0) -> int:
    return load_library().cb_int4_matmul_few(ctypes.byref(args), stream)


# ------------------------------------------------------- torch convenience
_cudart = None


def copy_from_device(dst_tensor, src_ptr: int, nbytes: int, stream=None) -> None:
    """Copy nbytes of library-owned device memory (e.g. a cb_routing_view_t
    array) into a torch CUDA tensor, with the CUDA runtime torch has loaded:
    in order on `stream`, or on the legacy default stream, which side streams
    do not wait for."""
    global _cudart
    if _cudart is None:
        import glob
        import sys
        names = ["libcudart.so.13", "libcudart.so.12", "libcudart.so"]
        for p in sys.path:
            names += glob.glob(os.path.join(p, "nvidia", "cu*", "lib", "libcudart.so*"))
            names += glob.glob(os.path.join(p, "nvidia", "cuda_runtime", "lib", "libcudart.so*"))
        names += glob.glob("/usr/local/cuda/lib64/libcudart.so*")
        for n in names:
            try:
                lib = ctypes.CDLL(n)
                break
            except OSError:
                continue
        else:
            raise RuntimeError("no CUDA runtime library found")
        lib.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
        lib.cudaMemcpy.restype = ctypes.c_int
        lib.cudaMemcpyAsync.argtypes = lib.cudaMemcpy.argtypes + [ctypes.c_void_p]
        lib.cudaMemcpyAsync.restype = ctypes.c_int
        _cudart = lib
    if nbytes:
        args = dst_tensor.data_ptr(), src_ptr, nbytes, 3  # device to device
        rc = _cudart.cudaMemcpy(*args) if stream is None else _cudart.cudaMemcpyAsync(*args, stream.cuda_stream)
        if rc != 0:
            raise RuntimeError(f"cudaMemcpy failed ({rc})")


def _ptr(t):
    return None if t is None else t.data_ptr()


class MoELayer:
    """One layer handle over torch device tensors (bf16 as torch.bfloat16 or int16 bits,
    int8 as torch.int8, e4m3 as uint8 bytes or torch.float8_e4m3fn).  Raises CbMoeError on
    any non-zero status."""

    def __init__(self, T, d, f, E, k, w_router, w_gate, w_up, w_down, router_bias=None,
                 s_gate=None, s_up=None, s_down=None, device=0, keep_logits=False, stage_timing=False,
                 flags=0, router="softmax", w_hash=None, z_gate=None, z_up=None, z_down=None, wdtype=None):
        """Expert weights: bf16; int8 codes with scales (s_*); packed int4 codes (two per
        byte along the input dimension) with scales and uint8 zero points (z_*); or e4m3
        bytes with scales (wdtype="fp8", or weights of dtype torch.float8_e4m3fn).  Without
        `wdtype` the format follows from which of s_* and z_* are given."""
        flags |= (CB_FLAG_KEEP_LOGITS if keep_logits else 0) | (CB_FLAG_STAGE_TIMING if stage_timing else 0)
        mode = ROUTER_MODES[router]
        hash_dims = 0 if w_hash is None else int(w_hash.shape[0])
        if wdtype is None:
            fp8 = str(getattr(w_gate, "dtype", "")).endswith("float8_e4m3fn")
            wdtype = (CB_W_INT4 if z_gate is not None else CB_W_FP8 if fp8 else
                      CB_W_INT8 if s_gate is not None else CB_W_BF16)
        elif isinstance(wdtype, str):
            wdtype = WDTYPES[wdtype]
        self.cfg = cb_moe_config_t(T, d, f, E, k, wdtype, device, flags, mode, hash_dims)
        w = cb_moe_weights_t(_ptr(w_router), _ptr(router_bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                             _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(w_hash),
                             _ptr(z_gate), _ptr(z_up), _ptr(z_down))
        st, h = cb_moe_init(self.cfg, w)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_init")
        self.handle = h

    def _check_given(self, routing, n):
        """The caller's routing (ids int32, w fp32, both [n][k] on the handle's device), e.g. route()'s."""
        torch, k = _torch or _load_torch(), self.cfg.top_k
        ids, w = routing
        for name, t, kind in (("ids", ids, torch.int32), ("w", w, torch.float32)):
            if t.dtype is not kind or tuple(t.shape) != (n, k) or not t.is_contiguous() or t.get_device() != self.cfg.device:
                raise ValueError(f"routing: {name} {tuple(t.shape)} {t.dtype} on {t.device}: contiguous {kind} of "
                                 f"{(n, k)} on device {self.cfg.device} is needed")
        return ids.data_ptr(), w.data_ptr()

    def forward(self, x, out, stream=None, f32out=False, routing=None):
        """The layer for the handle's T tokens: x bf16 (or int16 bits), out bf16 (fp32 with f32out),
        contiguous and of T d elements (more are left alone).  Runs on `stream`, or on the legacy
        default stream.  routing: (ids, w) in place of the handle's router, as cb_moe_forward_routed;
        made on another stream, they are the caller's to wait for."""
        need = self.cfg.n_tokens * self.cfg.d_model
        for name, t, size in (("x", x, 2), ("out", out, 4 if f32out else 2)):
            if not t.is_contiguous() or t.numel() * t.element_size() < need * size:
                raise ValueError(f"forward: {name} {tuple(t.shape)} {t.dtype} is not contiguous or holds less than "
                                 f"{self.cfg.n_tokens} x {self.cfg.d_model} elements of {size} bytes")
        s = 0 if stream is None else stream.cuda_stream
        if routing is not None:
            ids, w = self._check_given(routing, self.cfg.n_tokens)
            fn = cb_moe_forward_routed_f32out if f32out else cb_moe_forward_routed
            st = fn(self.handle, x.data_ptr(), ids, w, out.data_ptr(), s)
        else:
            fn = cb_moe_forward_f32out if f32out else cb_moe_forward
            st = fn(self.handle, x.data_ptr(), out.data_ptr(), s)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_forward")
        return out

    def forward_few(self, x, out, stream=None, f32out=False, routing=None):
        """The layer for x.shape[0] <= CB_MOE_MAX_FEW tokens, whatever T the handle was made for.
        x bf16 (or int16 bits) and out the same (fp32 with f32out), both contiguous [n][d] on the
        handle's device.  Runs on `stream`, or on torch's current stream there, as the 4-bit calls do.
        routing: (ids, w) in place of the handle's router, as cb_moe_forward_few_routed."""
        torch, device = _torch or _load_torch(), self.cfg.device
        if x.shape != out.shape or x.dim() != 2 or x.shape[1] != self.cfg.d_model:
            raise ValueError(f"forward_few: x {tuple(x.shape)}, out {tuple(out.shape)}, d = {self.cfg.d_model}")
        bits = (torch.bfloat16, torch.int16)
        if x.dtype not in bits or (out.dtype is not torch.float32 if f32out else out.dtype not in bits) or \
                not (x.is_contiguous() and out.is_contiguous()):
            raise ValueError(f"forward_few: x {x.dtype}, out {out.dtype}: contiguous bf16 (or its bits as int16) are "
                             f"needed, out fp32 with f32out and only then")
        if x.get_device() != device or out.get_device() != device:
            raise ValueError(f"forward_few: x on {x.device}, out on {out.device}, the handle on device {device}")
        s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
        if routing is not None:
            ids, w = self._check_given(routing, x.shape[0])
            fn = cb_moe_forward_few_routed_f32out if f32out else cb_moe_forward_few_routed
            st = fn(self.handle, x.data_ptr(), int(x.shape[0]), ids, w, out.data_ptr(), s)
        else:
            fn = cb_moe_forward_few_f32out if f32out else cb_moe_forward_few
            st = fn(self.handle, x.data_ptr(), int(x.shape[0]), out.data_ptr(), s)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_forward_few")
        return out

    def forward_host(self, x_host, out_host, stream=None):
        s = 0 if stream is None else stream.cuda_stream
        st = cb_moe_forward_host(self.handle, x_host.data_ptr(), out_host.data_ptr(), s)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_forward_host")
        return out_host

    def routing(self):
        st, v = cb_moe_routing(self.handle)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_routing")
        return v

    def stage_times(self):
        st, ms = cb_moe_stage_times(self.handle)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_stage_times")
        return ms

    def set_stage_timing(self, on: bool):
        """Stage events on or off for later forwards (handle made with stage_timing=True)."""
        st = load_library().cb_moe_set_stage_timing(self.handle, 1 if on else 0)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_set_stage_timing")

    def last_error(self) -> int:
        return cb_moe_last_error(self.handle)

    def check_guards(self) -> int:
        """CB_OK when every guard band of a CB_FLAG_GUARDS handle is intact."""
        return cb_moe_check_guards(self.handle)

    def kernels_per_forward(self) -> int:
        st, n = cb_moe_kernels_per_forward(self.handle)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_kernels_per_forward")
        return n

    def close(self):
        if getattr(self, "handle", None) is not None:
            st = cb_moe_free(self.handle)
            self.handle = None
            if st != CB_OK:
                raise CbMoeError(st, "cb_moe_free")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------ 4-bit floats with block scales, over torch tensors
# A decode step makes these calls with a few microseconds of GPU work each, so
# the way to the library is kept short: torch is looked up once, and a call on
# torch's current stream and device enters no context.
_torch = None
_FP4_TYPES = {}


def _load_torch():
    global _torch
    if _torch is None:
        import torch
        _FP4_TYPES.update({torch.bfloat16: CB_T_BF16, torch.float32: CB_T_F32})
        _torch = torch
    return _torch


def _stream_here(device, stream):
    """torch's current stream on `device` (an index) as an int, or None where a context has to
    be entered first: another stream is asked for, or another device is current."""
    if device < 0:
        raise ValueError("CUDA tensors are needed")
    if stream is None and device == _torch._C._cuda_getDevice():
        return _torch._C._cuda_getCurrentRawStream(device)
    return None


def _check_device(device, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on several devices: {t.device} beside device {device}")


class _On:
    """The device and the stream (torch's current one unless given) as a context."""

    def __init__(self, device, stream):
        self.device = _torch.cuda.device(device)
        self.stream = _torch.cuda.stream(_torch.cuda.current_stream(device) if stream is None else stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *a):
        self.stream.__exit__(*a)
        self.device.__exit__(*a)


def _fp4_type(dtype):
    kind = _FP4_TYPES.get(dtype)
    if kind is None:
        raise ValueError(f"4-bit floats are made from and turned into bfloat16 or float32, not {dtype}")
    return kind


def _fp4_scale_bytes(format, rows, cols):
    """cb_fp4_scale_bytes in Python."""
    if cols <= 0 or cols % 32:
        raise CbMoeError(CB_ERR_INVALID_ARG, f"a 4-bit matrix of {cols} columns (a positive multiple of 32 is needed)")
    return -(-rows // 128) * -(-cols // (4 * FP4_BLOCK[format])) * 512


def _row_stride(t):
    """Elements between the rows of a 2-D tensor whose rows are contiguous."""
    s = t.stride()
    if len(s) != 2 or (s[1] != 1 and t.shape[1] > 1):
        raise ValueError(f"a 2-D tensor with contiguous rows is needed, not one of shape {tuple(t.shape)}, strides {s}")
    return s[0] if s[0] >= t.shape[1] or t.shape[0] > 1 else t.shape[1]


class Fp4Matrix:
    """A matrix of 4-bit floats with block scales, as include/cb_fp4.h lays it out: `codes`
    uint8 [rows][cols / 2] and `scales` uint8; format "mx" or "nv", the latter with
    `tensor_scale` (fp32 [1]).  One matrix per expert: codes [E][rows][cols / 2], scales of
    E arrays, tensor_scale [E].  The tensors are kept as they are given, not copied: writing another
    scale into the caller's tensor_scale changes the matrix."""

    __slots__ = ("format", "rows", "cols", "groups", "codes", "scales", "tensor_scale")

    def __init__(self, format, rows, cols, codes, scales, tensor_scale=None):
        torch = _torch or _load_torch()
        if format not in FP4_FORMATS:
            raise ValueError(f"unknown 4-bit format {format!r}: one of {sorted(FP4_FORMATS)}")
        self.format = format
        self.rows = rows
        self.cols = cols
        self.codes = codes
        self.scales = scales
        self.tensor_scale = tensor_scale
        shape, kind, device = codes.shape, torch.uint8, codes.get_device()
        dims = len(shape)
        self.groups = groups = shape[0] if dims == 3 else 1
        need = _fp4_scale_bytes(format, rows, cols) * groups
        if dims not in (2, 3) or shape[-2] != rows or shape[-1] != cols // 2 or scales.numel() != need or \
                codes.dtype is not kind or scales.dtype is not kind or \
                not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError(f"codes {tuple(shape)} {codes.dtype}, scales {tuple(scales.shape)} {scales.dtype}: not "
                             f"{groups} contiguous {format} matrices of {rows} x {cols} ({need} scale bytes)")
        if (tensor_scale is not None) != (format == "nv") or \
                (tensor_scale is not None and (tensor_scale.dtype is not torch.float32 or
                                               tensor_scale.numel() != groups or not tensor_scale.is_contiguous())):
            raise ValueError("format nv has one fp32 tensor scale per matrix, format mx none")
        if scales.get_device() != device or (tensor_scale is not None and tensor_scale.get_device() != device):
            _check_device(device, scales, tensor_scale)


def fp4_quantize(x, format, tensor_scale=None, stream=None) -> Fp4Matrix:
    """x (2-D, bf16 or fp32, contiguous rows with any stride) as an Fp4Matrix; format "nv"
    takes tensor_scale, an fp32 CUDA tensor of one element, e.g. max|x| / (6 * 448), which the
    matrix keeps (0, as for zeros: every value is 0).  Runs on `stream`, or on torch's current
    stream; its result belongs to that stream."""
    torch = _load_torch()
    fmt, kind, ld = FP4_FORMATS.get(format), _fp4_type(x.dtype), _row_stride(x)
    if fmt is None:
        raise ValueError(f"unknown 4-bit format {format!r}: one of {sorted(FP4_FORMATS)}")
    rows, cols = x.shape
    nbytes = _fp4_scale_bytes(format, rows, cols)
    if tensor_scale is not None and (tensor_scale.dtype is not torch.float32 or tensor_scale.numel() != 1):
        raise ValueError("tensor_scale: one fp32 element")
    device = x.get_device()
    if tensor_scale is not None:
        _check_device(device, tensor_scale)
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return fp4_quantize(x, format, tensor_scale)
    m = Fp4Matrix.__new__(Fp4Matrix)
    m.format, m.rows, m.cols, m.groups, m.tensor_scale = format, rows, cols, 1, tensor_scale
    where = x.device
    m.codes = codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=where)
    m.scales = scales = torch.empty(nbytes, dtype=torch.uint8, device=where)
    st = (_lib or load_library()).cb_fp4_quantize(
        fmt, x.data_ptr(), kind, rows, cols, ld, None if tensor_scale is None else tensor_scale.data_ptr(),
        codes.data_ptr(), scales.data_ptr(), s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_fp4_quantize")
    return m


def fp4_dequantize(m: Fp4Matrix, dtype=None, out=None, stream=None):
    """The values that m stands for, as bf16 (or `dtype`), or into `out` (2-D, contiguous rows
    with any stride)."""
    torch = _load_torch()
    codes, g = m.codes, m.tensor_scale
    if m.groups != 1:
        raise ValueError("fp4_dequantize: one matrix at a time")
    if out is not None and (tuple(out.shape) != (m.rows, m.cols) or (dtype is not None and out.dtype != dtype)):
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} for a {m.rows} x {m.cols} matrix")
    kind = _fp4_type((dtype or torch.bfloat16) if out is None else out.dtype)
    device = codes.get_device()
    if out is not None:
        _check_device(device, out)
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return fp4_dequantize(m, dtype, out)
    if out is None:
        ld = m.cols
        out = torch.empty((m.rows, ld), dtype=dtype or torch.bfloat16, device=codes.device)
    else:
        ld = _row_stride(out)
    st = (_lib or load_library()).cb_fp4_dequantize(
        FP4_FORMATS[m.format], codes.data_ptr(), m.scales.data_ptr(), None if g is None else g.data_ptr(), m.rows,
        m.cols, out.data_ptr(), kind, ld, s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_fp4_dequantize")
    return out


def _check_int32(t, n, name):
    if t.dtype is not _torch.int32 or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 CUDA tensor of {n} is needed")


def fp4_matmul(a: Fp4Matrix, b: Fp4Matrix, dtype=None, out=None, tile_offsets=None, status=None, stream=None):
    """a b^T ([a.rows][b.rows], bf16 or `dtype`, or into `out`).  With `tile_offsets` (int32
    CUDA tensor [b.groups + 1], cb_routing_view_t's) rows 128 tile_offsets[e] .. 128
    tile_offsets[e + 1] of `a` meet b's e-th matrix; rows past the last are not written.
    `status`: an int32 CUDA tensor that receives CB_ERR_TIMEOUT if a device-side wait ran out and the
    result is garbage; without one fp4_last_error says so."""
    torch = _load_torch()
    if a.format != b.format or a.cols != b.cols or a.groups != 1:
        raise ValueError(f"fp4_matmul: {a.groups} x [{a.rows} x {a.cols}] {a.format} by [{b.rows} x {b.cols}] {b.format}")
    if tile_offsets is not None:
        _check_int32(tile_offsets, b.groups + 1, "tile_offsets")
    if status is not None:
        _check_int32(status, 1, "status")
    if out is not None and (tuple(out.shape) != (a.rows, b.rows) or (dtype is not None and out.dtype != dtype)):
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} for a {a.rows} x {b.rows} product")
    kind = _fp4_type((dtype or torch.bfloat16) if out is None else out.dtype)
    device = a.codes.get_device()
    if b.codes.get_device() != device or out is not None or tile_offsets is not None or status is not None:
        _check_device(device, b.codes, out, tile_offsets, status)
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return fp4_matmul(a, b, dtype, out, tile_offsets, status)
    rows, cols = a.rows, b.rows
    if out is None:
        ld = cols
        out = torch.empty((rows, cols), dtype=dtype or torch.bfloat16, device=a.codes.device)
    else:
        ld = _row_stride(out)
    nv = a.tensor_scale is not None
    st = (_lib or load_library()).cb_fp4_matmul(_FP4_MATMUL.pack(
        FP4_FORMATS[a.format], kind, rows, cols, a.cols, a.codes.data_ptr(), a.scales.data_ptr(),
        a.tensor_scale.data_ptr() if nv else 0, b.codes.data_ptr(), b.scales.data_ptr(),
        b.tensor_scale.data_ptr() if nv else 0, b.groups, 0 if tile_offsets is None else tile_offsets.data_ptr(),
        out.data_ptr(), ld, 0 if status is None else status.data_ptr()), s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_fp4_matmul")
    return out


def fp4_last_error(device=None):
    """Waits for the GPU (torch's current one unless given); CB_OK, or CB_ERR_TIMEOUT if since the
    last such call a product without a `status` gave up a device-side wait."""
    torch = _load_torch()
    with torch.cuda.device(torch.cuda.current_device() if device is None else device):
        return cb_fp4_last_error()


# ----------------------------------------------- around the layer, over torch tensors
class Fp8Rows:
    """Rows of e4m3 codes (torch.float8_e4m3fn, or its bytes as uint8, [rows][cols]) with an fp32 scale per
    row and 128 columns ([rows][ceil(cols / 128)]), both contiguous: X = scale * code.  The tensors
    are kept as they are given."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales):
        torch = _torch or _load_torch()
        self.codes = codes
        self.scales = scales
        shape = codes.shape
        if len(shape) != 2 or codes.dtype not in (torch.float8_e4m3fn, torch.uint8) or scales.dtype is not torch.float32 or \
                tuple(scales.shape) != (shape[0], -(-shape[1] // CB_FP8_COLS)) or \
                not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError(f"codes {tuple(shape)} {codes.dtype}, scales {tuple(scales.shape)} {scales.dtype}: not "
                             f"contiguous e4m3 rows with an fp32 scale per {CB_FP8_COLS} columns")
        self.rows, self.cols = shape
        _check_device(codes.get_device(), scales)


class RmsNormed:
    """What rms_norm returns: `out`, `fp8` (Fp8Rows) and `sum`, None where not asked for."""

    __slots__ = ("out", "fp8", "sum")

    def __init__(self, out, fp8, sum):
        self.out, self.fp8, self.sum = out, fp8, sum


def rms_norm(x, weight, eps=1e-6, residual=None, want="out", dtype=None, out=None, sum=None, stream=None) -> RmsNormed:
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual (2-D, bf16 or fp32, contiguous
    rows with any stride; h = x without a residual), as cb_rms_norm.  want: "out" (y in x's type or
    `dtype`, or into `out`), "fp8" (y as Fp8Rows) or "both".  With a residual h is returned too, in x's
    type (into `sum`, which may be x or residual itself).  `out` may be x itself."""
    torch = _torch or _load_torch()
    xtype, shape, device = x.dtype, x.shape, x.get_device()
    kind = _FP4_TYPES.get(xtype)
    wkind = kind if weight.dtype is xtype else _FP4_TYPES.get(weight.dtype)
    if kind is None or wkind is None:
        raise ValueError(f"rms_norm: x {xtype}, weight {weight.dtype}: bfloat16 or float32 are needed")
    ld = _row_stride(x)
    rows, cols = shape
    if weight.dim() != 1 or weight.shape[0] != cols or not weight.is_contiguous():
        raise ValueError(f"rms_norm: a weight of {tuple(weight.shape)} for {cols} columns")
    if weight.get_device() != device:
        _check_device(device, weight)
    want_out, want_fp8 = want != "fp8", want != "out"
    if want_out and want_fp8 and want != "both":
        raise ValueError(f"rms_norm: want {want!r} is none of 'out', 'fp8', 'both'")
    otype = dtype or xtype
    ld_out = ld_sum = cols
    if out is not None:
        if not want_out or out.shape != shape or (dtype is not None and out.dtype != dtype):
            raise ValueError(f"rms_norm: out {tuple(out.shape)} {out.dtype} for rows of {tuple(shape)}, want {want!r}")
        otype, ld_out = out.dtype, _row_stride(out)
        _check_device(device, out)
    okind = kind if otype is xtype else _FP4_TYPES.get(otype)
    if okind is None:
        raise ValueError("rms_norm: a result in bfloat16 or float32")
    if residual is None:
        if sum is not None:
            raise ValueError("rms_norm: a sum without a residual")
        r_ptr = ld_r = 0
    else:
        if residual.dtype is not xtype or residual.shape != shape:
            raise ValueError(f"rms_norm: a residual of {tuple(residual.shape)} {residual.dtype} beside x {tuple(shape)} {xtype}")
        if sum is not None:
            if sum.dtype is not xtype or sum.shape != shape:
                raise ValueError(f"rms_norm: a sum of {tuple(sum.shape)} {sum.dtype} beside x {tuple(shape)} {xtype}")
            ld_sum = _row_stride(sum)
            _check_device(device, sum)
        if residual.get_device() != device:
            _check_device(device, residual)
        r_ptr, ld_r = residual.data_ptr(), _row_stride(residual)
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return rms_norm(x, weight, eps, residual, want, dtype, out, sum)
    where, fp8, codes, scales = x.device, None, 0, 0
    if want_out and out is None:
        out = torch.empty(shape, dtype=otype, device=where)
    if residual is not None and sum is None:
        sum = torch.empty(shape, dtype=xtype, device=where)
    if want_fp8:
        fp8 = Fp8Rows.__new__(Fp8Rows)
        fp8.rows, fp8.cols = rows, cols
        fp8.codes = c = torch.empty(shape, dtype=torch.float8_e4m3fn, device=where)
        fp8.scales = f = torch.empty((rows, (cols + 127) // 128), dtype=torch.float32, device=where)
        codes, scales = c.data_ptr(), f.data_ptr()
    st = (_lib or load_library()).cb_rms_norm(_RMS_NORM.pack(
        rows, cols, x.data_ptr(), ld, r_ptr, ld_r, weight.data_ptr(), 0 if sum is None else sum.data_ptr(), ld_sum,
        out.data_ptr() if want_out else 0, ld_out, codes, scales, eps, kind, wkind, okind), s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_rms_norm")
    return RmsNormed(out, fp8, sum)


def route(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=None, group_score="top2", renormalise=True,
          scale=1.0, stream=None):
    """(ids int32 [T][top_k], w fp32 [T][top_k]) from logits [T][E] (bf16 or fp32, contiguous rows with any
    stride), as cb_route: the top_k experts by score ("sigmoid" or "softmax") + bias (fp32 [E]) of the best
    `top_groups` (all unless given) of `groups` groups of consecutive experts (by "top2" or "max"); weights
    are the scores, divided by their sum with `renormalise`, times `scale`."""
    torch = _torch or _load_torch()
    kind, how, by = _FP4_TYPES.get(logits.dtype), SCORES.get(score), GROUP_SCORES.get(group_score)
    if kind is None or how is None or by is None:
        raise ValueError(f"route: logits {logits.dtype} (bfloat16 or float32), score {score!r} (one of {sorted(SCORES)}), "
                         f"group_score {group_score!r} (one of {sorted(GROUP_SCORES)})")
    ld, device = _row_stride(logits), logits.get_device()
    tokens, experts = logits.shape
    b_ptr = 0
    if bias is not None:
        if bias.dtype is not torch.float32 or bias.numel() != experts or not bias.is_contiguous():
            raise ValueError(f"route: a contiguous fp32 bias of {experts} is needed")
        if bias.get_device() != device:
            _check_device(device, bias)
        b_ptr = bias.data_ptr()
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return route(logits, top_k, score, bias, groups, top_groups, group_score, renormalise, scale)
    if top_k < 1:
        raise CbMoeError(CB_ERR_INVALID_ARG, f"route: top_k = {top_k}")
    shape, where = (tokens, top_k), logits.device
    ids = torch.empty(shape, dtype=torch.int32, device=where)
    w = torch.empty(shape, dtype=torch.float32, device=where)
    st = (_lib or load_library()).cb_route(_ROUTE.pack(
        tokens, logits.data_ptr(), ld, b_ptr, ids.data_ptr(), w.data_ptr(), scale, kind, experts, top_k, how, groups,
        groups if top_groups is None else top_groups, by, 1 if renormalise else 0), s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_route")
    return ids, w


class Int4Matrix:
    """4-bit integer weights with a scale and a zero point per group of 32, 64 or 128 elements of a row, as
    include/cb_serve.h lays them out: codes uint8 [rows][cols / 2] (element 2i in the low nibble), scales
    fp32 [cols / group][rows], zeros uint8 of the same shape, or None for 8 everywhere.  One matrix per
    expert: codes [E][rows][cols / 2], scales and zeros [E][cols / group][rows].  The tensors are kept as
    they are given."""

    __slots__ = ("rows", "cols", "group", "experts", "codes", "scales", "zeros")

    def __init__(self, codes, scales, zeros=None):
        torch = _torch or _load_torch()
        self.codes, self.scales, self.zeros = codes, scales, zeros
        shape, meta, device = codes.shape, scales.shape, codes.get_device()
        dims = len(shape)
        if dims not in (2, 3) or len(meta) != dims or codes.dtype is not torch.uint8 or scales.dtype is not torch.float32 or \
                (dims == 3 and meta[0] != shape[0]) or meta[-1] != shape[-2] or meta[-2] == 0 or \
                not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError(f"codes {tuple(shape)} {codes.dtype}, scales {tuple(meta)} {scales.dtype}: not contiguous "
                             f"4-bit weights [..][rows][cols / 2] with scales [..][cols / group][rows]")
        if zeros is not None and (zeros.dtype is not torch.uint8 or zeros.shape != meta or not zeros.is_contiguous()):
            raise ValueError(f"zeros {tuple(zeros.shape)} {zeros.dtype}: contiguous uint8 of {tuple(meta)}, as the scales, are needed")
        self.experts = shape[0] if dims == 3 else None
        self.rows, self.cols = rows, cols = shape[-2], 2 * shape[-1]
        self.group = group = cols // meta[-2]
        if group not in (32, 64, 128) or group * meta[-2] != cols:
            raise ValueError(f"{meta[-2]} groups in {cols} columns: groups of 32, 64 or 128 are needed")
        if scales.get_device() != device or (zeros is not None and zeros.get_device() != device):
            _check_device(device, scales, zeros)


def int4_matmul_few(x, m: Int4Matrix, ids=None, weights=None, swiglu=False, dtype=None, out=None, status=None,
                    stream=None):
    """x m^T for 1 to CB_INT4_MAX_ROWS rows of x (bf16, contiguous rows, or Fp8Rows), in bf16 or `dtype`
    (or into `out`), as cb_int4_matmul_few.  One matrix: [T][rows].  With ids (int32 CUDA tensor [T][k]) each row
    meets its experts' matrices: [T][k][rows]; x may then be [T][k][cols] (Fp8Rows: T k rows), a row per slot.  With
    weights too (fp32 [T][k]) their weighted sum: [T][rows].  swiglu: the rows are gates, then the values they
    open: half as many columns.  `status`: an int32 CUDA tensor that receives CB_ERR_DEVICE where an id is no expert
    (that row is NaN)."""
    torch = _torch or _load_torch()
    experts, per_slot, tokens, top, i_ptr, w_ptr, x_scales = m.experts, 0, 0, 1, 0, 0, 0
    if ids is None:
        if experts is not None or weights is not None:
            raise ValueError("int4_matmul_few: ids come with a matrix per expert, and weights with ids")
    else:
        if experts is None:
            raise ValueError("int4_matmul_few: ids need a matrix per expert")
        if ids.dim() != 2 or ids.dtype is not torch.int32 or not ids.is_contiguous():
            raise ValueError("int4_matmul_few: ids: a contiguous int32 CUDA tensor [T][k] is needed")
        tokens, top = ids.shape
        i_ptr = ids.data_ptr()
        if weights is not None:
            if swiglu or weights.dtype is not torch.float32 or weights.shape != ids.shape or not weights.is_contiguous():
                raise ValueError(f"int4_matmul_few: weights: a contiguous fp32 tensor of {tuple(ids.shape)} is needed, "
                                 f"without swiglu")
            w_ptr = weights.data_ptr()
    if isinstance(x, Fp8Rows):
        data, x_scales, cols = x.codes, x.scales.data_ptr(), x.cols
        x_rows, ld = x.rows, cols
        if ids is not None and x_rows != tokens:
            per_slot = 1
    else:
        data, shape = x, x.shape
        if x.dtype is not torch.bfloat16:
            raise ValueError(f"int4_matmul_few: x {x.dtype}: rows of bfloat16, or Fp8Rows, are needed")
        if len(shape) == 3:
            if ids is None or not x.is_contiguous() or shape[:2] != ids.shape:
                raise ValueError(f"int4_matmul_few: x {tuple(shape)}: a contiguous x of [T][k][cols] comes with ids [T][k]")
            x_rows, cols, per_slot = tokens * top, shape[2], 1
            ld = cols
        else:
            ld = _row_stride(x)
            x_rows, cols = shape
    if cols != m.cols:
        raise ValueError(f"int4_matmul_few: rows of {cols} by a matrix of {m.cols} columns")
    if ids is None:
        tokens = x_rows
    elif x_rows != (tokens * top if per_slot else tokens):
        raise ValueError(f"int4_matmul_few: {x_rows} rows of x for ids of {tuple(ids.shape)}")
    width = m.rows // 2 if swiglu else m.rows
    shape = (tokens, width) if ids is None or weights is not None else (tokens, top, width)
    otype, ld_out, device = dtype or torch.bfloat16, width, data.get_device()
    if out is not None:
        if tuple(out.shape) != shape or (dtype is not None and out.dtype != dtype) or (len(shape) == 3 and not out.is_contiguous()):
            raise ValueError(f"int4_matmul_few: out {tuple(out.shape)} {out.dtype} for a result of {shape}")
        otype = out.dtype
        if len(shape) == 2:
            ld_out = _row_stride(out)
    kind = _FP4_TYPES.get(otype)
    if kind is None:
        raise ValueError("int4_matmul_few: a result in bfloat16 or float32")
    if status is not None:
        _check_int32(status, 1, "status")
    if m.codes.get_device() != device or ids is not None or out is not None or status is not None:
        _check_device(device, m.codes, ids, weights, out, status)
    s = _stream_here(device, stream)
    if s is None:
        with _On(device, stream):
            return int4_matmul_few(x, m, ids, weights, swiglu, dtype, out, status)
    if out is None:
        out = torch.empty(shape, dtype=otype, device=data.device)
    zeros = m.zeros
    st = (_lib or load_library()).cb_int4_matmul_few(_INT4.pack(
        data.data_ptr(), x_scales, m.codes.data_ptr(), m.scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), i_ptr,
        w_ptr, out.data_ptr(), 0 if status is None else status.data_ptr(), ld, ld_out, m.rows, cols, tokens, top,
        experts or 1, m.group, per_slot, 1 if swiglu else 0, kind), s)
    if st != CB_OK:
        raise CbMoeError(st, "cb_int4_matmul_few")
    return out
