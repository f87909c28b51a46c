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
               "cb_moe_set_stage_timing", "cb_moe_check_guards", "cb_moe_forward_few", "cb_moe_forward_few_f32out")


CB_MOE_MAX_FEW = 16
# every symbol include/cb_fp4.h declares
FP4_SYMBOLS = ("cb_fp4_scale_bytes", "cb_fp4_quantize", "cb_fp4_dequantize", "cb_fp4_matmul", "cb_fp4_last_error")
CB_FP4_MX, CB_FP4_NV = 0, 1
CB_T_BF16, CB_T_F32 = 0, 1
FP4_FORMATS = {"mx": CB_FP4_MX, "nv": CB_FP4_NV}
FP4_BLOCK = {"mx": 32, "nv": 16}
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
                 "cb_moe_forward_few", "cb_moe_forward_few_f32out"):
        getattr(lib, name).restype = i32
    i64 = ctypes.c_int64
    lib.cb_fp4_scale_bytes.argtypes = [ctypes.c_int32, i64, i64, ctypes.POINTER(ctypes.c_uint64)]
    lib.cb_fp4_quantize.argtypes = [ctypes.c_int32, vp, ctypes.c_int32, i64, i64, i64, vp, vp, vp, vp]
    lib.cb_fp4_dequantize.argtypes = [ctypes.c_int32, vp, vp, vp, i64, i64, vp, ctypes.c_int32, i64, vp]
    lib.cb_fp4_matmul.argtypes = [vp, vp]
    lib.cb_fp4_last_error.argtypes = []
    for name in FP4_SYMBOLS:
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

    def forward(self, x, out, stream=None, f32out=False):
        """The layer for the handle's T tokens: x bf16 (or int16 bits), out bf16 (fp32 with f32out),
        contiguous and of T d elements (more are left alone).  Runs on `stream`, or on the legacy
        default stream."""
        need = self.cfg.n_tokens * self.cfg.d_model
        for name, t, size in (("x", x, 2), ("out", out, 4 if f32out else 2)):
            if not t.is_contiguous() or t.numel() * t.element_size() < need * size:
                raise ValueError(f"forward: {name} {tuple(t.shape)} {t.dtype} is not contiguous or holds less than "
                                 f"{self.cfg.n_tokens} x {self.cfg.d_model} elements of {size} bytes")
        s = 0 if stream is None else stream.cuda_stream
        fn = cb_moe_forward_f32out if f32out else cb_moe_forward
        st = fn(self.handle, x.data_ptr(), out.data_ptr(), s)
        if st != CB_OK:
            raise CbMoeError(st, "cb_moe_forward")
        return out

    def forward_few(self, x, out, stream=None, f32out=False):
        """The layer for x.shape[0] <= CB_MOE_MAX_FEW tokens, whatever T the handle was made for.
        x bf16 (or int16 bits) and out the same (fp32 with f32out), both contiguous [n][d] on the
        handle's device.  Runs on `stream`, or on torch's current stream there, as the 4-bit calls do."""
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
        raise ValueError("4-bit matrices are made from and kept in CUDA tensors")
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
