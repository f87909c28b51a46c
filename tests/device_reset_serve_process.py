"""Child process of tests/test_zz_device_reset_serve.py: the operators around the layer, before and after a
cudaDeviceReset of this process's own context, with plain CUDA allocations (no torch on the GPU).
Prints RESET_OK and exits 0 when every result is right."""
import ctypes
import glob
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import mixture_experts_router_gb300 as cb  # noqa: E402

rt = ctypes.CDLL(sorted(glob.glob("/usr/local/cuda/lib64/libcudart.so*"))[0])
vp = ctypes.c_void_p
rt.cudaMalloc.argtypes = [ctypes.POINTER(vp), ctypes.c_size_t]
rt.cudaMemset.argtypes = [vp, ctypes.c_int, ctypes.c_size_t]
rt.cudaMemcpy.argtypes = [vp, vp, ctypes.c_size_t, ctypes.c_int]


def alloc(nbytes, fill=0):
    p = vp()
    assert rt.cudaMalloc(ctypes.byref(p), nbytes) == 0 and rt.cudaMemset(p, fill, nbytes) == 0
    return p.value


def put(a):
    p = alloc(a.nbytes)
    assert rt.cudaMemcpy(p, a.ctypes.data, a.nbytes, 1) == 0
    return p


def get(p, shape, dtype):
    a = np.empty(shape, dtype)
    assert rt.cudaMemcpy(a.ctypes.data, p, a.nbytes, 2) == 0
    return a


ONES16 = lambda n: put(np.full(n, 0x3F80, np.uint16))  # noqa: E731
ONES = lambda n: put(np.ones(n, np.float32))  # noqa: E731


def product(rows, n, k, group, experts=None, top=1, summed=False):
    """Ones by ones (codes 9, zero points of 8): every sum is k, or k top with the sum over slots."""
    e = experts or 1
    out_rows = rows if summed or experts is None else rows * top
    out, status = alloc(out_rows * n * 4), alloc(4)
    ids = None if experts is None else put((np.arange(rows * top) % experts).astype(np.int32))
    a = cb.cb_int4_matmul_t(ONES16(rows * k), None, alloc(e * n * k // 2, 0x99), ONES(e * n * (k // group)), None, ids,
                            ONES(rows * top) if summed else None, out, status, k, n, n, k, rows, top, e, group, 0, 0, cb.CB_T_F32)
    assert cb.cb_int4_matmul_few(a) == cb.CB_OK and rt.cudaDeviceSynchronize() == 0
    assert get(status, 1, np.int32)[0] == 0
    assert (get(out, out_rows * n, np.float32) == (k * top if summed else k)).all()


def norm(rows, cols):
    out = alloc(rows * cols * 4)
    a = cb.cb_rms_norm_t(rows, cols, ONES(rows * cols), cols, None, 0, ONES(cols), None, 0, out, cols, None, None, 0.0,
                         cb.CB_T_F32, cb.CB_T_F32, cb.CB_T_F32)
    assert cb.cb_rms_norm(a) == cb.CB_OK and rt.cudaDeviceSynchronize() == 0
    assert (get(out, rows * cols, np.float32) == 1).all()


def route(tokens, experts, k):
    ids, w = alloc(tokens * k * 4), alloc(tokens * k * 4)
    a = cb.cb_route_t(tokens, ONES(tokens * experts), experts, None, ids, w, 1.0, cb.CB_T_F32, experts, k,
                      cb.CB_SCORE_SOFTMAX, 1, 1, cb.CB_GROUP_MAX, 1)
    assert cb.cb_route(a) == cb.CB_OK and rt.cudaDeviceSynchronize() == 0
    assert (get(ids, (tokens, k), np.int32) == np.arange(k)).all() and (get(w, tokens * k, np.float32) == 1 / k).all()


for reset in (False, True, True):
    if reset:
        assert rt.cudaDeviceReset() == 0
        held = alloc(64 << 20)           # (addresses need not be the same again)
    for _ in range(2):
        product(1, 512, 256, 32)
        product(16, 2304, 1024, 128)
        product(8, 4096, 14336, 64)      # clusters
        product(6, 512, 1024, 64, experts=8, top=2)
        product(6, 512, 1024, 64, experts=8, top=2, summed=True)
        norm(4, 4096)
        norm(2000, 4096)
        route(100, 64, 4)
print("RESET_OK")
