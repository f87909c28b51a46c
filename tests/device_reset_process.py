"""Child process of tests/test_zz_device_reset.py: the calls that keep no handle, before and after a
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


def dispatch(T=3000, k=4, E=64):
    rng = np.random.default_rng(1)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32).copy()
    counts, offsets, tok, inv, status = (alloc(4 * n, 0xFF) for n in (E, E + 1, T * k, T * k, 1))
    st = cb.cb_moe_dispatch_noalloc(put(ids), T, k, E, counts, offsets, tok, inv, status, 0)
    assert st == cb.CB_OK and rt.cudaDeviceSynchronize() == 0
    assert get(status, 1, np.int32)[0] == 0
    order = np.argsort(ids.ravel(), kind="stable")
    assert np.array_equal(get(counts, E, np.int32), np.bincount(ids.ravel(), minlength=E))
    assert np.array_equal(get(tok, T * k, np.int32), order // k)
    assert np.array_equal(get(inv, T * k, np.int32), np.argsort(order, kind="stable"))


def product(m, n=2304, k=1024):
    """Ones by ones: every sum is k."""
    ones = lambda rows: alloc(rows * k // 2, 0x22)  # noqa: E731
    unit = lambda rows: alloc(cb.cb_fp4_scale_bytes(cb.CB_FP4_MX, rows, k)[1], 127)  # noqa: E731
    out, status = alloc(m * n * 4), alloc(4)
    a = cb.cb_fp4_matmul_t(cb.CB_FP4_MX, cb.CB_T_F32, m, n, k, ones(m), unit(m), None, ones(n), unit(n), None, 1, None, out, n,
                           status)
    assert cb.cb_fp4_matmul(a) == cb.CB_OK and rt.cudaDeviceSynchronize() == 0
    assert get(status, 1, np.int32)[0] == 0 and (get(out, m * n, np.float32) == k).all()


for reset in (False, True, True):
    if reset:
        assert rt.cudaDeviceReset() == 0
        held = alloc(64 << 20)           # (addresses need not be the same again)
    for _ in range(2):
        dispatch()
        for m in (4, 200, 2400):         # swapped, single CTAs, CTA pairs
            product(m)
print("RESET_OK")
