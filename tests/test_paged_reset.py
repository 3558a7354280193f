"""The paged calls in a process that resets its device between them: what the
library caches belongs to a context. In a process of its own, which holds no
other CUDA state."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CODE = r"""
import ctypes
import numpy as np
import torch                                    # for its libcudart; no CUDA call goes through it
from depth_kv_attention_b200 import lib
rt = ctypes.CDLL("libcudart.so.12")
vp, f, sz, ll = ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
rng = np.random.default_rng(1)

def put(a):
    p = vp()
    assert rt.cudaMalloc(ctypes.byref(p), sz(a.nbytes)) == 0
    assert rt.cudaMemcpy(p, a.ctypes.data_as(vp), sz(a.nbytes), 1) == 0
    return p

def get(p, n):
    a = np.empty(n, np.uint16)
    assert rt.cudaMemcpy(a.ctypes.data_as(vp), p, sz(a.nbytes), 2) == 0
    return a

N, Hq, Hkv, d, P, pages = 4096, 8, 2, 128, 16, 256
bf = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
q, k, v = bf(N, Hq, d), bf(N, Hkv, d), bf(N, Hkv, d)
zero = lambda n: np.zeros(n, np.uint8)
i32 = lambda *x: np.array(x, np.int32)

def calls():
    # the bulk-copy append, then attention by the kernels for few rows and for chunks
    dq, dk, dv, qo = put(q), put(k), put(v), put(np.zeros_like(q))
    size = pages * Hkv * P * d * 2
    kp, vpg, ws = put(zero(size)), put(zero(size)), put(zero(64 << 20))
    table, cu, ctx = put(np.arange(pages, dtype=np.int32)), put(i32(0, N)), put(i32(N))
    res = [lib.moda_paged_append(dq, dk, dv, ll(Hq * d), ll(Hkv * d), ll(Hkv * d), None, 0, 0, 0, cu, ctx, table, N, 1, Hq,
                                 Hkv, d, pages, P, pages, 0, kp, vpg, qo, None, None, 0, 0, None)]
    outs = [get(kp, size // 2)]
    for new in (1, 90):
        cu, out = put(i32(0, new)), put(np.zeros_like(q[:new]))
        res.append(lib.moda_fwd_paged(qo, kp, vpg, None, None, cu, ctx, table, new, 1, new, Hq, Hkv, d, 0, 0, pages, P, pages,
                                      0, f(0.1), out, None, ws, sz(64 << 20), None, 0))
        outs.append(get(out, new * Hq * d))
    assert res == [0, 0, 0] and lib.moda_device_status(None) == 0, res
    return outs

first = calls()
assert all(o.any() for o in first)
for _ in range(2):
    assert rt.cudaDeviceReset() == 0
    assert all(np.array_equal(a, b) for a, b in zip(first, calls()))
    assert all(np.array_equal(a, b) for a, b in zip(first, calls()))
"""


def test_calls_after_a_device_reset():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
