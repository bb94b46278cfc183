"""Calls from a thread whose current context is the caller's own (cuCtxCreate), on a
stream of that context: it stays current and the kernels run in it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import ctypes
import numpy as np
import oracle
from exact_io_aware_96_b200 import fa

cu = ctypes.CDLL("libcuda.so.1")
def ok(status): assert status == 0, status
ok(cu.cuInit(0))
dev, ctx, stream = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_void_p()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, dev))
ok(cu.cuStreamCreate(ctypes.byref(stream), 1))
def current():
    now = ctypes.c_void_p()
    ok(cu.cuCtxGetCurrent(ctypes.byref(now)))
    return now.value
def device(a):
    p = ctypes.c_uint64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
    ok(cu.cuMemcpyHtoD_v2(p, a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes)))
    return p.value
B, H, S, D = 1, 2, 130, 64
rng = np.random.default_rng(3)
q, k, v = (rng.standard_normal((B, S, H, D)).astype(np.float16) for _ in range(3))
o, lse = np.full_like(q, np.nan), np.full((B, H, S), np.nan, np.float32)
dq, dk, dv, do, dl = (device(a) for a in (q, k, v, o, lse))
assert current() == ctx.value
assert fa.fa_fwd(dq, dk, dv, do, dl, B, H, S, S, D, D ** -0.5, 1, fa.FA_FP16, stream.value) == 0
assert current() == ctx.value, "another context has become current"
ok(cu.cuCtxSynchronize())
for a, p in ((o, do), (lse, dl)):
    ok(cu.cuMemcpyDtoH_v2(a.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(p), ctypes.c_size_t(a.nbytes)))
o_ref, lse_ref = oracle.attention_forward(*(x.astype(np.float64) for x in (q, k, v)), D ** -0.5, True)
assert np.abs(o - o_ref).max() <= 1e-2 and np.abs(lse - lse_ref).max() <= 1e-3
assert fa.fa_last_device_status()[0] == 0 and current() == ctx.value
print("own context")
"""


def test_forward_in_an_own_context(fa_lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=200)
    assert "own context" in out.stdout, out.stderr[-1500:]
