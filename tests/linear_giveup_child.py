"""Child process of test_linear_giveup_gpu.py: linear layers on the short-wait build of
the library, in which every pipeline wait inside the kernels gives up as soon as its
phase has not completed at the first probe.  Prints one JSON line with each call's
status and how long it took; it loads only that build."""
import ctypes
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from paged_fp8_gated_b200 import build  # noqa: E402

vp, i64 = ctypes.c_void_p, ctypes.c_int64
lib = ctypes.CDLL(build.SHORT_WAIT_LIB)
lib.gad_linear.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64] + [ctypes.c_int] * 6 + [vp]
lib.gad_linear_status.argtypes = [ctypes.POINTER(ctypes.c_int), vp]
BF16, F32 = 1, 6


def status():
    st = ctypes.c_int(-1)
    assert lib.gad_linear_status(ctypes.byref(st), None) == 0
    torch.cuda.synchronize()
    return int(st.value)


res = {}
for name, T, K, N, out in json.loads(sys.argv[1]):
    x = torch.ones(T, K, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(N, K, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(T, N, device="cuda", dtype=torch.float32 if out == F32 else torch.bfloat16)
    torch.cuda.synchronize()
    t0 = time.time()
    assert lib.gad_linear(x.data_ptr(), K, w.data_ptr(), K, None, None, 0, y.data_ptr(), N, T, K, N, BF16, out, 0,
                          None) == 0
    torch.cuda.synchronize()
    res[name] = [status(), status(), time.time() - t0]
# the context still works
a = torch.arange(1000, device="cuda", dtype=torch.float32)
res["after"] = float((a * 2).sum())
print(json.dumps(res), flush=True)
