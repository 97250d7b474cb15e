"""The bounds-checked build run over the few-token operators' shapes must
record no out-of-range address.  Runs in a child process so that the debug
library is the only one loaded."""
import os
import subprocess
import sys

import pytest

from mixture_experts_router_amd import build as b

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, sys
sys.path.insert(0, "tests")
import torch
import mixture_experts_router_amd as moe
lib = moe.load(sys.argv[1])
lib.moe_debug_bounds.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
from few_helpers import Layer, Gemv
import test_gpu_few as few, test_gpu_gemv_w4 as gemv

def bounds(label):
    v, w = ctypes.c_uint32(), ctypes.c_uint32()
    assert lib.moe_debug_bounds(ctypes.byref(v), ctypes.byref(w)) == 0
    print(f"{label}: violations {v.value} first at {w.value}", flush=True)
    assert v.value == 0, (label, w.value)

for fmt in few.FMTS:
    for name, s in few.SHAPES.items():
        print(name, fmt, flush=True)
        l = Layer(**s, fmt=fmt)
        l.check(l.run(), f"{name} {fmt}")
        bounds(f"few {name} {fmt}")
    l = Layer(16, 2816, 10, 4, 704, I_sh=2112, fmt=fmt)
    l.check(l.run(), f"model width {fmt}")
    bounds(f"few model width {fmt}")
for fmt, group in gemv.FORMATS:
    for T, N, K in gemv.SIZES + [(4, 50, 1408), (3, 6, 8192)]:
        print(fmt, group, T, N, K, flush=True)
        for geglu in (False, True):
            g = Gemv(T, N + (N % 2 if geglu else 0), K, fmt, group, zeros=fmt == "int4", bias=True, geglu=geglu, pad_x=8, pad_y=1)
            g.check(g.run(), "gemv")
        bounds(f"gemv {fmt} {group} {T}x{N}x{K}")
for fmt in ("mxfp4", "nvfp4"):
    for K in (32, 96, 160, 224):
        g = Gemv(16, 20, K, fmt)
        g.check(g.run(), "gemv")
        bounds(f"gemv {fmt} K={K}")
print("__FEW_BOUNDS_OK__", flush=True)
'''


def test_few_token_operators_stay_in_bounds():
    if not os.path.exists(b.DEBUG_LIB):
        pytest.fail(f"{b.DEBUG_LIB} is missing: build it with build(debug=True)")
    r = subprocess.run([sys.executable, "-u", "-c", CHILD, b.DEBUG_LIB], cwd=ROOT, capture_output=True, text=True,
                       timeout=900)
    print(r.stdout[-6000:])
    assert r.returncode == 0 and "__FEW_BOUNDS_OK__" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
