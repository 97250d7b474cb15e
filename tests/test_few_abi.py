"""Argument checks of moe_forward_few and moe_gemv_w4 on the CPU: every call
here fails validation, so nothing is launched."""
import ctypes
import os
import re

import pytest

import mixture_experts_router_amd as moe
from mixture_experts_router_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F, MIS, BIG = 0x100000, 0x100002, 1 << 40     # an aligned and a misaligned address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return moe.load(os.environ.get("MOE_TEST_LIB", _lib.LIB_PATH))


def S(T=8, H=256, E=8, k=2, I=128, f=0):
    return _lib.MoeShape(T, H, E, k, I, f)


def few(lib, s, **kw):
    a = dict(x=F, wr=F, bias=None, gu=F, gus=None, d=F, ds=None, I_sh=0, sgu=None, sgus=None, sd=None, sds=None, out=F,
             ids=None, w=None, ws=F, n=BIG)
    a.update(kw)
    return lib.moe_forward_few(ctypes.byref(s) if s else None, *a.values(), None)


def W(T=4, N=100, K=256, f=5, group=64, flags=0, ldx=0, ldy=0):
    return _lib.MoeW4Shape(T, N, K, f, group, flags, ldx, ldy)


def gemv(lib, s, **kw):
    a = dict(x=F, w=F, scales=F, zeros=None, bias=None, y=F, ws=F, n=BIG)
    a.update(kw)
    return lib.moe_gemv_w4(ctypes.byref(s) if s else None, *a.values(), None)


def test_header_constants():
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    assert re.search(r"#define MOE_FEW_MAX_TOKENS (\d+)", text).group(1) == str(moe.FEW_MAX_TOKENS)
    assert re.search(r"#define MOE_FEW_ZERO_BYTES (\d+)", text).group(1) == str(moe.FEW_ZERO_BYTES)
    assert f"MOE_W_INT4 = {moe.MOE_W_INT4}" in text
    assert f"MOE_GEMV_GEGLU = {moe.MOE_GEMV_GEGLU}" in text and f"MOE_GEMV_Y_FP32 = {moe.MOE_GEMV_Y_FP32}" in text
    assert ctypes.sizeof(_lib.MoeW4Shape) == 40


@pytest.mark.parametrize("s,expect", [
    (None, -1), (S(T=0), -1), (S(H=0), -1), (S(E=0), -1), (S(k=0), -1), (S(I=0), -1), (S(k=9), -1), (S(T=17), -2),
    (S(T=1 << 20), -2), (S(H=96), -2), (S(I=100), -2), (S(E=2000), -2), (S(E=64, k=33), -2), (S(f=2), -2),
    (S(f=4), -2), (S(f=5), -2), (S(f=-1), -2), (S(H=65600), -2), (S(I=65600), -2), (S(H=1 << 28), -2),
])
def test_few_shapes(lib, s, expect):
    assert few(lib, s, gus=F, ds=F) == expect
    assert lib.moe_few_workspace_bytes(ctypes.byref(s) if s else None, 0) == 0


def test_few_arguments(lib):
    for name in ("x", "wr", "gu", "d", "out"):
        assert few(lib, S(), **{name: None}) == -1
        assert few(lib, S(), **{name: MIS}) == -1
    for name in ("bias", "ids", "w"):
        assert few(lib, S(), **{name: MIS}) == -1
    assert few(lib, S(), gus=F) == -1                                     # bf16 weights come without scales
    assert few(lib, S(f=1)) == -1                                         # MXFP4 weights need them
    assert few(lib, S(f=1), gus=F, ds=F, gu=F + 4) == -1                  # 4-bit codes 16-byte aligned
    assert few(lib, S(f=1), gus=MIS, ds=F) == -1                          # scales 4-byte aligned
    assert few(lib, S(f=3), gus=F, ds=MIS) == -1                          # NVFP4 scale buffers 4-byte aligned
    assert few(lib, S(), I_sh=-64) == -1
    assert few(lib, S(), I_sh=100, sgu=F, sd=F) == -2 and few(lib, S(), I_sh=65600, sgu=F, sd=F) == -2
    assert few(lib, S(), I_sh=128, sgu=F) == -1
    assert few(lib, S(), I_sh=128, sgu=F, sd=F, sds=F) == -1
    assert few(lib, S(f=3), gus=F, ds=F, I_sh=128, sgu=F, sd=F, sgus=F) == -1
    need = lib.moe_few_workspace_bytes(ctypes.byref(S()), 0)
    assert need >= moe.FEW_ZERO_BYTES + 8 * 8 * 4 + 8 * 2 * 128 * 2
    assert few(lib, S(), ws=None) == -3 and few(lib, S(), n=need - 1) == -3 and few(lib, S(), ws=F + 8) == -3
    assert lib.moe_few_workspace_bytes(ctypes.byref(S()), 128) > need
    assert lib.moe_few_workspace_bytes(ctypes.byref(S()), 100) == 0
    assert lib.moe_few_workspace_bytes(ctypes.byref(S()), -64) == 0


@pytest.mark.parametrize("s,expect", [
    (None, -1), (W(T=0), -1), (W(N=0), -1), (W(K=0), -1), (W(group=-32), -1), (W(ldx=-1), -1), (W(ldy=-1), -1),
    (W(T=17), -2), (W(N=(1 << 30) + 1), -2), (W(K=(1 << 20) + 128), -2), (W(K=100), -2), (W(K=96, group=64), -2),
    (W(group=16), -2), (W(group=0), -2), (W(f=1), -1), (W(f=0, group=0), -2), (W(f=2, group=0), -2), (W(f=6), -2),
    (W(f=3, group=0, K=48), -2), (W(flags=4), -1), (W(N=101, flags=1), -1), (W(ldx=255), -1), (W(ldx=260), -2),
    (W(ldy=99), -1), (W(ldx=1 << 41), -1), (W(ldy=1 << 41), -1),
])
def test_gemv_shapes(lib, s, expect):
    assert gemv(lib, s) == expect
    assert lib.moe_gemv_w4_workspace_bytes(ctypes.byref(s) if s else None) == 0


def test_gemv_arguments(lib):
    for name in ("x", "w", "scales", "y"):
        assert gemv(lib, W(), **{name: None}) == -1
    assert gemv(lib, W(), x=F + 8) == -1 and gemv(lib, W(), w=F + 8) == -1 and gemv(lib, W(), scales=F + 1) == -1
    assert gemv(lib, W(), y=F + 1) == -1 and gemv(lib, W(flags=2), y=MIS) == -1 and gemv(lib, W(), bias=MIS) == -1
    assert gemv(lib, W(f=3, group=0), scales=MIS) == -1
    assert gemv(lib, W(), scales=MIS) == -1 and gemv(lib, W(), zeros=MIS) == -1 and gemv(lib, W(f=1, group=0), scales=MIS) == -1
    assert gemv(lib, W(f=1, group=0), zeros=F) == -1 and gemv(lib, W(f=3, group=0), zeros=F) == -1
    # few rows and a long K: partial sums, so a workspace
    s = W(T=16, K=1 << 16)
    need = lib.moe_gemv_w4_workspace_bytes(ctypes.byref(s))
    assert need > moe.FEW_ZERO_BYTES
    assert gemv(lib, s, ws=None) == -3 and gemv(lib, s, n=need - 1) == -3 and gemv(lib, s, ws=F + 4) == -3
    # many rows, or a short K: none
    assert lib.moe_gemv_w4_workspace_bytes(ctypes.byref(W(T=16, N=1 << 20, K=1 << 20))) == 0
    assert lib.moe_gemv_w4_workspace_bytes(ctypes.byref(W(T=16, K=2816))) == 0
    assert lib.moe_gemv_w4_workspace_bytes(ctypes.byref(W(T=1, K=16384))) == 0


def test_binding_refusals():
    with pytest.raises(ValueError, match="unknown 4-bit format"):
        moe.w4_shape(1, 16, 64, "int8")
    import torch
    cpu = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.gemv_w4(moe.w4_shape(2, 16, 64, "mxfp4"), cpu, F, F, None, None, F)
    with pytest.raises(ValueError, match="device tensor"):
        moe.gemv_w4(moe.w4_shape(2, 16, 64, "mxfp4", ldx=72), cpu, F, F, None, None, F)
    with pytest.raises(ValueError, match="device tensor"):
        moe.forward_few(S(), cpu, F, None, F, None, F, None, F)


@pytest.mark.parametrize("var", ["hostsan"])
def test_checks_under_sanitizers(var):
    """The same checks against the build whose host code runs under the
    address and undefined-behaviour sanitizers."""
    if "MOE_TEST_LIB" in os.environ:
        pytest.skip("this is that run")
    import subprocess
    import sys
    import test_sanitizers as t
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_few_abi.py"],
                       cwd=ROOT, env=t._env(), capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
