"""Argument checks of the 8-bit operators and the norm in the C ABI (no GPU): every call here is refused, or has nothing
to do, before the library touches HIP, so the fake device addresses are compared and never read.  The same checks run
against a sanitized host build."""
import ctypes
import os
import subprocess
import sys

import pytest

from tests.test_host_sanitized import (COMMON, CSRC, GXX, HOST, ROCM, ROOT, SAN, SAN_ENV, _run,  # noqa: F401
                                       san_build)

nf4 = pytest.importorskip("quantized_lora_fine_amd", reason="libnf4lora.so not built")
lib = nf4._lib

needs_host_build = pytest.mark.skipif(GXX is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"),
                                      reason="needs g++ and the HIP host runtime")

GB = 1 << 30
A, S, W, T, C, A2, B2, OFF = ((i + 1) * 64 * GB for i in range(8))  # aligned fake addresses, far apart


def odd(name):
    """An address that is not aligned enough: 4 bytes for scales, rstd and offsets, 16 for the others."""
    return 64 * GB * 9 + (2 if name in ("scales", "s", "ws", "off", "rstd") else 8)


def quantize(X=A, bf16=0, rows=8, cols=272, fmt=0, block_rows=1, codes=C, scales=S):
    return lib.nf4_fp8_quantize(X, bf16, rows, cols, fmt, block_rows, codes, scales, None)


def dequantize(codes=A, scales=S, rows=8, cols=272, fmt=0, block_rows=1, out=C, bf16=0):
    return lib.nf4_fp8_dequantize(codes, scales, rows, cols, fmt, block_rows, out, bf16, None)


def matmul(a=A, fmt=0, s=S, M=8, w=W, ws=T, rows=144, cols=272, tr=0, a2=A2, b2=B2, R=16, c=C, work=None, n=0):
    return lib.nf4_fp8_matmul(a, fmt, s, M, w, ws, rows, cols, tr, a2, b2, R, c, work, n, None)


def grouped(a=A, fmt=0, s=S, M=8, w=W, ws=T, E=4, rows=144, cols=272, off=OFF, tr=0, a2=A2, b2=B2, R=16, c=C,
            work=None, n=0):
    return lib.nf4_fp8_matmul_grouped(a, fmt, s, M, w, ws, E, rows, cols, off, tr, a2, b2, R, c, work, n, None)


def norm(X=A, res=S, w=W, M=8, H=272, eps=1e-6, h=T, Y=C, codes=A2, scales=B2, rstd=OFF):
    return lib.nf4_rmsnorm_fwd(X, res, w, M, H, eps, h, Y, codes, scales, rstd, None)


def norm_grad(dY=A, h=S, w=W, rstd=T, dH=C, M=8, H=272, dX=A2, dw=B2, ws=OFF, n=1 << 20):
    return lib.nf4_rmsnorm_bwd(dY, h, w, rstd, dH, M, H, dX, dw, ws, n, None)


@pytest.mark.parametrize("call,inp,out", [(quantize, "X", "codes"), (dequantize, "codes", "out")])
def test_quantize_refuses(call, inp, out):
    assert call(fmt=2) == nf4.NF4_ERR_ARG and call(block_rows=64) == nf4.NF4_ERR_ARG
    for bad in ({"cols": 24}, {"rows": -1}, {"cols": -16}, {"cols": (1 << 22) + 16}, {"rows": (1 << 31), "cols": 1024}):
        assert call(**bad) == nf4.NF4_ERR_SHAPE, bad
    for p in (inp, "scales", out):
        assert call(**{p: None}) == nf4.NF4_ERR_NULL and call(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN
    assert call(**{out: A + 16}) == nf4.NF4_ERR_ALIAS
    assert call(rows=0) == nf4.NF4_OK and call(cols=0) == nf4.NF4_OK
    if call is quantize:
        assert call(scales=C + 16) == nf4.NF4_ERR_ALIAS  # scales inside the codes


@pytest.mark.parametrize("call", [matmul, grouped])
def test_products_refuse(call):
    assert call(fmt=2) == nf4.NF4_ERR_ARG and call(tr=2) == nf4.NF4_ERR_ARG
    for bad in ({"rows": 8}, {"cols": 24}, {"rows": 0}, {"cols": -16}, {"rows": (1 << 22) + 16}, {"M": -1},
                {"rows": 1 << 20, "cols": 1 << 13}, {"M": (1 << 31) + 1}, {"R": 8}, {"R": 272}, {"R": -16}):
        assert call(**bad) == nf4.NF4_ERR_SHAPE, bad
    ptrs = ["a", "s", "w", "ws", "a2", "b2", "c"] + (["off"] if call is grouped else [])
    for p in ptrs:
        assert call(**{p: None}) == nf4.NF4_ERR_NULL, p
        assert call(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    for p in ptrs[:-2] + ptrs[-1:]:
        if p != "c":
            assert call(c={"a": A, "s": S, "w": W, "ws": T, "a2": A2, "b2": B2, "off": OFF}[p]) == nf4.NF4_ERR_ALIAS, p
    assert call(M=0) == nf4.NF4_OK
    assert call(M=0, a=None, c=None) == nf4.NF4_OK


def test_product_workspace():
    n = ctypes.c_size_t()
    size = lib.nf4_fp8_matmul_workspace_bytes
    assert size(8, 144, 272, 0, 0, None) == nf4.NF4_ERR_NULL
    assert size(8, 144, 272, 2, 0, ctypes.byref(n)) == nf4.NF4_ERR_ARG
    for bad in ((8, 8, 272, 0, 0), (8, 144, 24, 0, 0), (-1, 144, 272, 0, 0), (8, 144, 272, 0, 4097), (8, 144, 272, 0, -1),
                ((1 << 30) + 1, 144, 272, 0, 4), ((1 << 31) + 1, 144, 272, 0, 0)):
        assert size(*bad, ctypes.byref(n)) == nf4.NF4_ERR_SHAPE, bad
    assert nf4.fp8_matmul_workspace_bytes(0, 144, 272) == 0
    # few tiles and a long contraction: split
    for call, E in ((matmul, 0), (grouped, 3)):
        need = nf4.fp8_matmul_workspace_bytes(260, 80, 33040, False, E)
        assert 0 < need <= 1 << 26
        big = {"M": 260, "rows": 80, "cols": 33040, **({"E": 3} if E else {})}
        assert call(**big, work=64 * GB * 10, n=need - 1) == nf4.NF4_ERR_WORKSPACE
        assert call(**big, work=64 * GB * 10 + 8, n=need) == nf4.NF4_ERR_ALIGN
        for at in (A, S, W, T, A2, B2, C):
            assert call(**big, work=at, n=need) == nf4.NF4_ERR_ALIAS


def test_grouped_refuses():
    for E in (0, -1, 4097):
        assert grouped(E=E) == nf4.NF4_ERR_SHAPE
    assert grouped(M=1 << 31) == nf4.NF4_ERR_SHAPE and grouped(M=(1 << 30) + 1) == nf4.NF4_ERR_SHAPE
    # more tiles than one launch holds
    assert grouped(M=1 << 30, rows=1 << 20, cols=16) == nf4.NF4_ERR_SHAPE
    # the last expert's weight counts as input
    assert grouped(c=W + 3 * 144 * 272) == nf4.NF4_ERR_ALIAS


def test_norm_refuses():
    for bad in ({"H": 24}, {"H": 0}, {"H": 32784}, {"M": -1}, {"M": (1 << 31) + 1}):
        assert norm(**bad) == nf4.NF4_ERR_SHAPE and norm_grad(**bad) == nf4.NF4_ERR_SHAPE, bad
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == nf4.NF4_ERR_ARG
    for bad in ({"X": None}, {"w": None}, {"h": None}, {"codes": None}, {"scales": None},
                {"Y": None, "codes": None, "scales": None}):
        assert norm(**bad) == nf4.NF4_ERR_NULL, bad
    for p in ("X", "res", "w", "h", "Y", "codes", "scales", "rstd"):
        assert norm(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    for bad in ({"Y": A}, {"h": S}, {"codes": A + 64}, {"rstd": W}, {"h": C + 16}):
        assert norm(**bad) == nf4.NF4_ERR_ALIAS, bad
    assert norm(M=0) == nf4.NF4_OK


def test_norm_grad_refuses():
    for p in ("dY", "h", "w", "rstd", "dX", "dw"):
        assert norm_grad(**{p: None}) == nf4.NF4_ERR_NULL, p
    for p in ("dY", "h", "w", "rstd", "dH", "dX", "dw", "ws"):
        assert norm_grad(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    need = nf4.rmsnorm_workspace_bytes(8, 272)
    assert norm_grad(n=need - 1) == nf4.NF4_ERR_WORKSPACE and norm_grad(ws=None) == nf4.NF4_ERR_WORKSPACE
    for bad in ({"dX": A}, {"dX": C}, {"dw": T}, {"ws": S}, {"dw": OFF + 16}):
        assert norm_grad(**bad) == nf4.NF4_ERR_ALIAS, bad


def test_norm_workspace_sizes():
    assert 0 < nf4.rmsnorm_workspace_bytes(0, 16) <= nf4.rmsnorm_workspace_bytes(1 << 31, 32768)
    n = ctypes.c_size_t()
    assert lib.nf4_rmsnorm_workspace_bytes(1, 272, None) == nf4.NF4_ERR_NULL
    assert lib.nf4_rmsnorm_workspace_bytes(1, 8, ctypes.byref(n)) == nf4.NF4_ERR_SHAPE


@needs_host_build
def test_refusals_sanitized(san_build):  # noqa: F811
    asan = subprocess.run([GXX, "-print-file-name=libasan.so"], stdout=subprocess.PIPE, text=True).stdout.strip()
    env = {**os.environ, **SAN_ENV, "NF4LORA_LIB": san_build[0], "LD_PRELOAD": asan}
    out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not sanitized",
                os.path.join(ROOT, "tests", "test_abi_fp8.py")], env=env, cwd=ROOT)
    assert "passed" in out and "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-3000:]


@needs_host_build
def test_sanitized_build_without_kernels_reports_hip(san_build):  # noqa: F811
    # a build without the kernels refuses a call that would launch one
    code = ("import tests.test_abi_fp8 as t; n = t.nf4.NF4_ERR_HIP; "
            "assert [t.quantize(), t.dequantize(), t.matmul(), t.grouped(), t.norm(), t.norm_grad()] == [n] * 6; print('ok')")
    asan = subprocess.run([GXX, "-print-file-name=libasan.so"], stdout=subprocess.PIPE, text=True).stdout.strip()
    env = {**os.environ, **SAN_ENV, "NF4LORA_LIB": san_build[0], "LD_PRELOAD": asan}
    assert "ok" in _run([sys.executable, "-c", code], env=env, cwd=ROOT)



@needs_host_build
def test_plan_units_sanitized(tmp_path):
    exe = str(tmp_path / "fp8_plan_units")
    _run([GXX, *COMMON, *SAN, "-o", exe, os.path.join(HOST, "fp8_plan_units.cpp"), os.path.join(CSRC, "plan.cpp")])
    assert "fp8 plan units: ok" in _run([exe], env={**os.environ, **SAN_ENV})
