"""Argument checks of the layer norm, the rows' sorting and the adapters in the C ABI (no GPU): every call here is refused,
or has nothing to do, before the library touches HIP, so the fake device addresses are compared and never read.  The same
checks run against a sanitized host build."""
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
P = [(i + 1) * 512 * GB for i in range(16)]  # aligned fake addresses, far apart
FOUR = ("s", "order", "offsets", "ids", "mean", "rstd", "scales", "xs")  # pointers that need 4 bytes


def odd(name):
    return 512 * GB * 20 + (2 if name in FOUR else 8)


def norm(X=P[0], res=P[1], w=P[2], b=P[3], M=8, H=272, eps=1e-5, h=P[4], Y=P[5], codes=P[6], scales=P[7], mean=P[8],
         rstd=P[9]):
    return lib.nf4_layernorm_fwd(X, res, w, b, M, H, eps, h, Y, codes, scales, mean, rstd, None)


def norm_grad(dY=P[0], h=P[1], w=P[2], mean=P[3], rstd=P[4], dH=P[5], M=8, H=272, dX=P[6], dw=P[7], db=P[8], ws=P[9],
              size=1 << 30):
    return lib.nf4_layernorm_bwd(dY, h, w, mean, rstd, dH, M, H, dX, dw, db, ws, size, None)


def route(ids=P[0], M=8, n=4, order=P[1], offsets=P[2], ws=P[3], size=1 << 40):
    return lib.nf4_route(ids, M, n, order, offsets, ws, size, None)


def fwd(X=P[0], M=400, L1=P[1], L2=P[2], s=P[3], n=4, o=144, h=272, r=16, order=P[4], offsets=P[5], base=P[6], Y=P[7],
        T=P[8], ws=P[9], size=1 << 40):
    return lib.nf4_adapters_fwd(X, M, L1, L2, s, n, o, h, r, order, offsets, base, Y, T, ws, size, None)


def bwd(X=P[0], xs=None, fmt=0, dY=P[1], T=P[2], M=400, L1=P[3], L2=P[4], s=P[5], n=4, o=144, h=272, r=16, order=P[6],
        offsets=P[7], base=P[8], dX=P[9], dL1=P[10], dL2=P[11], ws=P[12], size=1 << 40):
    return lib.nf4_adapters_bwd(X, xs, fmt, dY, T, M, L1, L2, s, n, o, h, r, order, offsets, base, dX, dL1, dL2, ws, size,
                                None)


def test_norm_refuses():
    for bad in ({"H": 24}, {"H": 0}, {"H": 32784}, {"M": -1}, {"M": (1 << 31) + 1}):
        assert norm(**bad) == nf4.NF4_ERR_SHAPE and norm_grad(**bad) == nf4.NF4_ERR_SHAPE, bad
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == nf4.NF4_ERR_ARG
    for bad in ({"X": None}, {"w": None}, {"h": None}, {"codes": None}, {"scales": None},
                {"Y": None, "codes": None, "scales": None}):
        assert norm(**bad) == nf4.NF4_ERR_NULL, bad
    for p in ("X", "res", "w", "b", "h", "Y", "codes", "scales", "mean", "rstd"):
        assert norm(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    for bad in ({"Y": P[0]}, {"h": P[1]}, {"codes": P[0] + 64}, {"rstd": P[2]}, {"mean": P[3]}, {"h": P[5] + 16},
                {"rstd": P[8]}):
        assert norm(**bad) == nf4.NF4_ERR_ALIAS, bad
    assert norm(M=0) == nf4.NF4_OK and norm(M=0, X=None, Y=None) == nf4.NF4_OK


def test_norm_grad_refuses():
    for p in ("dY", "h", "w", "mean", "rstd", "dX", "dw"):
        assert norm_grad(**{p: None}) == nf4.NF4_ERR_NULL, p
    for p in ("dY", "h", "w", "mean", "rstd", "dH", "dX", "dw", "db", "ws"):
        assert norm_grad(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    need = nf4.layernorm_workspace_bytes(8, 272)
    assert norm_grad(size=need - 1) == nf4.NF4_ERR_WORKSPACE and norm_grad(ws=None) == nf4.NF4_ERR_WORKSPACE
    for bad in ({"dX": P[0]}, {"dX": P[5]}, {"dw": P[4]}, {"db": P[3]}, {"ws": P[1]}, {"db": P[7] + 16}, {"ws": P[6]}):
        assert norm_grad(**bad) == nf4.NF4_ERR_ALIAS, bad
    n = ctypes.c_size_t()
    assert lib.nf4_layernorm_workspace_bytes(1, 272, None) == nf4.NF4_ERR_NULL
    assert lib.nf4_layernorm_workspace_bytes(1, 8, ctypes.byref(n)) == nf4.NF4_ERR_SHAPE
    assert 0 < nf4.layernorm_workspace_bytes(0, 16) <= nf4.layernorm_workspace_bytes(1 << 31, 32768)


def test_route_refuses():
    n = ctypes.c_size_t()
    size = lib.nf4_route_workspace_bytes
    for bad in ({"M": -1}, {"M": (1 << 30) + 1}, {"n": 0}, {"n": -1}, {"n": 4097}):
        assert route(**bad) == nf4.NF4_ERR_SHAPE, bad
        assert size(bad.get("M", 8), bad.get("n", 4), ctypes.byref(n)) == nf4.NF4_ERR_SHAPE, bad
    assert size(8, 4, None) == nf4.NF4_ERR_NULL
    for p in ("ids", "order", "offsets"):
        assert route(**{p: None}) == nf4.NF4_ERR_NULL, p
        assert route(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    assert route(M=0, ids=None, order=None, offsets=None) == nf4.NF4_ERR_NULL  # offsets are written all the same
    assert nf4.route_workspace_bytes(0, 4) == nf4.route_workspace_bytes(1000, 64) == 0
    need = nf4.route_workspace_bytes(1 << 20, 64)
    assert 0 < need <= 1 << 24
    big = {"M": 1 << 20, "n": 64}
    assert route(**big, size=need - 1) == nf4.NF4_ERR_WORKSPACE and route(**big, ws=None) == nf4.NF4_ERR_WORKSPACE
    assert route(**big, ws=odd("ws")) == nf4.NF4_ERR_ALIGN
    for bad in ({"order": P[0]}, {"offsets": P[0] + 16}, {"order": P[2]}, {"ws": P[0]}, {"ws": P[2] + 16}):
        assert route(**big, **bad) == nf4.NF4_ERR_ALIAS, bad


SHAPES = ({"M": -1}, {"M": (1 << 26) + 1}, {"n": 0}, {"n": 4097}, {"o": 0}, {"o": 24}, {"o": (1 << 22) + 16}, {"h": 8},
          {"h": -16}, {"h": (1 << 22) + 16}, {"r": 0}, {"r": 4}, {"r": 12}, {"r": 264})


@pytest.mark.parametrize("call", [fwd, bwd])
def test_adapters_refuse(call):
    for bad in SHAPES:
        assert call(**bad) == nf4.NF4_ERR_SHAPE, bad
    needed = ["X", "L1", "L2", "s", "offsets"] + (["Y"] if call is fwd else ["dY", "T", "dL1", "dL2"])
    for p in needed:
        assert call(**{p: None}) == nf4.NF4_ERR_NULL, p
    for p in needed + ["order", "base", "ws", "T" if call is fwd else "dX"]:
        assert call(**{p: odd(p)}) == nf4.NF4_ERR_ALIGN, p
    need = nf4.adapters_workspace_bytes(nf4.NF4_OP_FWD if call is fwd else nf4.NF4_OP_BWD, 400, 144, 272, 4, 16)
    assert need > 0
    assert call(size=need - 1) == nf4.NF4_ERR_WORKSPACE and call(ws=None) == nf4.NF4_ERR_WORKSPACE


def test_adapters_aliases():
    for bad in ({"Y": P[0]}, {"Y": P[6] + 16}, {"T": P[0]}, {"T": P[7]}, {"ws": P[6]}, {"ws": P[8]}, {"Y": P[5]},
                {"T": P[4]}, {"Y": P[1] + 64}, {"ws": P[2] + 16 * 4 * 144 * 2 - 16}):
        assert fwd(**bad) == nf4.NF4_ERR_ALIAS, bad
    for bad in ({"dX": P[0]}, {"dX": P[8] + 16}, {"dX": P[1]}, {"dL1": P[3]}, {"dL2": P[10]}, {"dL1": P[11]},
                {"ws": P[2]}, {"ws": P[9]}, {"dL2": P[7]}, {"dL1": P[6]}, {"dL2": P[5]}):
        assert bwd(**bad) == nf4.NF4_ERR_ALIAS, bad
    # codes are one byte each: what follows them is free, and their scales are inputs
    assert bwd(xs=P[13], dX=P[0] + 400 * 272 - 16) == nf4.NF4_ERR_ALIAS
    assert bwd(xs=P[13], dX=P[13]) == nf4.NF4_ERR_ALIAS
    # a few rows of a small rank need no workspace: whatever is given is not looked at
    assert nf4.adapters_workspace_bytes(nf4.NF4_OP_FWD, 40, 144, 272, 4, 16) == 0
    assert fwd(M=40, ws=odd("ws"), Y=P[0]) == fwd(M=40, ws=P[0], Y=P[0]) == nf4.NF4_ERR_ALIAS


def test_adapters_formats():
    assert bwd(xs=P[13], fmt=2) == nf4.NF4_ERR_ARG and bwd(xs=P[13], fmt=-1) == nf4.NF4_ERR_ARG
    assert bwd(xs=odd("xs")) == nf4.NF4_ERR_ALIGN


def test_adapters_without_rows():
    assert fwd(M=0, X=None, Y=None, ws=None) == nf4.NF4_OK
    assert bwd(M=0, dL1=None) == nf4.NF4_ERR_NULL and bwd(M=0, dL2=odd("dL2")) == nf4.NF4_ERR_ALIGN
    assert bwd(M=0, dL2=P[10] + 64) == nf4.NF4_ERR_ALIAS


def test_adapters_workspace():
    n = ctypes.c_size_t()
    size = lib.nf4_adapters_workspace_bytes
    assert size(nf4.NF4_OP_FWD, 40, 144, 272, 4, 16, None) == nf4.NF4_ERR_NULL
    for op in (0, 3):
        assert size(op, 40, 144, 272, 4, 16, ctypes.byref(n)) == nf4.NF4_ERR_ARG
    d = {"M": 40, "o": 144, "h": 272, "n": 4, "r": 16}
    for op in (nf4.NF4_OP_FWD, nf4.NF4_OP_BWD):
        for bad in SHAPES:
            a = {**d, **bad}
            assert size(op, a["M"], a["o"], a["h"], a["n"], a["r"], ctypes.byref(n)) == nf4.NF4_ERR_SHAPE, bad
        assert nf4.adapters_workspace_bytes(op, 0, 144, 272, 4, 16) == 0
    # one token of a small rank needs none in the forward pass
    assert nf4.adapters_workspace_bytes(nf4.NF4_OP_FWD, 1, 4096, 4096, 64, 16) == 0
    assert nf4.adapters_workspace_bytes(nf4.NF4_OP_FWD, 1, 4096, 4096, 64, 24) > 0
    # the largest call's is no more than its gradients' and its rows' own
    M, o, r = 1 << 26, 1 << 22, 256
    most = nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, M, o, o, 4096, r)
    assert 0 < most < 6 * 4096 * r * 2 * o * 4 + 16 * M * r * 4


@needs_host_build
def test_refusals_sanitized(san_build):  # noqa: F811
    asan = subprocess.run([GXX, "-print-file-name=libasan.so"], stdout=subprocess.PIPE, text=True).stdout.strip()
    env = {**os.environ, **SAN_ENV, "NF4LORA_LIB": san_build[0], "LD_PRELOAD": asan}
    out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not sanitized",
                os.path.join(ROOT, "tests", "test_abi_adapters.py")], env=env, cwd=ROOT)
    assert "passed" in out and "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-3000:]


@needs_host_build
def test_sanitized_build_without_kernels_reports_hip(san_build):  # noqa: F811
    # a build without the kernels refuses a call that would launch one
    code = ("import tests.test_abi_adapters as t; n = t.nf4.NF4_ERR_HIP; "
            "assert [t.norm(), t.norm_grad(), t.route(), t.fwd(), t.bwd()] == [n] * 5; print('ok')")
    asan = subprocess.run([GXX, "-print-file-name=libasan.so"], stdout=subprocess.PIPE, text=True).stdout.strip()
    env = {**os.environ, **SAN_ENV, "NF4LORA_LIB": san_build[0], "LD_PRELOAD": asan}
    assert "ok" in _run([sys.executable, "-c", code], env=env, cwd=ROOT)


@needs_host_build
def test_plan_units_sanitized(tmp_path):
    exe = str(tmp_path / "adapter_plan_units")
    _run([GXX, *COMMON, *SAN, "-o", exe, os.path.join(HOST, "adapter_plan_units.cpp"), os.path.join(CSRC, "plan.cpp")])
    assert "adapter plan units: ok" in _run([exe], env={**os.environ, **SAN_ENV})
