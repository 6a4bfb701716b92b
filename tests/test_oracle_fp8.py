"""The 8-bit oracle on its own (CPU): its grids and rounding against torch's 8-bit types, the norm's gradient
against differences of its forward."""
import numpy as np
import pytest
import torch

from oracle import fp8

DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_values(fmt):
    want = torch.arange(256, dtype=torch.uint8).view(DTYPES[fmt]).to(torch.float64).numpy()
    assert np.array_equal(fp8.code_values(fmt), want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode(fmt):
    rng = np.random.default_rng(1)
    vals = fp8.code_values(fmt)
    grid = np.unique(np.abs(vals[np.isfinite(vals)]))
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        rng.uniform(0, grid[-1], 5000), np.exp(rng.uniform(np.log(1e-9), np.log(grid[-1]), 5000))])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(DTYPES[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(x, fmt), want)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_error(fmt, block_rows):
    # half a step of the code, or of the smallest code, plus the two fp32 roundings
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((200, 272)) * np.exp(rng.standard_normal((200, 1)))).astype(np.float32)
    codes, scales = fp8.quantize(x, block_rows, fmt)
    man, bias, _ = fp8.FORMATS[fmt]
    s = fp8._spread(scales.astype(np.float64), block_rows, *x.shape)
    d = fp8.code_values(fmt)[codes] * s
    bound = np.maximum(np.abs(x) * 2.0 ** -(man + 1), s * 2.0 ** (-bias - man)) * (1 + 2.0 ** -20)
    assert np.all(np.abs(d - x) <= bound)


def test_rmsnorm_grad_by_differences():
    rng = np.random.default_rng(3)
    h, w, dy = rng.standard_normal((5, 48)), rng.standard_normal(48), rng.standard_normal((5, 48))
    eps, d = 1e-5, 1e-5
    f = lambda hh, ww: float(np.sum(fp8.rmsnorm(hh, ww, eps)[0] * dy))
    dx, dw = fp8.rmsnorm_grad(dy, h, w, fp8.rmsnorm(h, w, eps)[1])
    for i, j in [(0, 0), (2, 17), (4, 47)]:
        p, m = h.copy(), h.copy()
        p[i, j] += d
        m[i, j] -= d
        assert abs((f(p, w) - f(m, w)) / (2 * d) - dx[i, j]) < 1e-8
    for j in (0, 31):
        p, m = w.copy(), w.copy()
        p[j] += d
        m[j] -= d
        assert abs((f(h, p) - f(h, m)) / (2 * d) - dw[j]) < 1e-8


def test_matmul_both_ways():
    rng = np.random.default_rng(4)
    W = rng.standard_normal((144, 272)).astype(np.float32)
    w, ws = fp8.quantize(W, 128, "e4m3")
    Wd = fp8.dequantize(w, ws, 128, "e4m3").astype(np.float64)
    for tr, K in ((False, 272), (True, 144)):
        a, s = fp8.quantize(rng.standard_normal((7, K)).astype(np.float32), 1, "e5m2")
        Ad = fp8.dequantize(a, s, 1, "e5m2").astype(np.float64)
        C, _, _ = fp8.matmul(a, s, "e5m2", w, ws, tr)
        want = sum(Ad[:, k:k + 1] * (Wd[k] if tr else Wd[:, k])[None] for k in range(K))
        assert np.allclose(C, want, rtol=1e-6, atol=1e-6 * np.abs(want).max())
