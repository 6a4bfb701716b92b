"""The norm where its 8-bit output and its sums can go wrong, against the fp64 oracle (needs an MI355X): zero blocks and
tiny or huge rows at any eps, and every width held to the stated precision.

y is formed in fp32 with one rounding, 2^-24 of its value, and rstd likewise.  Then, relative to the value:
- Y: half a step of bf16, 2^-8, of a value that is 2^-24 off: 2^-8 * (1 + 2^-8) covers both.
- scales: the largest |y| of the block (2^-24) over 448 (another 2^-24).
- codes: half a step of e4m3, 2^-4 of the value, or of the least step of 2^-9, of a value that is a few 2^-24 off
  (y, the multiplier's two roundings and the scale's): the factor 1 + 2^-8 covers these.
"""
import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

try:
    import quantized_lora_fine_amd as nf4
except ImportError as exc:
    if torch.cuda.is_available():
        raise
    pytest.skip(f"libnf4lora.so not loaded: {exc}", allow_module_level=True)

DEV = "cuda"
ONE = 2.0 ** -24 * (1 + 2.0 ** -16)  # a fp32 rounding, and what is left of 64-bit sums and of rstd's second part


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def bf16_np(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def check_norm(X, w, eps, R=None):
    """All outputs of the rows X against the oracle; returns (codes as bytes, Y)."""
    Y, h, codes, scales, rstd = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), eps, None if R is None else R.to(DEV),
                                                want_fp8=True, want_rstd=True)
    hw = X if R is None else (X.float() + R.float()).to(torch.bfloat16)
    if R is not None:
        assert torch.equal(h.cpu().view(torch.int16), hw.view(torch.int16))
    M, H = X.shape
    y, r = fp8.rmsnorm(f64(hw), f64(w), float(np.float32(eps)))
    # rstd: below fp32's normal values half of their step as well, past its range an infinity
    with np.errstate(over="ignore"):
        far = np.isinf(r.astype(np.float32))
    got = f64(rstd)
    assert np.all(np.isinf(got[far])) and np.all(np.abs(got[~far] - r[~far]) <= r[~far] * ONE + 2.0 ** -149)
    assert np.all(np.abs(f64(Y) - y) <= np.abs(y) * 2.0 ** -8 * (1 + 2.0 ** -8))
    by_block = np.stack([np.abs(y[:, j:j + 128]).max(1) for j in range(0, H, 128)], 1)
    want = np.maximum(by_block, 2.0 ** -100) / 448
    assert np.all(np.abs(f64(scales) - want) <= want * 2 * ONE)
    b = codes.view(torch.uint8).cpu().numpy()
    assert np.all((b & 0x7F) != 0x7F), "a NaN code"
    assert np.all((b & 0x7F)[y == 0] == 0)
    d = f64(nf4.fp8_dequantize(codes, scales))
    step = fp8._spread(want, 1, M, H) * 2.0 ** -10
    assert np.all(np.abs(d - y) <= np.maximum(np.abs(y) * 2.0 ** -4, step) * (1 + 2.0 ** -8))
    return b, Y


@pytest.mark.parametrize("H", [16, 272, 1040, 4096, 8208, 16400])
@pytest.mark.parametrize("eps", [1e-6, 1e-11, 1e-12, 1e-30])
def test_rows_of_zeros(H, eps):
    # padding: y and the codes are zeros whatever the rstd, which is up to 1e15 here
    X = torch.zeros(5, H, dtype=torch.bfloat16)
    w = bf16_np(1 + 0.1 * np.random.default_rng(H).standard_normal(H))
    X[3] = bf16_np(np.random.default_rng(1).standard_normal(H))
    b, Y = check_norm(X, w, eps)
    for i in (0, 1, 2, 4):
        assert np.all((b[i] & 0x7F) == 0) and torch.all(Y[i] == 0)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-12])
@pytest.mark.parametrize("H", [272, 1040, 4096, 8208, 16400])
@pytest.mark.parametrize("scale", [1e37, 1e18, 1.0, 1e-5, 1e-7, 1e-18, 2.0 ** -120, 2.0 ** -126, 2.0 ** -131])
def test_a_zero_block_beside_others(scale, H, eps):
    # a block of zeros in the row, one of zero weights, blocks far smaller than the row; down to bf16's subnormals
    rng = np.random.default_rng(H)
    x = np.clip(rng.standard_normal((6, H)) * scale, -3.3e38, 3.3e38)
    x[1, :128] = 0
    x[2, H - H % 128 or H - 128:] = 0
    x[3, :128] *= 1e-30
    X, w = bf16_np(x), bf16_np(1 + 0.1 * rng.standard_normal(H))
    w[128:256] = 0
    w[7] = 60.0  # the row's size times its weight goes past fp32's largest value
    if scale == 2.0 ** -131:  # a few values of the subnormal grid: none of the rows may be all zeros
        X[:, 9] = 2.0 ** -131
    check_norm(X, w, eps)


@pytest.mark.parametrize("H", [64, 272, 2064])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -34, 2.0 ** -36, 1e-9])
def test_rows_of_every_power(H, eps):
    # one launch of rows whose sizes differ by powers of two, some zeros among them: neighbours in a wave may differ
    rng = np.random.default_rng(H)
    x = rng.standard_normal((161, H)) * 2.0 ** np.arange(-40, 121, dtype=np.float64)[:, None]
    x[::3, :min(H // 2, 128)] = 0
    if eps:
        x[5::16] = 0
    w = bf16_np(1 + 0.1 * rng.standard_normal(H))
    check_norm(bf16_np(x[:160]), w, eps)
    check_norm(bf16_np(x[160:]), w, eps)


@pytest.mark.parametrize("value", [2.0 ** -133, 2.0 ** -126, 2.0 ** -125, 2.0 ** 127])
@pytest.mark.parametrize("H", [16, 144, 4096])
def test_rows_of_one_value_without_eps(H, value):
    # 1 / rms is past fp32's range for the smallest; y is the weight all the same
    X = torch.full((3, H), value, dtype=torch.bfloat16)
    X[1] *= -1
    w = bf16_np(1 + 0.1 * np.random.default_rng(3).standard_normal(H))
    _, Y = check_norm(X, w, 0.0)
    assert torch.equal(Y[0].cpu().view(torch.int16), w.view(torch.int16)) and torch.equal(Y[1], -Y[0])


@pytest.mark.parametrize("H", [272, 4096])
def test_codes_of_small_rows_through_a_product(H):
    # a padded row stays zero in the product of its codes, and alone
    rng = np.random.default_rng(2)
    X = bf16_np(rng.standard_normal((7, H)))
    X[2], X[6] = 0, 0
    w = torch.ones(H, dtype=torch.bfloat16)
    _, _, codes, scales, _ = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), 1e-12, want_y=False, want_fp8=True)
    W, ws = nf4.fp8_quantize(torch.from_numpy(rng.standard_normal((144, H)).astype(np.float32)).to(DEV), 128)
    C = nf4.fp8_matmul(codes, scales, W, ws)
    assert torch.isfinite(C).all() and torch.all(C[2] == 0) and torch.all(C[6] == 0) and torch.all(C[1] != 0)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M", [1, 21])
@pytest.mark.parametrize("H", [16, 128, 144, 512, 528, 1024, 1040, 2048, 2064, 4096, 5120, 8192, 8208, 16384, 16400, 32768])
def test_every_width_to_one_rounding(H, M, residual):
    rng = np.random.default_rng(M + H)
    rows = lambda: bf16_np(rng.standard_normal((M, H)) * np.exp(3 * rng.standard_normal((M, 1))))
    check_norm(rows(), bf16_np(1 + 0.1 * rng.standard_normal(H)), 1e-6, rows() if residual else None)
