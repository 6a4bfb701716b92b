"""8-bit storage, its products and the norm against the fp64 oracle (needs an MI355X).

Codes, scales, dequantized values and the norm's residual sum are bit-exact.
Computed outputs are held to the roundings they go through: half a step of the
output's type relative to the value, plus fp32 accumulation in proportion to the
sum of the terms' magnitudes.  EPS32 is one fp32 step, taken per addition (the
matrix cores' order of the 128 products of a block is theirs).
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
DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BF16 = 2.0 ** -8      # half a step, relative
E4M3 = 2.0 ** -4
EPS32 = 2.0 ** -23


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def bf16_np(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def rows_of(rng, rows, cols):
    """Activations: token sizes that differ, a few channels far larger."""
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    x[:, rng.integers(0, cols, max(1, cols // 100))] *= 30
    return x.astype(np.float32)


def check_within(name, got, want, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = np.abs(got - want) / np.maximum(bound, 1e-300)
    worst = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    print(f"  {name}: {off.max() if off.size else 0:.3f} of the bound", flush=True)
    assert np.all(np.abs(got - want) <= bound), (name, worst, got[worst], want[worst], bound[worst])


# ---------------------------------------------------------------------------------------------------------
# quantization
# ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 272), (127, 128), (129, 1040), (260, 384)])
def test_quantize(rows, cols, bf16, block_rows, fmt):
    rng = np.random.default_rng(rows * 7 + cols)
    x = rows_of(rng, rows, cols)
    t = bf16_np(x) if bf16 else torch.from_numpy(x)
    x = t.float().numpy()
    codes, scales = nf4.fp8_quantize(t.to(DEV), block_rows, DTYPES[fmt])
    want, ws = fp8.quantize(x, block_rows, fmt)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    assert np.array_equal(bits(codes), want)
    d = nf4.fp8_dequantize(codes, scales, block_rows)
    dw = fp8.dequantize(want, ws, block_rows, fmt)
    assert np.array_equal(d.cpu().numpy().view(np.uint32), dw.view(np.uint32))
    db = nf4.fp8_dequantize(codes, scales, block_rows, bf16=True)
    assert torch.equal(db.cpu().view(torch.int16), bf16_np(dw).view(torch.int16))


@pytest.mark.parametrize("fmt,most", [("e4m3", 448.0), ("e5m2", 57344.0)])
def test_quantize_as_an_array_expression(fmt, most):
    # enough values that a multiplier off by its last bit would move some codes over a tie
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(4096, 4096, generator=g, device=DEV)
    b = x.view(4096, 32, 128)
    amax = b.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    codes, _ = nf4.fp8_quantize(x, 1, DTYPES[fmt])
    assert np.array_equal(bits(codes), bits((b * (most / amax)).to(DTYPES[fmt]).view(4096, 4096)))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_every_code_and_tie(fmt):
    # a block whose largest value is F has scale 1: its codes are the rounding itself
    vals = fp8.code_values(fmt)
    grid = np.unique(np.abs(vals[np.isfinite(vals)]))
    mid = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    x = np.concatenate([grid, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    x = np.concatenate([x, -x]).astype(np.float32)
    x = x[np.abs(x) <= grid[-1]]
    per = 127
    n = -(-x.size // per)
    X = np.zeros((n, 128), np.float32)
    X[:, 0] = grid[-1]
    X[:, 1:].reshape(-1)[:] = 0
    flat = np.zeros(n * per, np.float32)
    flat[:x.size] = x
    X[:, 1:] = flat.reshape(n, per)
    for block_rows in (1, 128):
        codes, scales = nf4.fp8_quantize(torch.from_numpy(X).to(DEV), block_rows, DTYPES[fmt])
        assert torch.all(scales == 1)
        assert np.array_equal(bits(codes), fp8.encode(X, fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_edges(block_rows, fmt):
    x = np.zeros((130, 272), np.float32)
    x[0, 1] = 3e38                     # the largest magnitudes
    x[129, 130] = 2.0 ** -120          # below the floor
    x[129, 131] = 1e-42                # subnormal
    x[0, 256:] = np.float32(2.0 ** -100)
    x[1, 140] = np.nan                 # a NaN alone keeps its block's scale
    x[1, 141] = -2.0
    codes, scales = nf4.fp8_quantize(torch.from_numpy(x).to(DEV), block_rows, DTYPES[fmt])
    want, ws = fp8.quantize(x, block_rows, fmt)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    v, vw = f64(codes), fp8.code_values(fmt)[want]
    assert np.array_equal(v, vw, equal_nan=True)
    x[2, 5] = np.inf
    codes, scales = nf4.fp8_quantize(torch.from_numpy(x).to(DEV), block_rows, DTYPES[fmt])
    d = nf4.fp8_dequantize(codes, scales, block_rows).cpu().numpy()
    block = d[2:3, :128] if block_rows == 1 else d[:128, :128]
    assert np.all(np.isnan(block)) and np.all(np.isfinite(d[129, :128]))


# ---------------------------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------------------------

WIDTHS = [16, 128, 144, 512, 528, 2048, 2064, 4096, 5120, 8192, 8208, 16400, 32768]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,H", [(1, h) for h in WIDTHS] + [(5, h) for h in WIDTHS] + [(300, 272), (67, 4096)])
def test_rmsnorm(M, H, residual):
    rng = np.random.default_rng(M + H)
    eps = 1e-6
    X, w = bf16_np(rows_of(rng, M, H)), bf16_np(1 + 0.1 * rng.standard_normal(H))
    R = bf16_np(rows_of(rng, M, H)) if residual else None
    Y, h, codes, scales, rstd = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), eps, R.to(DEV) if residual else None,
                                                want_fp8=True, want_rstd=True)
    hw = X if R is None else (X.float() + R.float()).to(torch.bfloat16)
    assert (h is None) == (R is None)
    if R is not None:
        assert torch.equal(h.cpu().view(torch.int16), hw.view(torch.int16))
    y, r = fp8.rmsnorm(f64(hw), f64(w), eps)
    # the sum of squares: at most 32 terms a thread, then a tree, halved by the root
    acc = 32 * EPS32
    check_within("rstd", rstd, r, np.abs(r) * acc)
    check_within("y", Y, y, np.abs(y) * (BF16 * (1 + 2.0 ** -8) + acc))
    sw = np.maximum(np.abs(fp8._spread(fp8.block_scales(y.astype(np.float32), 1, "e4m3")[0], 1, M, H)), 0)
    check_within("scales", scales, fp8.block_scales(y.astype(np.float32), 1, "e4m3")[0].astype(np.float64),
                 scales.double().cpu().numpy() * 2 * acc)
    d = nf4.fp8_dequantize(codes, scales)
    check_within("codes", d, y, np.maximum(np.abs(y) * E4M3, sw * 2.0 ** -10) * (1 + 2.0 ** -8) + np.abs(y) * acc)
    # each output alone is what it is beside the other
    Y1 = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), eps, R.to(DEV) if residual else None)[0]
    assert torch.equal(Y1.view(torch.int16), Y.view(torch.int16))
    _, _, c1, s1, _ = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), eps, R.to(DEV) if residual else None, want_y=False,
                                      want_fp8=True)
    assert np.array_equal(bits(c1), bits(codes)) and torch.equal(s1, scales)


def test_rmsnorm_any_magnitude():
    # squares past and below fp32's range; an infinity or NaN stays in its row
    rng = np.random.default_rng(6)
    M, H = 12, 1040
    x = rng.standard_normal((M, H)) * np.array([1e30, 1e25, 1e19, 1e18, 1, 1e-10, 1e-18, 1e-19, 1e-22, 1e-30, 1, 1])[:, None]
    X, w = bf16_np(x), bf16_np(1 + 0.1 * rng.standard_normal(H))
    X[10, 7], X[11, 9] = float("inf"), float("nan")
    Y, _, codes, scales, rstd = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), 0.0, want_fp8=True, want_rstd=True)
    y, r = fp8.rmsnorm(f64(X[:10]), f64(w), 0.0)
    check_within("rstd", rstd[:10], r, np.abs(r) * 2.0 ** -24 * (1 + 2.0 ** -16))
    check_within("y", Y[:10], y, np.abs(y) * BF16 * (1 + 2.0 ** -8))
    d = f64(nf4.fp8_dequantize(codes, scales)[:10])
    sw = fp8._spread(fp8.block_scales(y.astype(np.float32), 1, "e4m3")[0], 1, 10, H)
    assert np.all(np.abs(d - y) <= np.maximum(np.abs(y) * E4M3, sw * 2.0 ** -10) * (1 + 2.0 ** -8))
    assert torch.isnan(Y[10, 7]) and torch.isnan(Y[11]).all() and float(rstd[10]) == 0 and torch.isnan(rstd[11])


def test_rmsnorm_rounds_once():
    # codes against those of y in 64 bits: a fp32 value of y and its product with the multiplier, at most 2^-23 off
    # together, move a value over a tie where it lies within 2^-23 * |v| of one; ties are 2^-4 |v| apart or more, so
    # at most 2 * 2^-23 * 2^4 of the values lie there: 4 of a million, 1.3 of these.  (With rstd and the
    # two products in fp32 as well, it is 50 of a million.)
    rng = np.random.default_rng(5)
    M, H = 84, 4096
    X, w = bf16_np(rows_of(rng, M, H)), bf16_np(1 + 0.1 * rng.standard_normal(H))
    _, _, codes, _, rstd = nf4.rmsnorm_fwd(X.to(DEV), w.to(DEV), 1e-6, want_y=False, want_fp8=True, want_rstd=True)
    y, r = fp8.rmsnorm(f64(X), f64(w), 1e-6)
    _, mul = fp8.block_scales(y.astype(np.float32), 1, "e4m3")
    want = fp8.encode((y * fp8._spread(mul, 1, M, H).astype(np.float64)).astype(np.float32), "e4m3")
    assert np.sum(bits(codes) != want) <= 6  # of 1.3 expected at most, more than 6 in one of 10^3 draws
    check_within("rstd", rstd, r, np.abs(r) * 2.0 ** -24 * (1 + 2.0 ** -16))


def test_rmsnorm_rows_of_zeros():
    X = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    X[1] = 2.0
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    Y, _, codes, scales, rstd = nf4.rmsnorm_fwd(X, w, 1e-6, want_fp8=True, want_rstd=True)
    assert torch.all(Y[0] == 0) and torch.all(Y[1] == 1)
    assert torch.all(codes[0].float() == 0)
    assert abs(float(rstd[0]) - 1000.0) < 1e-2
    Y, _, _, _, _ = nf4.rmsnorm_fwd(X, w, 0.0)
    assert torch.all(torch.isnan(Y[0])) and torch.all(Y[1] == 1)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("M,H", [(1, h) for h in WIDTHS] + [(37, h) for h in (16, 144, 528, 2064, 5120, 8208, 16400)] +
                         [(2500, 144), (1100, 1040), (700, 4096), (1999, 5120)])
def test_rmsnorm_grad(M, H, with_dh):
    rng = np.random.default_rng(M * 3 + H)
    h, w = bf16_np(rows_of(rng, M, H)), bf16_np(1 + 0.1 * rng.standard_normal(H))
    dy = bf16_np(1e-3 * rows_of(rng, M, H))
    dh = bf16_np(1e-3 * rows_of(rng, M, H)) if with_dh else None
    _, r = fp8.rmsnorm(f64(h), f64(w), 1e-6)
    rstd = torch.from_numpy(r.astype(np.float32))
    dX, dw = nf4.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh.to(DEV) if with_dh else None)
    r = f64(rstd)
    dx64, dw64 = fp8.rmsnorm_grad(f64(dy), f64(h), f64(w), r, f64(dh) if with_dh else None)
    u, xhat = np.abs(f64(dy) * f64(w)), np.abs(f64(h)) * r[:, None]
    size = r[:, None] * (u + xhat * np.mean(u * xhat, 1, keepdims=True))
    # the dot product: at most 64 additions deep; then a handful of roundings
    check_within("dx", dX, dx64, np.abs(dx64) * BF16 * (1 + 2.0 ** -8) + size * 40 * EPS32)
    # dw: the rows of one workgroup in turn (at most ceil(M / 512)), 256 / 16 teams, then the parts
    deep = -(-M // 512) + 16 + 64
    check_within("dw", dw, dw64, np.sum(np.abs(f64(dy)) * xhat, 0) * deep * EPS32)
    dX2, dw2 = nf4.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh.to(DEV) if with_dh else None)
    assert torch.equal(dX2.view(torch.int16), dX.view(torch.int16)) and torch.equal(dw2, dw)


# ---------------------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------------------

def product_case(seed, M, o, h, transpose, R, fmt, experts=None):
    rng = np.random.default_rng(seed)
    K, N = (o, h) if transpose else (h, o)
    a, s = fp8.quantize(rows_of(rng, M, K), 1, fmt) if M else (np.zeros((0, K), np.uint8),
                                                                np.zeros((0, -(-K // 128)), np.float32))
    many = experts or 1
    w, ws, b2 = [], [], []
    for _ in range(many):
        c, t = fp8.quantize((0.02 * rows_of(rng, o, h)), 128, "e4m3")
        w.append(c)
        ws.append(t)
        b2.append(bf16_np(0.05 * rng.standard_normal((N, R))))
    A2 = bf16_np(rng.standard_normal((M, R))) if R else None
    return a, s, w, ws, A2, (b2 if R else None)


def t8(c, fmt="e4m3"):
    return torch.from_numpy(np.ascontiguousarray(c)).to(DEV).view(DTYPES[fmt])


def check_product(C, oracle, K, R):
    """The matrix cores add the products of 8 neighbouring k aligned to the largest, p, of them and cut each off
    below 2^-13 p; the groups of 8 are added in fp32.  So a group is off by less than 7 * 2^-13 p, p at most the sum
    of the group's magnitudes: in all by less than 7 * 2^-13 S, and fp32 additions.  For the whole result: a product
    of a group is cut by something between 0 and 2^-13 p, of either sign, whose square is 2^-26 p^2 / 3 on average, and
    p^2 is at most the sum of the group's squares: a root mean square of at most 2^-13 sqrt(7 / 3) Q.  A rounding to bf16
    is evenly spread up to 2^-8 of the value: a mean square of 2^-16 / 3 of its square."""
    want, S, Q = oracle
    check_within("C", C, want, np.abs(want) * BF16 * (1 + 2.0 ** -8) +
                 S * (7 * 2.0 ** -13 + (128 + 2 * (K // 128 + 1) + R) * EPS32))
    # each value's error over its own expectation, so that no large value stands for all
    expected = want ** 2 * BF16 ** 2 / 3 + Q ** 2 * 2.0 ** -26 * 7 / 3
    rms = np.sqrt(np.mean((f64(C) - want) ** 2 / np.maximum(expected, 1e-300)))
    print(f"  rms: {rms:.3f} of its bound", flush=True)
    assert rms <= 1 + 4 / np.sqrt(want.size)  # a mean over few values strays from its expectation


SHAPES = [  # M, o, h
    (1, 16, 16), (1, 272, 400), (1, 1024, 4096), (2, 144, 528), (5, 400, 272), (16, 528, 1040), (17, 512, 512),
    (31, 272, 2064), (33, 1040, 656), (64, 256, 384), (65, 384, 256), (100, 144, 144), (128, 128, 128),
    (129, 160, 1296), (255, 400, 272), (257, 272, 528), (513, 784, 400), (700, 2064, 1040),
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,fmt", [(0, "e4m3"), (16, "e4m3"), (48, "e5m2"), (256, "e4m3")])
@pytest.mark.parametrize("M,o,h", SHAPES)
def test_matmul(M, o, h, R, fmt, transpose):
    a, s, w, ws, A2, B2 = product_case(M * 5 + o + h, M, o, h, transpose, R, fmt)
    want = fp8.matmul(a, s, fmt, w[0], ws[0], transpose, f64(A2) if R else None, f64(B2[0]) if R else None)
    args = (t8(a, fmt), torch.from_numpy(s).to(DEV), t8(w[0]), torch.from_numpy(ws[0]).to(DEV), transpose,
            A2.to(DEV) if R else None, B2[0].to(DEV) if R else None)
    C = nf4.fp8_matmul(*args)
    check_product(C, want, h if not transpose else o, R)
    assert torch.equal(nf4.fp8_matmul(*args).view(torch.int16), C.view(torch.int16))


@pytest.mark.parametrize("M,N,K", [(1, 48, 33024), (3, 272, 16400), (17, 144, 33040), (40, 80, 65680), (64, 272, 8208),
                                   (300, 528, 16400), (520, 400, 8320), (1030, 1296, 9232)])
@pytest.mark.parametrize("transpose", [False, True])
def test_matmul_long_contraction(M, N, K, transpose):
    # beyond 64 blocks of the contraction the weight's scales are fetched again
    o, h = (K, N) if transpose else (N, K)
    a, s, w, ws, A2, B2 = product_case(M + K, M, o, h, transpose, 16, "e4m3")
    want = fp8.matmul(a, s, "e4m3", w[0], ws[0], transpose, f64(A2), f64(B2[0]))
    C = nf4.fp8_matmul(t8(a), torch.from_numpy(s).to(DEV), t8(w[0]), torch.from_numpy(ws[0]).to(DEV), transpose,
                       A2.to(DEV), B2[0].to(DEV))
    check_product(C, want, K, 16)


@pytest.mark.parametrize("M,N,K,transpose", [  # one of every kind of tile, and of split rows
    (8, 4096, 512, False), (16, 11008, 256, False), (32, 16384, 256, False), (64, 4096, 400, False),
    (128, 4096, 272, False), (256, 8192, 272, False), (600, 11008, 144, False), (2048, 4096, 272, False),
    (4096, 4096, 272, False), (4099, 4096, 1040, False), (16, 4096, 256, True), (128, 4096, 272, True),
    (64, 11008, 272, True), (300, 8192, 144, True), (1024, 4096, 272, True), (2048, 4096, 272, True),
    (4099, 4096, 1040, True), (64, 4096, 4096, False), (256, 4096, 4096, False), (32, 8192, 4096, False)])
def test_matmul_tiles(M, N, K, transpose):
    rng = np.random.default_rng(M + N)
    o, h = (K, N) if transpose else (N, K)
    X = torch.from_numpy(rows_of(rng, M, K)).to(DEV)
    a, s = nf4.fp8_quantize(X)
    w, ws = nf4.fp8_quantize(torch.from_numpy(0.02 * rng.standard_normal((o, h)).astype(np.float32)).to(DEV), 128)
    C = nf4.fp8_matmul(a, s, w, ws, transpose)
    # all of it against the dequantized values' product in fp64 on the device
    A, W = nf4.fp8_dequantize(a, s).double(), nf4.fp8_dequantize(w, ws, 128).double()
    W = W if transpose else W.t().contiguous()
    check_product(C, (f64(A @ W), f64(A.abs() @ W.abs()), f64(((A * A) @ (W * W)).sqrt())), K, 0)


EVERY_TILE = [  # M, N, K, transpose, experts: each kind of tile, dense and grouped
    (5000, 1552, 1040, False, 0), (4099, 1040, 1040, False, 0), (390, 8208, 1040, False, 0),
    (130, 8208, 1040, False, 0), (70, 8208, 1040, False, 0), (5, 272, 1040, False, 0), (260, 272, 1040, False, 0),
    (520, 272, 1040, False, 0), (1030, 272, 1040, False, 0), (1030, 528, 1040, False, 0),
    (5000, 1552, 1040, True, 0), (6200, 528, 1040, True, 0), (70, 8208, 1040, True, 0), (5, 272, 1040, True, 0),
    (1030, 272, 1040, True, 0), (1030, 528, 1040, True, 0),
    (4099, 1040, 9232, False, 0), (390, 8208, 9232, False, 0), (200, 8208, 9232, False, 0), (70, 8208, 9232, False, 0),
    (1030, 272, 9232, False, 0), (200, 2064, 9232, False, 0), (2050, 528, 9232, True, 0), (1030, 272, 9232, True, 0),
    (1030, 528, 9232, True, 0), (6200, 528, 9232, True, 0),
    (5000, 1552, 1040, False, 5), (520, 6160, 1040, False, 5), (100, 8208, 1040, False, 5), (200, 4112, 1040, False, 5),
    (3000, 272, 1040, False, 5), (24, 272, 1040, False, 5), (5, 272, 1040, False, 5), (520, 272, 1040, False, 5),
    (130, 1552, 1040, False, 5), (1030, 528, 1040, False, 5), (6200, 1040, 1040, True, 5), (5000, 528, 1040, True, 5),
    (5, 8208, 1040, True, 5), (5, 272, 1040, True, 5), (130, 1552, 1040, True, 5), (1500, 272, 1040, True, 5),
    (4099, 1552, 9232, True, 5), (1030, 6160, 9232, False, 5), (6200, 272, 9232, False, 5),
]


def check_tiles(M, N, K, transpose, experts, R, fmt, spoil=False):
    """A product against fp64 on the device; spoil: with a workspace full of NaN, and again without one."""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    E = experts or 1
    o, h = (K, N) if transpose else (N, K)
    a, s = nf4.fp8_quantize(torch.randn(M, K, generator=g, device=DEV) *
                            torch.exp(torch.randn(M, 1, generator=g, device=DEV)), 1, DTYPES[fmt])
    W = torch.empty(E, o, h, dtype=torch.float8_e4m3fn, device=DEV)
    ws = torch.empty(E, -(-o // 128), -(-h // 128), device=DEV)
    for e in range(E):
        nf4.fp8_quantize(0.02 * torch.randn(o, h, generator=g, device=DEV), 128, codes=W[e], scales=ws[e])
    A2 = torch.randn(M, R, generator=g, device=DEV).bfloat16()
    B2 = (0.05 * torch.randn(E, N, R, generator=g, device=DEV)).bfloat16()
    if experts:
        counts = [M // 2, 0, 1, M - M // 2 - 3, 0] if experts == 5 else [M // 2, 0, M - M // 2 - 2]  # two rows behind
        ends = np.concatenate([[0], np.cumsum(counts)])
        C = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
        offsets = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    else:
        ends = np.array([0, M])
        C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)

    def product(work=None):
        if experts:
            nf4.fp8_matmul_grouped(a, s, W, ws, offsets, transpose, A2, B2, out=C, ws=work)
            assert torch.all(C[M - 2:] == 3.0)
        else:
            nf4.fp8_matmul(a, s, W[0], ws[0], transpose, A2, B2[0], out=C, ws=work)
        return C.clone()

    if spoil:
        n = nf4.fp8_matmul_workspace_bytes(M, o, h, transpose, experts)
        assert n > 0
        work = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device=DEV)
        got = product(work)
        assert torch.all(work[n:] == 0xFF)
        assert torch.equal(product().view(torch.int16), got.view(torch.int16))  # one of its own
    else:
        product()
    A, D2 = nf4.fp8_dequantize(a, s).double(), A2.double()
    for e in range(E):
        r = slice(int(ends[e]), int(ends[e + 1]))
        if ends[e] == ends[e + 1]:
            continue
        D = nf4.fp8_dequantize(W[e], ws[e], 128).double()
        D = D if transpose else D.t().contiguous()
        X, T, U = A[r], D2[r], B2[e].double().t().contiguous()
        check_product(C[r], (f64(X @ D + T @ U), f64(X.abs() @ D.abs() + T.abs() @ U.abs()),
                             f64(((X * X) @ (D * D) + (T * T) @ (U * U)).sqrt())), K, R)


@pytest.mark.parametrize("R,fmt", [(64, "e5m2"), (16, "e4m3")])
@pytest.mark.parametrize("M,N,K,transpose,experts", EVERY_TILE)
def test_matmul_every_tile(M, N, K, transpose, experts, R, fmt):
    check_tiles(M, N, K, transpose, experts, R, fmt)


SPLIT_TILES = [  # M, N, K, transpose, experts: each kind of tile with its contraction split
    (4099, 528, 16400, False, 0), (3000, 144, 33040, False, 0), (130, 2064, 16400, False, 0), (260, 4112, 16400, False, 0),
    (300, 1552, 33040, False, 0), (200, 784, 16400, False, 0), (1, 16, 16400, False, 0), (5, 1552, 65552, False, 0),
    (130, 80, 16400, False, 0), (260, 80, 33040, False, 0), (4099, 16, 16400, False, 0), (520, 144, 33040, False, 0),
    (3000, 272, 33040, True, 0), (3000, 80, 8208, True, 0), (2050, 80, 8208, True, 0), (48, 4112, 16400, True, 0),
    (1, 16, 4112, True, 0), (5, 144, 33040, True, 0), (700, 16, 4112, True, 0), (2050, 16, 4112, True, 0),
    (2050, 1040, 16400, False, 3), (4099, 144, 16400, False, 3), (200, 1552, 16400, False, 3), (1290, 784, 16400, False, 3),
    (1030, 144, 16400, False, 3), (17, 16, 16400, False, 3), (260, 80, 33040, False, 3), (4099, 16, 16400, False, 3),
    (800, 144, 16400, False, 3), (5, 528, 16400, False, 3), (3000, 272, 33040, True, 3), (1030, 1040, 16400, True, 3),
    (1290, 80, 8208, True, 3), (17, 1040, 4112, True, 3), (700, 16, 4112, True, 3), (2050, 16, 4112, True, 3),
]


@pytest.mark.parametrize("R,fmt", [(64, "e5m2"), (16, "e4m3")])
@pytest.mark.parametrize("M,N,K,transpose,experts", SPLIT_TILES)
def test_matmul_split_contraction(M, N, K, transpose, experts, R, fmt):
    check_tiles(M, N, K, transpose, experts, R, fmt, spoil=True)


@pytest.mark.parametrize("transpose", [False, True])
def test_matmul_zero_blocks_and_nan(transpose):
    # a zero row and zero weight blocks give exact zeros; a NaN stays in its row
    a, s, w, ws, _, _ = product_case(3, 40, 272, 272, transpose, 0, "e4m3")
    a[7] = 0
    w0 = np.zeros_like(w[0])
    z = nf4.fp8_matmul(t8(a), torch.from_numpy(s).to(DEV), t8(w0), torch.from_numpy(ws[0]).to(DEV), transpose)
    assert torch.all(z == 0)
    a[9, 3] = 0x7F
    C = nf4.fp8_matmul(t8(a), torch.from_numpy(s).to(DEV), t8(w[0]), torch.from_numpy(ws[0]).to(DEV), transpose)
    bad = torch.isnan(C).any(1).cpu()
    assert bad[9] and int(bad.sum()) == 1 and torch.isnan(C[9]).all() and torch.all(C[7] == 0)


GROUPED = [  # counts, rows before the first and behind the last
    ([5], 0, 0), ([0, 7, 0, 1], 0, 3), ([130, 0, 1, 64, 17], 2, 5), ([1] * 70, 0, 0), ([0] * 66 + [3], 1, 1),
    ([300, 5, 129, 0, 0, 40], 0, 9), ([0, 0], 0, 4), ([700, 0, 1], 5, 0), ([0] * 130 + [5, 0, 40], 0, 2),
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("o,h,R,fmt", [(144, 272, 0, "e4m3"), (272, 144, 32, "e5m2"), (400, 656, 16, "e4m3")])
@pytest.mark.parametrize("counts,before,after", GROUPED)
def test_matmul_grouped(counts, before, after, o, h, R, fmt, transpose):
    E, M = len(counts), before + sum(counts) + after
    a, s, w, ws, A2, B2 = product_case(E + M, M, o, h, transpose, R, fmt, E)
    N = h if transpose else o
    ends = before + np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    args = (t8(a, fmt), torch.from_numpy(s).to(DEV), t8(np.stack(w)), torch.from_numpy(np.stack(ws)).to(DEV), offsets,
            transpose, A2.to(DEV) if R else None, torch.stack(B2).to(DEV) if R else None)
    nf4.fp8_matmul_grouped(*args, out=out)
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        if counts[e]:
            want = fp8.matmul(a[r], s[r], fmt, w[e], ws[e], transpose, f64(A2[r]) if R else None,
                              f64(B2[e]) if R else None)
            check_product(out[r], want, h if not transpose else o, R)
    rest = torch.cat([out[:ends[0]], out[ends[-1]:]])
    assert torch.all(rest == 3.0)


@pytest.mark.parametrize("counts,N,K", [([40] * 8, 1040, 1040), ([100, 0, 300, 7], 2064, 528), ([900, 0, 33, 1200], 2048, 272),
                                        ([2000, 0, 1500, 33], 4096, 144), ([5000, 1, 0, 3000], 4096, 144)])
@pytest.mark.parametrize("transpose", [False, True])
def test_matmul_grouped_tiles(counts, N, K, transpose):
    rng = np.random.default_rng(sum(counts) + N)
    E, M = len(counts), sum(counts) + 5
    o, h = (K, N) if transpose else (N, K)
    a, s = nf4.fp8_quantize(torch.from_numpy(rows_of(rng, M, K)).to(DEV))
    W = torch.empty(E, o, h, dtype=torch.float8_e4m3fn, device=DEV)
    ws = torch.empty(E, -(-o // 128), -(-h // 128), device=DEV)
    for e in range(E):
        x = torch.from_numpy(0.02 * rng.standard_normal((o, h)).astype(np.float32)).to(DEV)
        nf4.fp8_quantize(x, 128, codes=W[e], scales=ws[e])
    ends = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    nf4.fp8_matmul_grouped(a, s, W, ws, offsets, transpose, out=out)
    A = nf4.fp8_dequantize(a, s).double()
    for e in range(E):
        if counts[e]:
            D, X = nf4.fp8_dequantize(W[e], ws[e], 128).double(), A[ends[e]:ends[e + 1]]
            D = D if transpose else D.t().contiguous()
            check_product(out[ends[e]:ends[e + 1]],
                          (f64(X @ D), f64(X.abs() @ D.abs()), f64(((X * X) @ (D * D)).sqrt())), K, 0)
    assert torch.all(out[ends[-1]:] == 3.0)


def test_matmul_grouped_offsets_outside():
    # offsets below 0 and above M are taken as 0 and M
    a, s, w, ws, _, _ = product_case(9, 20, 144, 272, False, 0, "e4m3", 3)
    args = (t8(a), torch.from_numpy(s).to(DEV), t8(np.stack(w)), torch.from_numpy(np.stack(ws)).to(DEV))
    wide = torch.tensor([-5, 8, 8, 1000], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 8, 8, 20], dtype=torch.int32, device=DEV)
    assert torch.equal(nf4.fp8_matmul_grouped(*args, wide), nf4.fp8_matmul_grouped(*args, good))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", [[5, 0, 12], [300, 0, 129], [2000, 0, 1500]])
def test_matmul_grouped_reads_its_rows_alone(counts, transpose):
    # NaN in the rows before and behind, and in the weights of experts without rows
    rng = np.random.default_rng(sum(counts))
    o, h = (528, 1040)
    K, N = (o, h) if transpose else (h, o)
    M = 3 + sum(counts) + 130
    a, s = nf4.fp8_quantize(torch.from_numpy(rows_of(rng, M, K)).to(DEV))
    W = torch.empty(3, o, h, dtype=torch.float8_e4m3fn, device=DEV)
    ws = torch.empty(3, -(-o // 128), -(-h // 128), device=DEV)
    for e in range(3):
        nf4.fp8_quantize(torch.from_numpy(0.02 * rng.standard_normal((o, h)).astype(np.float32)).to(DEV), 128,
                         codes=W[e], scales=ws[e])
    A2 = torch.from_numpy(rng.standard_normal((M, 48))).to(DEV).bfloat16()
    B2 = torch.from_numpy(0.05 * rng.standard_normal((3, N, 48))).to(DEV).bfloat16()
    offsets = torch.from_numpy((3 + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)).to(DEV)
    want = nf4.fp8_matmul_grouped(a, s, W, ws, offsets, transpose, A2, B2, out=torch.full((M, N), 3.0, device=DEV).bfloat16())
    for r in (slice(0, 3), slice(3 + sum(counts), M)):
        a.view(torch.uint8)[r] = 0x7F
        s[r] = float("nan")
        A2[r] = float("nan")
    W.view(torch.uint8)[1] = 0x7F
    ws[1] = float("inf")
    B2[1] = float("nan")
    got = nf4.fp8_matmul_grouped(a, s, W, ws, offsets, transpose, A2, B2, out=torch.full((M, N), 3.0, device=DEV).bfloat16())
    assert torch.isfinite(got).all() and torch.equal(got, want)


def test_matmul_grouped_offsets_that_do_not_ascend():
    # which rows are written is unspecified, but none outside C
    a, s, w, ws, _, _ = product_case(10, 40, 144, 272, False, 0, "e4m3", 4)
    args = (t8(a), torch.from_numpy(s).to(DEV), t8(np.stack(w)), torch.from_numpy(np.stack(ws)).to(DEV))
    for ends in ([0, 40, 5, 38, 40], [40, 30, 20, 10, 0], [0, -7, 90, -2147483648, 2147483647], [7, 7, 7, 7, 7]):
        room = torch.full((120, 144), 3.0, dtype=torch.bfloat16, device=DEV)
        nf4.fp8_matmul_grouped(*args, torch.tensor(ends, dtype=torch.int32, device=DEV), out=room[40:80])
        assert torch.all(room[:40] == 3.0) and torch.all(room[80:] == 3.0)


def test_matmul_grouped_replayed_with_other_offsets():
    a, s, w, ws, A2, B2 = product_case(11, 200, 272, 400, False, 16, "e4m3", 5)
    args = [t8(a), torch.from_numpy(s).to(DEV), t8(np.stack(w)), torch.from_numpy(np.stack(ws)).to(DEV)]
    more = (False, A2.to(DEV), torch.stack(B2).to(DEV))
    splits = [[0, 0, 200, 200, 200, 200], [0, 1, 2, 3, 4, 5], [10, 60, 61, 61, 190, 200], [200] * 6]
    offsets = torch.tensor(splits[0], dtype=torch.int32, device=DEV)
    out = torch.zeros(200, 272, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nf4.fp8_matmul_grouped(*args, offsets, *more, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.fp8_matmul_grouped(*args, offsets, *more, out=out)
    for ends in splits + splits[::-1]:
        offsets.copy_(torch.tensor(ends, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        want = nf4.fp8_matmul_grouped(*args, torch.tensor(ends, dtype=torch.int32, device=DEV), *more,
                                      out=torch.full_like(out, 3.0))
        assert torch.equal(out, want), ends


def tall(M, H):
    """bf16 [M][H] whose rows all differ, made without a host copy."""
    g = torch.Generator(device=DEV).manual_seed(H)
    base = torch.randn(512, H, generator=g, device=DEV).bfloat16()
    x = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
    for r0 in range(0, M, 512):
        n = min(512, M - r0)
        x[r0:r0 + n] = base[:n] * (1 + r0 / M)
    return x


def test_rows_past_32_bits():
    # more than 2^32 values: the last rows are what they are by themselves
    M, H = 131300, 32768
    X, w = tall(M, H), bf16_np(1 + 0.1 * np.random.default_rng(1).standard_normal(H)).to(DEV)
    ends = [slice(0, 65), slice(65500, 65600), slice(131050, 131090), slice(M - 70, M)]
    codes, scales = nf4.fp8_quantize(X)
    for r in ends:
        c, s = nf4.fp8_quantize(X[r])
        assert np.array_equal(bits(codes[r]), bits(c)) and torch.equal(scales[r], s)
    back = nf4.fp8_dequantize(codes, scales, bf16=True)
    for r in ends:
        assert torch.equal(back[r], nf4.fp8_dequantize(codes[r], scales[r], bf16=True))
    Y, h, nc, ns, rstd = nf4.rmsnorm_fwd(X, w, 1e-6, back, want_fp8=True, want_rstd=True)
    for r in ends:
        one = nf4.rmsnorm_fwd(X[r], w, 1e-6, back[r], want_fp8=True, want_rstd=True)
        for t, u in zip((Y, h, nc, ns, rstd), one):
            assert torch.equal(t[r].view(torch.uint8), u.view(torch.uint8))
    del codes, scales, nc, ns, back
    dX, dw = nf4.rmsnorm_bwd(Y, h, w, rstd, X)
    for r in ends:
        assert torch.equal(dX[r].view(torch.int16),
                           nf4.rmsnorm_bwd(Y[r].contiguous(), h[r], w, rstd[r], X[r])[0].view(torch.int16))
    dw64, size = torch.zeros(H, dtype=torch.float64, device=DEV), torch.zeros(H, dtype=torch.float64, device=DEV)
    for r0 in range(0, M, 4096):
        t = Y[r0:r0 + 4096].double() * h[r0:r0 + 4096].double() * rstd[r0:r0 + 4096, None].double()
        dw64 += t.sum(0)
        size += t.abs().sum(0)
    # a workgroup's rows in turn (at most ceil(M / 256)), then the parts
    check_within("dw", dw, f64(dw64), f64(size) * (-(-M // 256) + 64) * EPS32)
    del X, Y, h, dX
    x = tall(128 * 1024 + 200, 32768).float()  # and by blocks of 128 rows
    codes, scales = nf4.fp8_quantize(x, 128)
    r = slice(128 * 1024, None)
    c, s = nf4.fp8_quantize(x[r], 128)
    assert np.array_equal(bits(codes[r]), bits(c)) and torch.equal(scales[1024:], s)


@pytest.mark.parametrize("transpose", [False, True])
def test_products_past_32_bits(transpose):
    # A and C of more than 2^32 bytes
    M, N, K = 263000, 16400, 16512
    o, h = (K, N) if transpose else (N, K)
    a, s = nf4.fp8_quantize(tall(M, K))
    w, ws = nf4.fp8_quantize(tall(o, h), 128)
    C = nf4.fp8_matmul(a, s, w, ws, transpose)
    W = nf4.fp8_dequantize(w, ws, 128)
    rows = torch.tensor([0, 131071, 131072, 260096, 262143, 262144, M - 1], device=DEV)
    cols = torch.cat([torch.arange(0, 300, device=DEV), torch.arange(N - 300, N, device=DEV)])
    B = (W[:, cols] if transpose else W[cols].t()).double().contiguous()

    def check(C, rows, B):
        A = nf4.fp8_dequantize(a[rows].contiguous(), s[rows].contiguous()).double()
        check_product(C[rows][:, cols].contiguous(), (f64(A @ B), f64(A.abs() @ B.abs()),
                                                      f64(((A * A) @ (B * B)).sqrt())), K, 0)

    check(C, rows, B)
    # and a stack of weights of more than 2^32 bytes, the last expert with rows
    E = 17
    W17 = torch.empty(E, o, h, dtype=torch.float8_e4m3fn, device=DEV)
    s17 = torch.zeros(E, -(-o // 128), -(-h // 128), device=DEV)
    W17.view(torch.uint8)[:E - 1] = 0x7F  # NaN
    W17.view(torch.uint8)[E - 1] = w.view(torch.uint8)
    s17[E - 1] = ws
    offsets = torch.full((E + 1,), M - 300, dtype=torch.int32, device=DEV)
    offsets[E] = M
    C.fill_(3.0)
    nf4.fp8_matmul_grouped(a, s, W17, s17, offsets, transpose, out=C)
    assert torch.all(C[M - 1000:M - 300] == 3.0)
    check(C, torch.tensor([M - 300, M - 44, M - 1], device=DEV), B)


def test_empty():
    a = torch.empty(0, 272, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(0, 3, device=DEV)
    W, ws = nf4.fp8_quantize(torch.randn(144, 272, device=DEV), 128)
    assert nf4.fp8_matmul(a, s, W, ws).shape == (0, 144)
    X = torch.empty(0, 272, dtype=torch.bfloat16, device=DEV)
    c, sc = nf4.fp8_quantize(X)
    assert c.shape == (0, 272) and sc.shape == (0, 3)
    w = torch.ones(272, dtype=torch.bfloat16, device=DEV)
    assert nf4.rmsnorm_fwd(X, w)[0].shape == (0, 272)
    dX, dw = nf4.rmsnorm_bwd(X, X, w, torch.empty(0, device=DEV))
    assert dX.shape == (0, 272) and torch.all(dw == 0)


# ---------------------------------------------------------------------------------------------------------
# together, captured, refused
# ---------------------------------------------------------------------------------------------------------

def layer(x, res, w, W, ws, L1, L2, s, dY, dH):
    """Norm, frozen 8-bit linear with an adapter, and both gradients, as a training step makes them."""
    y, h, codes, scales, rstd = nf4.rmsnorm_fwd(x, w, 1e-6, res, want_y=True, want_fp8=True, want_rstd=True)
    T = y @ L1
    Y = nf4.fp8_matmul(codes, scales, W, ws, A2=(s * T.float()).to(torch.bfloat16), B2=L2.t().contiguous())
    G = (s * (dY.float() @ L2.float().t())).to(torch.bfloat16)
    dq, ds = nf4.fp8_quantize(dY, 1, torch.float8_e5m2)
    dy = nf4.fp8_matmul(dq, ds, W, ws, True, G, L1)
    dX, dw = nf4.rmsnorm_bwd(dy, h, w, rstd, dH)
    return Y, dX, dw


def layer_case(M=200, o=400, h=272, r=16):
    rng = np.random.default_rng(5)
    t = lambda a: bf16_np(a).to(DEV)
    W, ws = nf4.fp8_quantize(torch.from_numpy((0.05 * rng.standard_normal((o, h))).astype(np.float32)).to(DEV), 128)
    return (t(rows_of(rng, M, h)), t(rows_of(rng, M, h)), t(1 + 0.1 * rng.standard_normal(h)), W, ws,
            t(0.05 * rng.standard_normal((h, r))), t(0.05 * rng.standard_normal((r, o))), 2.0,
            t(1e-3 * rng.standard_normal((M, o))), t(1e-3 * rng.standard_normal((M, h))))


def test_layer_forward_and_gradient():
    x, res, w, W, ws, L1, L2, s, dY, dH = layer_case()
    Y, dX, dw = layer(x, res, w, W, ws, L1, L2, s, dY, dH)
    h = f64((x.float() + res.float()).to(torch.bfloat16))
    y, r = fp8.rmsnorm(h, f64(w), 1e-6)
    Wd = f64(nf4.fp8_dequantize(W, ws, 128))
    B = f64(L1) @ f64(L2) * s
    Yw = y @ (Wd.T + B)
    # 8-bit activations: each rounded by at most 2^-4, independent signs; relative rms of uniform rounding 2^-4 / sqrt(3)
    rms = lambda g, v: np.sqrt(np.mean((f64(g) - v) ** 2) / np.mean(v ** 2))
    assert rms(Y, Yw) < 2.0 ** -4
    dyw = f64(dY) @ (Wd + B.T)
    dxw, dww = fp8.rmsnorm_grad(dyw, h, f64(w), r, f64(dH))
    assert rms(dX, dxw) < 2.0 ** -3 and rms(dw, dww) < 2.0 ** -3


def test_layer_captured_and_replayed():
    args = layer_case()
    eager = layer(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(*args)
    for k in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b), k
        again = layer(*args)  # eager work between the replays
        assert all(torch.equal(a, b) for a, b in zip(again, eager))


def test_another_stream():
    args = layer_case(M=130)
    want = layer(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer(*args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("transpose", [False, True])
def test_split_captured_and_replayed(transpose):
    # its workspace comes from the graph's pool, or is the caller's, shared by two graphs that run in turn
    M, N, K = (260, 80, 33040) if not transpose else (5, 144, 33040)
    o, h = (K, N) if transpose else (N, K)
    a, s, w, ws, A2, B2 = product_case(21, M, o, h, transpose, 16, "e4m3")
    args = (t8(a), torch.from_numpy(s).to(DEV), t8(w[0]), torch.from_numpy(ws[0]).to(DEV), transpose, A2.to(DEV),
            B2[0].to(DEV))
    eager = nf4.fp8_matmul(*args)
    work = torch.empty(nf4.fp8_matmul_workspace_bytes(M, o, h, transpose), dtype=torch.uint8, device=DEV)
    assert work.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nf4.fp8_matmul(*args)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for given in (None, work, work):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = nf4.fp8_matmul(*args, ws=given)
        graphs.append((g, out))
    for k in range(4):
        for g, out in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            assert torch.equal(out, eager), k
        assert torch.equal(nf4.fp8_matmul(*args), eager)


def test_two_streams_at_once():
    cases = [layer_case(M=130), layer_case(M=700)]
    want = [layer(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(8):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(layer(*c))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2])), k


def test_binding_refuses():
    x = torch.randn(8, 272, device=DEV)
    a, s = nf4.fp8_quantize(x)
    W, ws = nf4.fp8_quantize(torch.randn(144, 272, device=DEV), 128)
    b = x.to(torch.bfloat16)
    w = torch.ones(272, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    W2, ws2 = torch.stack([W.view(torch.uint8)] * 2).view(torch.float8_e4m3fn), torch.stack([ws] * 2)
    r = torch.ones(8, device=DEV)
    A2, B2 = torch.zeros(8, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(144, 16, dtype=torch.bfloat16, device=DEV)
    bad = [
        lambda: nf4.fp8_quantize(x.half()), lambda: nf4.fp8_quantize(x.cpu()), lambda: nf4.fp8_quantize(x.t()),
        lambda: nf4.fp8_quantize(x, 1, torch.float16), lambda: nf4.fp8_quantize(x, 1, scales=s[:4]),
        lambda: nf4.fp8_quantize(x, 1, codes=a.view(torch.uint8)),
        lambda: nf4.fp8_dequantize(x, s), lambda: nf4.fp8_dequantize(a, ws), lambda: nf4.fp8_dequantize(a, s, out=b), lambda: nf4.fp8_matmul(a, s, W, ws, ws=x),
        lambda: nf4.fp8_matmul(a, ws, W, ws), lambda: nf4.fp8_matmul(a, s, W, ws, True),
        lambda: nf4.fp8_matmul(a, s, W.view(torch.float8_e5m2), ws), lambda: nf4.fp8_matmul(x, s, W, ws),
        lambda: nf4.fp8_matmul(a, s, W, ws, A2=A2), lambda: nf4.fp8_matmul(a, s, W, ws, A2=A2, B2=B2.t()),
        lambda: nf4.fp8_matmul(a, s, W, ws, out=b), lambda: nf4.fp8_matmul(a[:, ::2], s, W, ws),
        lambda: nf4.fp8_matmul_grouped(a, s, W, ws, off), lambda: nf4.fp8_matmul_grouped(a, s, W2, ws2, off.long()),
        lambda: nf4.fp8_matmul_grouped(a, s, W2, ws2, off[:2]),
        lambda: nf4.fp8_matmul_grouped(a, s, W2, ws2, off, A2=A2, B2=B2),
        lambda: nf4.rmsnorm_fwd(x, w), lambda: nf4.rmsnorm_fwd(b, w.float()), lambda: nf4.rmsnorm_fwd(b, w, residual=x),
        lambda: nf4.rmsnorm_fwd(b, w, outs=(None,) * 5), lambda: nf4.rmsnorm_bwd(b, b, w, r[:4]),
        lambda: nf4.rmsnorm_bwd(b, b, w, r, dH=x), lambda: nf4.rmsnorm_bwd(b, b, w, r, ws=x),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    status = [
        (lambda: nf4.fp8_quantize(x, 2), nf4.NF4_ERR_ARG), (lambda: nf4.fp8_quantize(x[:, :24].contiguous()), nf4.NF4_ERR_SHAPE),
        (lambda: nf4.fp8_matmul(a, s, W, ws, A2=A2[:, :8].contiguous(), B2=B2[:, :8].contiguous()), nf4.NF4_ERR_SHAPE),
        (lambda: nf4.rmsnorm_fwd(b, w, -1.0), nf4.NF4_ERR_ARG), (lambda: nf4.rmsnorm_fwd(b, w, want_y=False), nf4.NF4_ERR_NULL),
        (lambda: nf4.rmsnorm_fwd(b[:, :24].contiguous(), w[:24].contiguous()), nf4.NF4_ERR_SHAPE),
        (lambda: nf4.rmsnorm_fwd(b, w, outs=(b, None, None, None, None)), nf4.NF4_ERR_ALIAS),
        (lambda: nf4.rmsnorm_bwd(b, b, w, r, ws=torch.empty(16, dtype=torch.uint8, device=DEV)), nf4.NF4_ERR_WORKSPACE),
    ]
    for i, (f, want) in enumerate(status):
        with pytest.raises(nf4.NF4Error) as err:
            f()
        assert err.value.status == want, i
