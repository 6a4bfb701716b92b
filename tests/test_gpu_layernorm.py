"""The layer norm and its gradient against the fp64 oracle (needs an MI355X).

Outputs are held to the roundings they go through: half a step of the output's type relative to the value; the
forward's sums are fp64, the gradient's fp32 (EPS32 for each addition in turn, in proportion to the sum of the terms'
magnitudes)."""
import numpy as np
import pytest
import torch

from oracle import around, fp8

pytestmark = pytest.mark.gpu

try:
    import quantized_lora_fine_amd as nf4
except ImportError as exc:
    if torch.cuda.is_available():
        raise
    pytest.skip(f"libnf4lora.so not loaded: {exc}", allow_module_level=True)

from tests.test_gpu_fp8 import BF16, DEV, E4M3, EPS32, bf16_np, bits, check_within, f64, rows_of  # noqa: E402

FP32 = 2.0 ** -24     # half a step, relative
F64 = 2.0 ** -40      # what the fp64 arithmetic and its one Newton step leave (2^-44), with room
WIDTHS = [16, 128, 144, 512, 528, 1040, 2048, 2064, 4096, 8192, 8208, 16384, 16400, 32768]


def spread(v, M, H):
    return fp8._spread(v, 1, M, H).astype(np.float64)


def case(seed, M, H, residual, bias):
    rng = np.random.default_rng(seed)
    X = bf16_np(rows_of(rng, M, H) + 3 * rng.standard_normal((M, 1)))
    w = bf16_np(1 + 0.1 * rng.standard_normal(H))
    R = bf16_np(rows_of(rng, M, H)) if residual else None
    b = bf16_np(0.1 * rng.standard_normal(H)) if bias else None
    return X, w, R, b


def on(t):
    return None if t is None else t.to(DEV)


def check_forward(X, w, R, b, eps, exact=None):
    M, H = X.shape
    Y, h, codes, scales, mean, rstd = nf4.layernorm_fwd(on(X), on(w), on(b), eps, on(R), want_fp8=True,
                                                        want_stats=True)
    hw = X if R is None else (X.float() + R.float()).to(torch.bfloat16)
    assert (h is None) == (R is None)
    if R is not None:
        assert torch.equal(h.cpu().view(torch.int16), hw.view(torch.int16))
    y, m, r = around.layernorm(f64(hw), f64(w), None if b is None else f64(b), eps)
    size = np.abs(f64(hw) - m[:, None]) * r[:, None] * np.abs(f64(w)) + (0 if b is None else np.abs(f64(b)))
    # the difference h - mean carries the mean's own error, 2^-53 of the row's magnitudes for each of 64 additions
    far = np.mean(np.abs(f64(hw)), 1) * 2.0 ** -46
    size = size * F64 + (far * r)[:, None] * np.abs(f64(w))
    check_within("mean", mean, m, np.abs(m) * FP32 + far)
    check_within("rstd", rstd, r, np.abs(r) * (FP32 * (1 + 2.0 ** -8) + far * r))
    check_within("y", Y, y, np.abs(y) * BF16 * (1 + 2.0 ** -8) + size)
    s64 = fp8.block_scales(y.astype(np.float32), 1, "e4m3")[0].astype(np.float64)
    slack = spread(size.reshape(M, H).max(1, keepdims=True).repeat(s64.shape[1], 1), M, H)
    check_within("scales", scales, s64, s64 * 2.0 ** -22 + slack[:, :s64.shape[1]])
    d = f64(nf4.fp8_dequantize(codes, scales))
    check_within("codes", d, y, np.maximum(np.abs(y) * E4M3, spread(s64, M, H) * 2.0 ** -10) * (1 + 2.0 ** -8) + 2 * slack)
    return Y, codes, scales


@pytest.mark.parametrize("residual,bias", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("M,H", [(1, h) for h in WIDTHS] + [(5, h) for h in WIDTHS] + [(300, 272), (67, 4096)])
def test_layernorm(M, H, residual, bias):
    X, w, R, b = case(M + H, M, H, residual, bias)
    Y, codes, scales = check_forward(X, w, R, b, 1e-5)
    # each output alone is what it is beside the others, and a given output is the one that is returned
    Y1, _, none, _, _, _ = nf4.layernorm_fwd(on(X), on(w), on(b), 1e-5, on(R))
    assert none is None and torch.equal(Y1.view(torch.int16), Y.view(torch.int16))
    outs = (None, None if R is None else torch.empty_like(Y), torch.empty_like(codes), torch.empty_like(scales), None,
            None)
    got = nf4.layernorm_fwd(on(X), on(w), on(b), 1e-5, on(R), want_y=False, want_fp8=True, outs=outs)
    assert got[2] is outs[2] and np.array_equal(bits(outs[2]), bits(codes)) and torch.equal(outs[3], scales)


def test_layernorm_rounds_once():
    # as the root-mean-square norm's test: y in 64 bits, its fp32 value and that value's product with the multiplier
    # are 2^-23 off together, so 4 of a million codes lie on the other side of a tie at most: 1.4 of these
    X, w, _, b = case(5, 84, 4096, False, True)
    _, _, codes, _, mean, rstd = nf4.layernorm_fwd(on(X), on(w), on(b), 1e-5, want_y=False, want_fp8=True,
                                                   want_stats=True)
    y, m, r = around.layernorm(f64(X), f64(w), f64(b), 1e-5)
    _, mul = fp8.block_scales(y.astype(np.float32), 1, "e4m3")
    want = fp8.encode((y * spread(mul, 84, 4096)).astype(np.float32), "e4m3")
    assert np.sum(bits(codes) != want) <= 6  # of 1.4 expected at most, more than 6 in one of 10^3 draws
    check_within("rstd", rstd, r, np.abs(r) * FP32 * (1 + 2.0 ** -16))
    check_within("mean", mean, m, np.abs(m) * FP32 * (1 + 2.0 ** -16) + 2.0 ** -46 * np.mean(np.abs(f64(X)), 1))


def test_layernorm_any_magnitude():
    # squares past and below fp32's range, rows far from zero; an infinity or a NaN stays in its row
    rng = np.random.default_rng(6)
    M, H = 13, 1040
    x = rng.standard_normal((M, H)) * np.array([1e30, 1e25, 1e19, 1, 1e-10, 1e-18, 1e-22, 1e-30, 1, 1, 1, 1, 1])[:, None]
    x[8] = 1000 + 8 * rng.integers(0, 4, H)  # a mean hundreds of times the deviation
    x[9] = 1 + rng.integers(0, 2, H) * 2.0 ** -7
    X, w, b = bf16_np(x), bf16_np(1 + 0.1 * rng.standard_normal(H)), bf16_np(rng.standard_normal(H))
    check_forward(X[:10], w, None, b, 0.0)
    check_forward(X[:10], w, None, None, 1e-5)
    X[10, 7], X[11, 9], X[12, 11] = float("inf"), float("nan"), float("-inf")
    Y, _, codes, scales, _, rstd = nf4.layernorm_fwd(on(X), on(w), on(b), 1e-5, want_fp8=True, want_stats=True)
    assert torch.isnan(Y[10:]).all() and torch.isnan(rstd[10:]).all() and torch.isfinite(Y[:10]).all()
    assert torch.isnan(codes[10:].float()).all() and torch.isfinite(scales).all()


@pytest.mark.parametrize("H", [16, 272, 2064, 4096, 16400])
def test_layernorm_rows_of_equal_values(H):
    X = torch.tensor([0.0, 3.0, 1e30, -1.0 / 3, 1e-38], device=DEV).to(torch.bfloat16)[:, None].repeat(1, H)
    w = torch.full((H,), 1.5, dtype=torch.bfloat16, device=DEV)
    b = torch.linspace(-2, 2, H, device=DEV).to(torch.bfloat16)
    Y, _, codes, scales, mean, rstd = nf4.layernorm_fwd(X, w, b, 1e-5, want_fp8=True, want_stats=True)
    assert torch.equal(Y.view(torch.int16), b.expand(5, H).contiguous().view(torch.int16))
    assert torch.equal(mean, X[:, 0].float())
    Y, _, codes, scales, _, _ = nf4.layernorm_fwd(X, w, None, 1e-5, want_fp8=True)
    assert torch.all(Y == 0) and torch.all(codes.float() == 0)
    Y = nf4.layernorm_fwd(X, w, b, 0.0)[0]
    assert torch.all(torch.isnan(Y))


def grad_case(M, H, with_dh):
    rng = np.random.default_rng(M * 3 + H)
    h, w = bf16_np(rows_of(rng, M, H) + 2 * rng.standard_normal((M, 1))), bf16_np(1 + 0.1 * rng.standard_normal(H))
    dy = bf16_np(1e-3 * rows_of(rng, M, H))
    dh = bf16_np(1e-3 * rows_of(rng, M, H)) if with_dh else None
    _, m, r = around.layernorm(f64(h), f64(w), None, 1e-5)
    return dy, h, w, torch.from_numpy(m.astype(np.float32)), torch.from_numpy(r.astype(np.float32)), dh


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("M,H", [(1, h) for h in WIDTHS] + [(37, h) for h in (16, 144, 528, 2064, 5120, 8208, 16400)] +
                         [(2500, 144), (1100, 1040), (700, 4096), (1999, 5120)])
def test_layernorm_grad(M, H, with_dh):
    dy, h, w, mean, rstd, dh = grad_case(M, H, with_dh)
    dX, dw, db = nf4.layernorm_bwd(on(dy), on(h), on(w), on(mean), on(rstd), on(dh))
    m, r = f64(mean), f64(rstd)
    dx64, dw64, db64 = around.layernorm_grad(f64(dy), f64(h), f64(w), m, r, f64(dh) if with_dh else None)
    u, xhat = np.abs(f64(dy) * f64(w)), np.abs(f64(h) - m[:, None]) * r[:, None]
    size = r[:, None] * (u + np.mean(u, 1, keepdims=True) + xhat * np.mean(u * xhat, 1, keepdims=True))
    # the two sums: 32 terms of a thread, 6 steps of its wave, 16 waves; then a handful of roundings
    check_within("dx", dX, dx64, np.abs(dx64) * BF16 * (1 + 2.0 ** -8) + size * 64 * EPS32)
    # dw and db: the rows of one workgroup in turn (at most ceil(M / 256)), 16 teams, then the parts
    deep = -(-M // 256) + 16 + 64
    check_within("dw", dw, dw64, np.sum(np.abs(f64(dy)) * xhat, 0) * deep * EPS32)
    check_within("db", db, db64, np.sum(np.abs(f64(dy)), 0) * deep * EPS32)
    dX2, dw2, none = nf4.layernorm_bwd(on(dy), on(h), on(w), on(mean), on(rstd), on(dh), want_db=False)
    assert none is None and torch.equal(dX2.view(torch.int16), dX.view(torch.int16)) and torch.equal(dw2, dw)


def test_layernorm_grad_against_differences():
    # f(x, w, b) = sum of y * dy in 64 bits on the CPU; the kernel's gradient of it along random directions
    rng = np.random.default_rng(9)
    dy, h, w, mean, rstd, _ = grad_case(19, 272, False)
    dX, dw, db = (f64(t) for t in nf4.layernorm_bwd(on(dy), on(h), on(w), on(mean), on(rstd)))
    g, x, w, b = f64(dy), f64(h), f64(w), np.zeros(272)

    def f(x, w, b):
        return np.sum(around.layernorm(x, w, b, 1e-5)[0] * g)

    for _ in range(3):
        ex, ew, eb = rng.standard_normal(x.shape), rng.standard_normal(272), rng.standard_normal(272)
        for e, got, terms in ((1, np.sum(dX * ex), np.abs(dX * ex)), (2, np.sum(dw * ew), np.abs(dw * ew)),
                              (3, np.sum(db * eb), np.abs(db * eb))):
            t = 1e-5
            ends = [f(x + (e == 1) * s * t * ex, w + (e == 2) * s * t * ew, b + (e == 3) * s * t * eb) for s in (1, -1)]
            want = (ends[0] - ends[1]) / (2 * t)
            # dX's bf16 rounding and mean's and rstd's fp32 one; the difference's own error is t^2 and 2^-53 / t
            assert abs(got - want) <= np.sum(terms) * BF16 + 1e-6 * np.sum(terms), (e, got, want)


def test_layernorm_empty():
    bf = dict(dtype=torch.bfloat16, device=DEV)
    X, w = torch.empty(0, 256, **bf), torch.ones(256, **bf)
    f = torch.empty(0, device=DEV)
    Y, _, codes, scales, mean, _ = nf4.layernorm_fwd(X, w, w, want_fp8=True, want_stats=True)
    assert Y.shape == (0, 256) and codes.shape == (0, 256) and scales.shape == (0, 2) and mean.shape == (0,)
    out = (torch.empty(0, 256, **bf), torch.ones(256, device=DEV), torch.ones(256, device=DEV))
    nf4.layernorm_bwd(X, X, w, f, f, outs=out)
    assert torch.all(out[1] == 0) and torch.all(out[2] == 0)


def test_layernorm_captured_and_replayed():
    dy, h, w, mean, rstd, dh = (on(t) for t in grad_case(300, 1040, True))
    b = torch.zeros_like(w)

    def step():
        Y, _, codes, scales, m, r = nf4.layernorm_fwd(h, w, b, residual=dh, want_fp8=True, want_stats=True)
        return (Y, codes, scales, *nf4.layernorm_bwd(dy, h, w, m, r, dh))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        h.copy_(h.roll(k + 1, 0))
        dy.mul_(1.5)
        for t in outs:
            t.view(torch.uint8).fill_(17)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, c in zip(outs, want):
            assert np.array_equal(bits(a), bits(c)), k


def test_layernorm_refuses():
    X, w = torch.zeros(8, 272, dtype=torch.bfloat16, device=DEV), torch.zeros(272, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(8, device=DEV)
    for bad in (lambda: nf4.layernorm_fwd(X.float(), w), lambda: nf4.layernorm_fwd(X, w[:256]),
                lambda: nf4.layernorm_fwd(X, w, b=w[:16]), lambda: nf4.layernorm_fwd(X, w, residual=X[:4]),
                lambda: nf4.layernorm_fwd(X[:, ::2], w[::2]), lambda: nf4.layernorm_bwd(X, X, w, st, st[:4]),
                lambda: nf4.layernorm_bwd(X, X, w, st.double(), st), lambda: nf4.layernorm_bwd(X, X[:4], w, st, st),
                lambda: nf4.layernorm_bwd(X, X, w, st, st, outs=(X.clone(), st, None)),
                lambda: nf4.layernorm_fwd(X, w, outs=(None,) * 6), lambda: nf4.layernorm_fwd(X, w, outs=(X.clone(),))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nf4.NF4Error):
        nf4.layernorm_fwd(X, w, eps=-1.0)
    with pytest.raises(nf4.NF4Error):
        nf4.layernorm_bwd(X, X, w, st, st, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(nf4.NF4Error):
        nf4.layernorm_fwd(X, w, outs=(X, None, None, None, None, None))
