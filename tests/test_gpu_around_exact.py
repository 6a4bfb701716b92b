"""The operators around a shared projection on whole numbers, whose products and sums fp32 holds exactly, and on arrays
whose offsets pass 32 bits (needs an MI355X).

In whole numbers nothing is rounded but the bf16 outputs, so results are held to the exact ones bit for bit: T and G
of up to 24 bits that lost one in a product, or a sum that took a row twice or not at all, would show."""
import numpy as np
import pytest
import torch

from oracle import around

pytestmark = pytest.mark.gpu

try:
    import quantized_lora_fine_amd as nf4
except ImportError as exc:
    if torch.cuda.is_available():
        raise
    pytest.skip(f"libnf4lora.so not loaded: {exc}", allow_module_level=True)

from tests.test_gpu_fp8 import DEV  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEV)


def lists(counts, spare, rng):
    ids = np.concatenate([np.full(c, a) for a, c in enumerate(counts)] + [np.full(spare, -1)]).astype(np.int32)
    rng.shuffle(ids)
    return ids, *around.route(ids, len(counts))


# some of 1024 rows or fewer, some of more, some of more than 64 adapters, with rows for tiles of 16, 64 and 128
COUNTS = [[1], [12, 0, 3], [700], [300, 0, 129, 513], [3] * 70, [1100], [1, 1023], [500, 0, 561, 39],
          [5000, 0, 64, 65, 1, 3000], [700] * 12]
WIDTHS = [(272, 144, 16), (1040, 528, 32), (528, 272, 64), (144, 400, 136), (272, 528, 8), (1024, 2048, 64),
          (2048, 1024, 48), (8208, 144, 16)]


# enough rows and columns for the larger tiles of every product, whole ones and not
LARGE = [([3000, 0, 1500, 700], 8208, 8208, 16), ([170] * 30, 8208, 8208, 32), ([2600, 2624], 8192, 8192, 64),
         ([170] * 30, 4112, 8208, 64), ([2000, 96], 8208, 8208, 136), ([4096], 4096, 8192, 8),
         ([2000, 96], 8208, 8208, 96), ([170] * 16, 8192, 8192, 128), ([100] * 12, 4096, 4096, 128)]
CASES = [(c, *w) for c in COUNTS for w in WIDTHS] + LARGE


@pytest.mark.parametrize("counts,h,o,r", CASES, ids=str)
def test_forward_in_whole_numbers(counts, h, o, r):
    rng = np.random.default_rng(sum(counts) + h + r)
    ids, order, offsets = lists(counts, 5, rng)
    n, M = len(counts), len(ids)
    x, l1 = rng.integers(-3, 4, (M, h)), rng.integers(-2, 3, (n, h, r))
    l2, base, s = rng.integers(-1, 2, (n, r, o)), rng.integers(-64, 65, (M, o)), rng.choice([0.5, 1.0, 2.0], n)
    y, t, S, _, _ = around.adapters_fwd(x, l1, l2, s, order, offsets, base)
    # T is below 2^16, which two bf16 values hold, and every sum below 2^23 (an s of 1/2 needs one bit more)
    assert np.max(np.abs(t)) < 2 ** 16 and np.max(S) < 2 ** 23
    Y, T = nf4.adapters_fwd(dev(x, BF16), dev(l1, BF16), dev(l2, BF16), dev(s, F32), dev(offsets, torch.int32),
                            dev(order, torch.int32), dev(base, BF16))
    some = torch.from_numpy(ids >= 0)
    assert torch.equal(T.cpu().double()[some], torch.from_numpy(t)[some])
    assert torch.equal(Y.cpu()[some], torch.from_numpy(y).to(BF16)[some])


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("h,o,r", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_gradients_in_whole_numbers(counts, h, o, r, fmt):
    rng = np.random.default_rng(sum(counts) + 3 * h + r)
    ids, order, offsets = lists(counts, 5, rng)
    n, M = len(counts), len(ids)
    # every column of dY, and of X, has one row of each adapter, so that no sum passes 24 bits
    take = min(30, o)
    dy, x = np.zeros((M, o)), np.zeros((M, h))
    for a in range(n):
        rows = order[offsets[a]:offsets[a + 1]]
        if not len(rows):
            continue
        active = rng.permutation(rows)[:max(1, o // take)]
        for row, cols in zip(active, rng.permutation(o)[:take * (o // take)].reshape(-1, take), strict=False):
            dy[row, cols] = rng.choice([-1, 1], take)
        x[rng.choice(active, h), np.arange(h)] = rng.choice([-1, 1], h)
    l1 = rng.integers(-1, 2, (n, h, r))
    l2 = rng.integers(-127, 128, (n, r, o)) * 2.0 ** (6 * (np.arange(o) % 3))
    t = rng.integers(2 ** 23, 2 ** 24, (M, r)) * rng.choice([-1, 1], (M, r))
    s = rng.choice([0.5, 1.0, 2.0], n)
    sx = np.ones((M, (h + 127) // 128))
    if fmt:
        sx = 2.0 ** rng.integers(-2, 3, sx.shape)
        one = {"e4m3": 0x38, "e5m2": 0x3C}[fmt]
        codes = np.where(x == 0, 0, np.where(x > 0, one, one | 0x80)).astype(np.uint8)
        X = torch.from_numpy(codes).view({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]).to(DEV)
    else:
        x *= 2.0 ** rng.integers(-2, 3, x.shape)
        X = dev(x, BF16)
    x64 = x * np.repeat(sx, 128, 1)[:, :h]
    _, (dl1, S1), (dl2, S2) = around.adapters_bwd(dy, x64, t, l1, l2, s, order, offsets, None)
    # as fp32 holds them: one term of T's bits, G's terms below 2^24, and powers of two
    assert np.array_equal(np.abs(dl2), S2) and np.max(np.abs(dy) @ np.max(np.abs(l2), (0, 1))) < 2 ** 24
    dX, dL1, dL2 = nf4.adapters_bwd(dev(dy, BF16), X, dev(t, F32), dev(l1, BF16), dev(l2, BF16), dev(s, F32),
                                    dev(offsets, torch.int32), dev(order, torch.int32),
                                    dev(sx, F32) if fmt else None)
    assert torch.equal(dL1.cpu().double(), torch.from_numpy(dl1))
    assert torch.equal(dL2.cpu().double(), torch.from_numpy(dl2))
    # without dX the sums are joined by another kernel
    again = nf4.adapters_bwd(dev(dy, BF16), X, dev(t, F32), dev(l1, BF16), dev(l2, BF16), dev(s, F32),
                             dev(offsets, torch.int32), dev(order, torch.int32), dev(sx, F32) if fmt else None,
                             want_dX=False)
    assert torch.equal(again[1], dL1) and torch.equal(again[2], dL2)


@pytest.mark.parametrize("counts,h,o,r", CASES, ids=str)
def test_dense_gradients_in_whole_numbers(counts, h, o, r):
    # every row and column takes part; G is below 2^16, which two bf16 values hold
    rng = np.random.default_rng(sum(counts) + 5 * h + r)
    ids, order, offsets = lists(counts, 5, rng)
    n, M = len(counts), len(ids)
    dy, x, t = rng.integers(-1, 2, (M, o)), rng.integers(-2, 3, (M, h)), rng.integers(-8, 9, (M, r))
    l1, l2 = rng.integers(-1, 2, (n, h, r)), rng.integers(-1, 2, (n, r, o))
    s, base = rng.choice([0.5, 1.0, 2.0], n), rng.integers(-64, 65, (M, h))
    (dx, _), (dl1, S1), (dl2, S2) = around.adapters_bwd(dy, x, t, l1, l2, s, order, offsets, base)
    # dL1's terms are 2 |G|, of about 0.54 sqrt(o); its sums of magnitudes count G's own terms, which cancel
    g = np.abs(np.stack([dy[m] @ l2[a].T if a >= 0 else np.zeros(r) for m, a in enumerate(ids)]))
    assert np.max(g) < 2 ** 16 and 2 * np.max(np.sum(g, 0)) < 2 ** 23 and np.max(S2) < 2 ** 23 and r * np.max(g) < 2 ** 22
    dX, dL1, dL2 = nf4.adapters_bwd(dev(dy, BF16), dev(x, BF16), dev(t, F32), dev(l1, BF16), dev(l2, BF16), dev(s, F32),
                                    dev(offsets, torch.int32), dev(order, torch.int32), base=dev(base, BF16))
    some = torch.from_numpy(ids >= 0)
    assert torch.equal(dX.cpu()[some], torch.from_numpy(dx).to(BF16)[some])
    assert torch.equal(dL1.cpu().double(), torch.from_numpy(dl1))
    assert torch.equal(dL2.cpu().double(), torch.from_numpy(dl2))


def small(M, cols, top, seed):
    """bf16 whole numbers in [-top, top], made a slice of rows at a time."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = torch.empty(M, cols, dtype=BF16, device=DEV)
    for m in range(0, M, 8192):
        out[m:m + 8192] = torch.randint(-top, top + 1, (min(8192, M - m), cols), generator=g, device=DEV,
                                        dtype=torch.int8).to(BF16)
    return out


@pytest.mark.parametrize("wide", ["X", "dY"])
@pytest.mark.parametrize("fmt", [None, torch.float8_e4m3fn])
def test_adapters_past_32_bits(wide, fmt):
    # 2^32 and some values of X (and dX), or of Y (and dY); the last rows' adapters are checked, and rows of the first
    M, r = (1 << 17) + 777, 8
    h, o = (32784, 16) if wide == "X" else (16, 32784)
    counts = [M - 60, 20, 40]
    assert M * max(h, o) > 1 << 32
    offsets = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device=DEV)
    X, dY = small(M, h, 2, 1), small(M, o, 1, 2)
    rng = np.random.default_rng(3)
    l1, l2, s = rng.integers(-1, 2, (3, h, r)), rng.integers(-1, 2, (3, r, o)), np.array([1.0, 0.5, 2.0])
    L1, L2, S = dev(l1, BF16), dev(l2, BF16), dev(s, F32)
    Y, T = nf4.adapters_fwd(X, L1, L2, S, offsets)
    rows = np.concatenate([[0, 1, 65535, M // 2, M - 62, M - 61], np.arange(M - 60, M)])
    at = torch.from_numpy(rows).to(DEV)
    sub = np.searchsorted(rows, np.cumsum([0] + counts))
    x, dy = X[at].cpu().double().numpy(), dY[at].cpu().double().numpy()
    y, t, _, _, _ = around.adapters_fwd(x, l1, l2, s, None, sub, None)
    assert np.max(np.abs(t)) < 2 ** 16 and np.max(np.abs(y)) < 2 ** 23
    assert torch.equal(T[at].cpu().double(), torch.from_numpy(t))
    assert torch.equal(Y[at].cpu(), torch.from_numpy(y).to(BF16))
    del Y
    sx = None
    if fmt is not None:
        X = X.to(fmt)
        sx = torch.ones(M, (h + 127) // 128, device=DEV)
    base = small(M, h, 4, 4)
    dX, dL1, dL2 = nf4.adapters_bwd(dY, X, T, L1, L2, S, offsets, None, sx, base)
    (dx, _), (dl1, S1), (dl2, S2) = around.adapters_bwd(dy, x, t, l1, l2, s, None, sub, base[at].cpu().double().numpy())
    assert np.max(S1[1:]) < 2 ** 23 and np.max(S2[1:]) < 2 ** 23
    assert torch.equal(dX[at].cpu(), torch.from_numpy(dx).to(BF16))
    assert torch.equal(dL1[1:].cpu().double(), torch.from_numpy(dl1)[1:])
    assert torch.equal(dL2[1:].cpu().double(), torch.from_numpy(dl2)[1:])


def test_route_of_the_most_rows():
    M, n = 1 << 30, 3
    ids = torch.arange(M, dtype=torch.int32, device=DEV).remainder_(4)  # the fourth has no adapter
    order, offsets = nf4.route(ids, n)
    quarter = M // 4
    assert offsets.tolist() == [0, quarter, 2 * quarter, 3 * quarter]
    want = torch.arange(quarter, dtype=torch.int32, device=DEV).mul_(4)
    for k in range(4):
        assert torch.equal(order[k * quarter:(k + 1) * quarter], want + k)


def test_layernorm_past_32_bits():
    # more values than 32 bits count, and more rows than one launch takes
    M, H = (1 << 28) + 5, 16
    X = torch.zeros(M, H, dtype=BF16, device=DEV)
    rows = torch.tensor([0, 1, (1 << 26) - 1, 1 << 26, (1 << 27) + 3, M - 6, M - 2, M - 1])
    rng = np.random.default_rng(5)
    x = dev(rng.integers(-8, 9, (len(rows), H)), BF16)
    X[rows.to(DEV)] = x
    w, b = dev(rng.integers(1, 4, H), BF16), dev(rng.integers(-3, 4, H), BF16)
    Y, _, _, _, mean, rstd = nf4.layernorm_fwd(X, w, b, want_stats=True)
    y1, _, _, _, m1, r1 = nf4.layernorm_fwd(x, w, b, want_stats=True)  # these rows by themselves
    for got, want in ((Y, y1), (mean, m1), (rstd, r1)):
        assert torch.equal(got[rows.to(DEV)], want)
    assert torch.equal(Y[5], b) and torch.equal(Y[M - 3], b)  # rows of equal values
    del Y
    dY = torch.zeros_like(X)
    dy = dev(rng.integers(-4, 5, (len(rows), H)), BF16)
    dY[rows.to(DEV)] = dy
    dX, dw, db = nf4.layernorm_bwd(dY, X, w, mean, rstd)
    d1, w1, b1 = nf4.layernorm_bwd(dy, x, w, m1, r1)
    assert torch.equal(dX[rows.to(DEV)], d1)
    assert torch.equal(db, b1)                                       # whole numbers
    # 8 rows' terms in another order, each no more than 4 * 4 (|xhat| <= sqrt(H - 1))
    assert torch.max(torch.abs(dw - w1)).item() <= 8 * 8 * 16 * 2.0 ** -24
    assert not dX[5].any() and not dX[M - 3].any()
