"""The adapters where every product takes its larger tiles (needs an MI355X): the calls of test_gpu_adapters.py that its
sizes make in tiles of 16 rows, the largest batch and the largest pool."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

try:
    import quantized_lora_fine_amd as nf4
except ImportError as exc:
    if torch.cuda.is_available():
        raise
    pytest.skip(f"libnf4lora.so not loaded: {exc}", allow_module_level=True)

from tests.test_gpu_adapters import Case, graph_of, on  # noqa: E402
from tests.test_gpu_fp8 import DEV, bits  # noqa: E402

WIDTH, RANK = 8208, 40
# tiles of 128 rows, and of 64
COUNTS = [[1500, 0, 700], [180] * 12]


def same(a, b, rows):
    rows = torch.from_numpy(rows).to(DEV)
    return torch.equal(a[rows].view(torch.int16), b[rows].view(torch.int16))


@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_large_without_base_in_place_and_again(counts):
    c = Case(31, counts, 30, WIDTH, WIDTH, RANK, True, base=False)
    c.check_fwd()
    c.check_bwd()
    c = Case(32, counts, 30, WIDTH, WIDTH, RANK, True)
    some = ~c.none
    Y, T = c.fwd()
    dX, dL1, dL2 = c.bwd()
    off, order = c.lists()
    X, L1, L2, s, dY, t = (on(v) for v in (c.X, c.L1, c.L2, c.s, c.dY, c.T))
    keep, keep_x = on(c.base).clone(), on(c.base_x).clone()
    nf4.adapters_fwd(X, L1, L2, s, off, order, keep, out=keep, want_T=False)
    got = nf4.adapters_bwd(dY, X, t, L1, L2, s, off, order, base=keep_x, dX=keep_x)
    assert same(keep, Y, some) and same(keep_x, dX, some)
    assert same(keep, on(c.base), c.none) and same(keep_x, on(c.base_x), c.none)
    assert torch.equal(got[1], dL1) and torch.equal(got[2], dL2)
    _, a, b = c.bwd(want_dX=False)
    assert torch.equal(a, dL1) and torch.equal(b, dL2)


@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_large_rows_alone(counts):
    # rows without an adapter hold no number, one row of the last adapter an infinity
    c = Case(33, counts, 30, WIDTH, WIDTH, RANK, True)
    Y, T = c.fwd()
    got = c.bwd()
    none = torch.from_numpy(c.none)
    c.X[none], c.dY[none], c.T[none] = float("nan"), float("nan"), float("nan")
    c.base[none], c.base_x[none] = float("inf"), float("inf")
    row = int(np.flatnonzero(c.ids == len(counts) - 1)[3])
    c.X[row, 11] = float("inf")
    some = ~c.none
    some[row] = False
    Y2, T2 = c.fwd()
    again = c.bwd()
    assert same(Y, Y2, some) and torch.equal(T[torch.from_numpy(some)], T2[torch.from_numpy(some)])
    assert torch.isinf(T2[row]).all() and not torch.isfinite(Y2[row]).any()
    assert same(got[0], again[0], some) and torch.equal(got[2], again[2])
    # dL1: column 11 of the last adapter alone
    got[1][-1, 11], again[1][-1, 11] = 0, 0
    assert torch.equal(got[1], again[1])


@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_large_lists_that_hold_anything(counts):
    c = Case(34, counts, 30, WIDTH, WIDTH, RANK, True)
    M, n, big = c.M, c.n, 2 ** 31 - 1
    off, order = c.lists()
    X, L1, L2, s, dY, t, base, base_x = (on(v) for v in (c.X, c.L1, c.L2, c.s, c.dY, c.T, c.base, c.base_x))
    gy = torch.full((M + 400, WIDTH), 0.375, dtype=torch.bfloat16, device=DEV)
    gx = torch.full((M + 400, WIDTH), 0.375, dtype=torch.bfloat16, device=DEV)
    g1 = torch.full((n + 2, WIDTH, RANK), 0.375, device=DEV)
    g2 = torch.full((n + 2, RANK, WIDTH), 0.375, device=DEV)
    end = off.tolist()
    for offs in ([-5] + end[1:-1] + [big], end[::-1], [big, -big] * (n + 1), [0] * n + [-1], [M] * (n + 1),
                 [0] + [M] * n, [0, M] * (n + 1)):
        o = torch.tensor(offs[:n + 1], dtype=torch.int32, device=DEV)
        for orders in (order, None, torch.full_like(order, big), torch.where(order % 3 == 0, -7, order)):
            nf4.adapters_fwd(X, L1, L2, s, o, orders, base, out=gy[200:200 + M])
            nf4.adapters_bwd(dY, X, t, L1, L2, s, o, orders, base=base_x, dX=gx[200:200 + M], dL1=g1[1:1 + n],
                             dL2=g2[1:1 + n])
            torch.cuda.synchronize()
            for g, k in ((gy, 200), (gx, 200), (g1, 1), (g2, 1)):
                assert torch.all(g[:k] == 0.375) and torch.all(g[-k:] == 0.375)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_large_captured_and_replayed(counts, fmt):
    rng = np.random.default_rng(35)
    c = Case(35, counts, 0, WIDTH, WIDTH, RANK, True, fmt)
    X, L1, L2, s, dY, T, base_x, sx = (on(t) for t in (c.X, c.L1, c.L2, c.s, c.dY, c.T, c.base_x, c.sx))
    bf = on(c.base)
    ids = on(torch.from_numpy(c.ids))

    def step():
        order, offsets = nf4.route(ids, c.n)
        Y, t = nf4.adapters_fwd(dY, L1, L2, s, offsets, order, bf)  # as wide as X
        return (Y, t) + nf4.adapters_bwd(dY, X, T, L1, L2, s, offsets, order, sx, base_x)

    g, outs = graph_of(step)
    for k in range(3):
        ids.copy_(torch.from_numpy(rng.integers(0, c.n, c.M).astype(np.int32)))
        for t in outs:
            t.zero_()
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(outs, want, strict=True):
            assert np.array_equal(bits(a), bits(b)), k


def test_the_most_rows():
    # 2^26 rows of 16 columns in whole numbers; the last adapter's are checked, and some of the first's
    M, w, r = 1 << 26, 16, 8
    gen = torch.Generator(device=DEV).manual_seed(36)

    def draw(cols, top):
        return torch.randint(-top, top + 1, (M, cols), generator=gen, device=DEV, dtype=torch.int8).to(torch.bfloat16)

    X, dY, base = draw(w, 2), draw(w, 1), draw(w, 4)
    cpu = np.random.default_rng(37)
    l1, l2 = cpu.integers(-1, 2, (2, w, r)), cpu.integers(-1, 2, (2, r, w))
    L1, L2 = (torch.from_numpy(v).to(torch.bfloat16).to(DEV) for v in (l1, l2))
    s, off = torch.tensor([0.5, 2.0], device=DEV), torch.tensor([0, M - 50, M], dtype=torch.int32, device=DEV)
    Y, T = nf4.adapters_fwd(X, L1, L2, s, off, None, base)
    rows = [0, 1, (1 << 25) + 77, M - 51]
    for a, at in ((0, torch.tensor(rows, device=DEV)), (1, torch.arange(M - 50, M, device=DEV))):
        x, g = X[at].cpu().double(), dY[at].cpu().double()
        t = x @ torch.from_numpy(l1[a]).double()
        assert torch.equal(T[at].cpu().double(), t)
        want = base[at].cpu().double() + float(s[a]) * (t @ torch.from_numpy(l2[a]).double())
        assert torch.equal(Y[at].cpu(), want.to(torch.bfloat16))
    del Y
    dX, dL1, dL2 = nf4.adapters_bwd(dY, X, T, L1, L2, s, off, None, base=base)
    for a, at in ((0, torch.tensor(rows, device=DEV)), (1, torch.arange(M - 50, M, device=DEV))):
        g = float(s[a]) * (dY[at].cpu().double() @ torch.from_numpy(l2[a]).double().T)
        want = base[at].cpu().double() + g @ torch.from_numpy(l1[a]).double().T
        assert torch.equal(dX[at].cpu(), want.to(torch.bfloat16))
    x, y, t = X[M - 50:].cpu().double(), dY[M - 50:].cpu().double(), T[M - 50:].cpu().double()
    assert torch.equal(dL1[1].cpu().double(), x.T @ g)
    assert torch.equal(dL2[1].cpu().double(), 2 * t.T @ y)
    assert torch.isfinite(dL1).all() and torch.isfinite(dL2).all()


def test_the_most_adapters():
    rng = np.random.default_rng(38)
    for M in (3, 700):
        counts = np.bincount(rng.integers(0, 4096, M), minlength=4096)
        counts[-1] += 2
        c = Case(39, counts.tolist(), 1, 64, 48, 8, True)
        c.check_fwd()
        c.check_bwd()
