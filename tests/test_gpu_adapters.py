"""The adapters of many requests and their gradients against the fp64 oracle (needs an MI355X).

Outputs are held to the roundings they go through: half a step of the output's type relative to the value, EPS32 for
each fp32 addition in turn in proportion to the sum of the terms' magnitudes, and 2^-17 of T or G where it enters a
product as two bf16 values.  A row that no adapter has keeps what it held, bit for bit."""
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

from tests.test_gpu_fp8 import BF16, DEV, EPS32, bf16_np, bits, check_within, f64, rows_of  # noqa: E402

SPLIT = 2.0 ** -17    # what two bf16 values leave of an fp32 one


def deep(k):
    """Additions in turn in a contraction of k: an MFMA's 32 products count as 16, an order of its own among them; then
    4 waves, and the splits."""
    return k / 2 + 64


def on(t):
    return None if t is None else t.to(DEV)


class Case:
    """A pool and a batch; counts: rows of each adapter, spare rows without one."""

    def __init__(self, seed, counts, spare, h, o, r, ordered, fmt=None, base=True):
        rng = np.random.default_rng(seed)
        self.n, self.M, self.h, self.o, self.r = len(counts), sum(counts) + spare, h, o, r
        ids = np.concatenate([np.full(c, a) for a, c in enumerate(counts)] + [np.full(spare, -1)]).astype(np.int32)
        if ordered:
            rng.shuffle(ids)
        self.ids, (order, self.offsets) = ids, around.route(ids, self.n)
        self.order = order if ordered else None
        self.L1 = bf16_np(rng.standard_normal((self.n, h, r)) * h ** -0.5)
        self.L2 = bf16_np(rng.standard_normal((self.n, r, o)) * 0.05)
        self.s = torch.from_numpy((0.25 + 2 * rng.random(self.n)).astype(np.float32))
        self.X = bf16_np(rows_of(rng, self.M, h))
        self.dY = bf16_np(1e-3 * rows_of(rng, self.M, o))
        self.T = torch.from_numpy(rng.standard_normal((self.M, r)).astype(np.float32))
        self.base = bf16_np(rng.standard_normal((self.M, o))) if base else None
        self.base_x = bf16_np(1e-3 * rng.standard_normal((self.M, h))) if base else None
        self.x64, self.sx, self.fmt = f64(self.X), None, fmt
        if fmt:
            codes, sx = fp8.quantize(self.X.float().numpy(), 1, fmt)
            self.X = torch.from_numpy(codes).view({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt])
            self.sx = torch.from_numpy(sx)
            self.x64 = fp8.code_values(fmt)[codes] * fp8._spread(sx.astype(np.float64), 1, self.M, h)
        self.none = ids < 0

    def lists(self):
        return on(torch.from_numpy(self.offsets)), None if self.order is None else on(torch.from_numpy(self.order))

    def fwd(self, **kw):
        off, order = self.lists()
        return nf4.adapters_fwd(on(self.X), on(self.L1), on(self.L2), on(self.s), off, order, on(self.base), **kw)

    def bwd(self, **kw):
        off, order = self.lists()
        kw.setdefault("base", on(self.base_x))
        return nf4.adapters_bwd(on(self.dY), on(self.X), on(self.T), on(self.L1), on(self.L2), on(self.s), off, order,
                                on(self.sx), **kw)

    def check_fwd(self):
        out = torch.full((self.M, self.o), 0.375, dtype=torch.bfloat16, device=DEV)
        t = torch.full((self.M, self.r), 0.375, device=DEV)
        Y, T = self.fwd(out=out, T_out=t)
        assert Y is out and T is t
        y, t64, S, Q, R = around.adapters_fwd(self.x64, f64(self.L1), f64(self.L2), f64(self.s), self.order,
                                              self.offsets, None if self.base is None else f64(self.base))
        y[self.none], t64[self.none] = 0.375, 0.375
        check_within("T", T, t64, Q * deep(self.h) * EPS32)
        slack = R * deep(self.h) * EPS32 + S * (SPLIT + deep(2 * self.r) * EPS32)
        check_within("Y", Y, y, np.where(self.none[:, None], 0, np.abs(y) * BF16 + slack * (1 + BF16)))
        return Y, T

    def check_bwd(self):
        dX = torch.full((self.M, self.h), 0.375, dtype=torch.bfloat16, device=DEV)
        got = self.bwd(dX=dX)
        assert got[0] is dX
        (dx, Sx), (dl1, S1), (dl2, S2) = around.adapters_bwd(
            f64(self.dY), self.x64, f64(self.T), f64(self.L1), f64(self.L2), f64(self.s), self.order, self.offsets,
            None if self.base_x is None else f64(self.base_x))
        dx[self.none] = 0.375
        slack = Sx * (deep(self.o) * EPS32 + SPLIT + deep(2 * self.r) * EPS32)
        check_within("dX", dX, dx, np.where(self.none[:, None], 0, np.abs(dx) * BF16 + slack * (1 + BF16)))
        # dL1, dL2: fp32 all the way, three MFMAs for each 32 rows
        check_within("dL1", got[1], dl1, S1 * (deep(self.o) + deep(3 * self.M)) * EPS32)
        check_within("dL2", got[2], dl2, S2 * deep(3 * self.M) * EPS32)
        return got


COUNTS = [([1], 0), ([3], 2), ([0, 1, 0], 0), ([1] * 9, 0), ([5, 0, 12, 1], 3), ([16, 17, 15, 0, 2], 1), ([64], 0),
          ([65, 0, 63], 0), ([200, 1, 130, 0], 7), ([0, 0], 5), ([700], 0), ([300, 0, 129, 513], 20)]


@pytest.mark.parametrize("h,o,r", [(272, 144, 16), (64, 1040, 8), (1040, 272, 64), (528, 656, 40), (144, 272, 256),
                                   (16, 16, 24)])
@pytest.mark.parametrize("ordered", [False, True])
@pytest.mark.parametrize("counts,spare", COUNTS)
def test_adapters(counts, spare, ordered, h, o, r):
    c = Case(sum(counts) + h + r, counts, spare, h, o, r, ordered)
    c.check_fwd()
    c.check_bwd()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("h,o,r", [(272, 144, 16), (1040, 272, 64), (528, 400, 32), (144, 272, 200), (16, 48, 8)])
@pytest.mark.parametrize("counts,spare", [([1], 0), ([5, 0, 12, 1], 3), ([200, 1, 130, 0], 7), ([700], 0)])
def test_adapters_from_a_checkpoint(counts, spare, h, o, r, fmt):
    Case(sum(counts) * 3 + h + r, counts, spare, h, o, r, True, fmt).check_bwd()


@pytest.mark.parametrize("r", [8, 16, 32, 48, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("counts", [[7, 2, 0, 1], [150, 90]])
def test_adapters_of_every_rank(counts, r):
    c = Case(r, counts, 2, 400, 528, r, True)
    c.check_fwd()
    c.check_bwd()


@pytest.mark.parametrize("counts,spare,h,o,r", [([1], 0, 4096, 4096, 16), ([1] * 5 + [0] * 60 + [2], 1, 4096, 11008, 32),
                                                ([500, 1500], 3, 4096, 2064, 16), ([900], 0, 11008, 4096, 64)])
def test_adapters_of_real_widths(counts, spare, h, o, r):
    c = Case(h + o, counts, spare, h, o, r, True)
    c.check_fwd()
    c.check_bwd()


def test_adapters_long_contractions():
    c = Case(1, [3, 20], 0, 66000, 272, 16, False)
    c.check_fwd()
    c = Case(2, [3, 20], 0, 272, 66000, 16, False)
    c.check_bwd()


def test_adapters_many():
    rng = np.random.default_rng(12)
    counts = rng.integers(0, 3, 300).tolist() + [0] * 700 + [40] + [0] * 95 + [1]
    c = Case(3, counts, 5, 144, 272, 8, True)
    c.check_fwd()
    c.check_bwd()


def test_adapters_without_base_and_in_place():
    for counts in ([5, 0, 12], [200, 130]):
        c = Case(4, counts, 2, 272, 400, 16, True, base=False)
        c.check_fwd()
        c.check_bwd()
        c = Case(5, counts, 2, 272, 400, 16, True)
        Y, T = c.fwd()
        keep = on(c.base).clone()
        Y2, none = c.fwd(out=None, want_T=False)
        assert none is None
        off, order = c.lists()
        Y3, _ = nf4.adapters_fwd(on(c.X), on(c.L1), on(c.L2), on(c.s), off, order, keep, out=keep)
        assert Y3 is keep
        some = ~c.none
        assert np.array_equal(bits(Y)[some], bits(Y2)[some]) and np.array_equal(bits(Y)[some], bits(keep)[some])
        assert np.array_equal(bits(keep)[c.none], bits(c.base)[c.none])
        dX, dL1, dL2 = c.bwd()
        keep = on(c.base_x).clone()
        got = c.bwd(base=keep, dX=keep)
        assert np.array_equal(bits(dX)[some], bits(keep)[some])
        assert np.array_equal(bits(keep)[c.none], bits(c.base_x)[c.none])
        assert torch.equal(got[1], dL1) and torch.equal(got[2], dL2)
        none, a, b = c.bwd(want_dX=False)
        assert none is None and torch.equal(a, dL1) and torch.equal(b, dL2)


def test_adapters_gradients_against_differences():
    # f = sum of dY * Y in 64 bits on the CPU, along random directions of L1, L2 and X
    rng = np.random.default_rng(8)
    c = Case(6, [30, 0, 70], 4, 144, 272, 16, True, base=False)
    _, T = c.fwd()
    off, order = c.lists()
    dX, dL1, dL2 = (f64(t) for t in nf4.adapters_bwd(on(c.dY), on(c.X), T, on(c.L1), on(c.L2), on(c.s), off, order))

    def f(x, l1, l2):
        return np.sum(around.adapters_fwd(x, l1, l2, f64(c.s), c.order, c.offsets, None)[0] * f64(c.dY))

    x, l1, l2 = f64(c.X), f64(c.L1), f64(c.L2)
    dX[c.none] = 0
    for which, got in ((0, dX), (1, dL1), (2, dL2)):
        e = rng.standard_normal(got.shape)
        ends = []
        for t in (1e-4, -1e-4):
            v = [x, l1, l2]
            v[which] = v[which] + t * e
            ends.append(f(*v))
        want, terms = (ends[0] - ends[1]) / 2e-4, np.sum(np.abs(got * e))  # f is linear in each: no error of t^2
        assert abs(np.sum(got * e) - want) <= terms * ((BF16 if which == 0 else 0) + 1e-5), which


def test_adapters_rows_alone():
    # a row does not depend on what stands in the others, nor on rows that no adapter has
    for counts in ([5, 0, 12], [200, 0, 129]):
        c = Case(7, counts, 9, 272, 400, 16, True)
        Y, T = c.fwd()
        got = c.bwd()
        none = torch.from_numpy(c.none)
        c.X[none], c.dY[none], c.T[none] = float("nan"), float("nan"), float("nan")
        c.base[none], c.base_x[none] = float("inf"), float("inf")
        some = ~c.none
        Y2, T2 = c.fwd()
        assert np.array_equal(bits(Y)[some], bits(Y2)[some]) and np.array_equal(bits(T)[some], bits(T2)[some])
        for a, b in zip(got[1:], c.bwd()[1:]):
            assert torch.equal(a, b)
        # a NaN in one row: that row alone, and its adapter's gradients
        row = int(np.nonzero(c.ids == 2)[0][0])
        c.X[row, 3] = float("nan")
        Y3, _ = c.fwd()
        others = some & (np.arange(c.M) != row)
        assert torch.isnan(Y3[row]).all() and np.array_equal(bits(Y)[others], bits(Y3)[others])
        _, dL1, _ = c.bwd()
        assert torch.equal(dL1[:2], got[1][:2]) and torch.isnan(dL1[2, 3]).all()
        assert torch.equal(dL1[2, 4:], got[1][2, 4:])


def test_adapters_infinities():
    # an infinity in X is one in T and Y, not a NaN
    c = Case(9, [3, 30], 0, 272, 400, 16, False)
    c.X[2, 5] = float("inf")
    c.X[20, 7] = float("-inf")
    Y, T = c.fwd()
    for row in (2, 20):
        assert torch.isinf(T[row]).all()
    assert not torch.isinf(T[[0, 1, 3, 4]]).any()
    want = around.adapters_fwd(f64(c.X), f64(c.L1), f64(c.L2), f64(c.s), c.order, c.offsets, f64(c.base))[0]
    assert np.array_equal(np.isfinite(f64(Y)), np.isfinite(want))


def test_adapters_lists_that_hold_anything():
    # offsets outside [0, M] or not ascending, orders that name no row: nothing outside the outputs is written
    c = Case(10, [40, 30, 20], 10, 272, 400, 16, True)
    M = c.M
    off, order = c.lists()
    guard = torch.full((3 * M, c.o), 0.375, dtype=torch.bfloat16, device=DEV)
    gx = torch.full((3 * M, c.h), 0.375, dtype=torch.bfloat16, device=DEV)
    g1 = torch.full((9, c.h, c.r), 0.375, device=DEV)
    g2 = torch.full((9, c.r, c.o), 0.375, device=DEV)
    big = 2 ** 31 - 1
    for offs in ([0, 40, 70, 90], [-5, 40, 70, big], [0, 90, 20, 100], [big, -big, 50, 7], [0, 0, 0, -1],
                 [100, 100, 100, 100], [-big, -1, big, big]):
        for orders in (order, None, torch.full_like(order, -1), torch.full_like(order, big),
                       torch.where(order % 3 == 0, -7, order)):
            o = torch.tensor(offs, dtype=torch.int32, device=DEV)
            nf4.adapters_fwd(on(c.X), on(c.L1), on(c.L2), on(c.s), o, orders, on(c.base), out=guard[M:2 * M])
            nf4.adapters_bwd(on(c.dY), on(c.X), on(c.T), on(c.L1), on(c.L2), on(c.s), o, orders, base=on(c.base_x),
                             dX=gx[M:2 * M], dL1=g1[3:6], dL2=g2[3:6])
            torch.cuda.synchronize()
            for g, k in ((guard, M), (gx, M), (g1, 3), (g2, 3)):
                assert torch.all(g[:k] == 0.375) and torch.all(g[2 * k:] == 0.375)
    # orders that name no row among good ones: those rows alone are left
    Y, _ = c.fwd()
    bad = torch.where(order % 3 == 0, -7, order)
    out = torch.full_like(Y, 0.375)
    nf4.adapters_fwd(on(c.X), on(c.L1), on(c.L2), on(c.s), off, bad, on(c.base), out=out)
    left = (np.arange(M) % 3 == 0) | c.none
    assert torch.all(out[torch.from_numpy(left)] == 0.375)
    assert np.array_equal(bits(out)[~left], bits(Y)[~left])


def test_adapters_repeat_bit_for_bit():
    c = Case(11, [300, 0, 129, 513], 20, 1040, 528, 64, True)
    some = ~c.none
    Y, T = c.fwd()
    got = c.bwd()
    for _ in range(3):
        Y2, T2 = c.fwd()
        again = c.bwd()
        assert np.array_equal(bits(Y)[some], bits(Y2)[some]) and np.array_equal(bits(T)[some], bits(T2)[some])
        assert np.array_equal(bits(got[0])[some], bits(again[0])[some])
        assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])


def test_adapters_empty():
    bf = dict(dtype=torch.bfloat16, device=DEV)
    L1, L2 = torch.ones(2, 272, 16, **bf), torch.ones(2, 16, 400, **bf)
    s, off = torch.ones(2, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    X, dY, T = torch.empty(0, 272, **bf), torch.empty(0, 400, **bf), torch.empty(0, 16, device=DEV)
    Y, t = nf4.adapters_fwd(X, L1, L2, s, off)
    assert Y.shape == (0, 400) and t.shape == (0, 16)
    d1, d2 = torch.ones(2, 272, 16, device=DEV), torch.ones(2, 16, 400, device=DEV)
    dX, _, _ = nf4.adapters_bwd(dY, X, T, L1, L2, s, off, dL1=d1, dL2=d2)
    assert dX.shape == (0, 272) and torch.all(d1 == 0) and torch.all(d2 == 0)


def test_adapters_refuse():
    c = Case(13, [5, 3], 0, 272, 400, 16, True)
    X, L1, L2, s, dY, T = (on(t) for t in (c.X, c.L1, c.L2, c.s, c.dY, c.T))
    off, order = c.lists()
    base, base_x = on(c.base), on(c.base_x)
    for bad in (lambda: nf4.adapters_fwd(X.float(), L1, L2, s, off), lambda: nf4.adapters_fwd(X, L1[0], L2, s, off),
                lambda: nf4.adapters_fwd(X, L1, L2[:1], s, off), lambda: nf4.adapters_fwd(X, L1, L2, s[:1], off),
                lambda: nf4.adapters_fwd(X, L1, L2, s, off[:2]), lambda: nf4.adapters_fwd(X, L1, L2, s, off.long()),
                lambda: nf4.adapters_fwd(X, L1, L2, s, off, order[:4]),
                lambda: nf4.adapters_fwd(X[:, :256], L1, L2, s, off),
                lambda: nf4.adapters_fwd(X, L1, L2, s, off, order, base[:4]),
                lambda: nf4.adapters_fwd(X, L1, L2, s, off, order, out=base_x),
                lambda: nf4.adapters_fwd(X, L1, L2, s, off, order, T_out=T[:4]),
                lambda: nf4.adapters_fwd(X, L1, L2, s.cpu(), off),
                lambda: nf4.adapters_bwd(dY, X, T.double(), L1, L2, s, off),
                lambda: nf4.adapters_bwd(X, X, T, L1, L2, s, off),
                lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, x_scales=torch.ones(8, 3, device=DEV)),
                lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, base=base),
                lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, dL1=L1)):
        with pytest.raises(ValueError):
            bad()
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    # these few rows need no workspace, and take any; 40 rows of two adapters need one
    assert nf4.adapters_workspace_bytes(nf4.NF4_OP_FWD, 8, 400, 272, 2, 16) == 0
    some = nf4.adapters_fwd(X, L1, L2, s, off, order, base, ws=small)
    assert torch.equal(some[0], nf4.adapters_fwd(X, L1, L2, s, off, order, base)[0])
    d = Case(21, [20, 20], 0, 272, 400, 16, True)
    XX, offd = on(d.X), d.lists()[0]
    for bad, status in ((lambda: nf4.adapters_fwd(XX, L1, L2, s, offd, ws=small), nf4.NF4_ERR_WORKSPACE),
                        (lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, ws=small), nf4.NF4_ERR_WORKSPACE),
                        (lambda: nf4.adapters_fwd(X, L1[:, :, :12].contiguous(), L2[:, :12].contiguous(), s, off),
                         nf4.NF4_ERR_SHAPE),
                        (lambda: nf4.adapters_fwd(X[:, :264].contiguous(), L1[:, :264].contiguous(), L2, s, off),
                         nf4.NF4_ERR_SHAPE),
                        (lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, dX=X), nf4.NF4_ERR_ALIAS)):
        with pytest.raises(nf4.NF4Error) as e:
            bad()
        assert e.value.status == status


def graph_of(step):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    return g, outs


@pytest.mark.parametrize("M", [40, 900])
def test_adapters_captured_and_replayed(M):
    # the routing is inside the graph: replays with other ids, with eager work and synchronizations in between
    rng = np.random.default_rng(M)
    c = Case(14, [M // 2, 0, M - M // 2], 0, 272, 400, 16, True)
    X, L1, L2, s, dY, base, base_x = (on(t) for t in (c.X, c.L1, c.L2, c.s, c.dY, c.base, c.base_x))
    ids = on(torch.from_numpy(c.ids))
    zero = torch.zeros((), device=DEV)

    def step():
        order, offsets = nf4.route(ids, 3)
        Y, T = nf4.adapters_fwd(X, L1, L2, s, offsets, order, base)
        dX, dL1, dL2 = nf4.adapters_bwd(dY, X, T, L1, L2, s, offsets, order, base=base_x)
        return Y, T, dX, dL1, dL2

    g, outs = graph_of(step)
    for k in range(4):
        ids.copy_(torch.from_numpy(rng.integers(0, 3, M).astype(np.int32)))
        for t in outs:
            t.zero_().add_(zero)
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert np.array_equal(bits(a), bits(b)), k


def test_adapters_two_graphs_share_a_workspace():
    c, d = Case(15, [300, 200], 0, 272, 400, 16, False), Case(16, [20, 30], 0, 272, 400, 16, False)
    n = max(nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, v.M, v.o, v.h, v.n, v.r) for v in (c, d))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    graphs = []
    for v in (c, d):
        X, L1, L2, s, dY, T, bx = (on(t) for t in (v.X, v.L1, v.L2, v.s, v.dY, v.T, v.base_x))
        off, _ = v.lists()
        graphs.append(graph_of(lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, off, base=bx, ws=ws)) + (v, (X, L1, L2, s, dY,
                                                                                                        T, bx, off)))
    for k in range(3):
        for g, outs, v, _ in graphs[:: 1 if k % 2 else -1]:
            g.replay()
        torch.cuda.synchronize()
        for g, outs, v, _ in graphs:
            for a, b in zip(outs, v.bwd()):
                assert np.array_equal(bits(a), bits(b)), k


def test_adapters_two_streams_at_once():
    cs = [Case(17, [300, 200, 40], 0, 1040, 528, 32, True), Case(18, [3, 1, 9], 2, 528, 1040, 16, True)]
    want = [(c.fwd(), c.bwd()) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = [[on(t) for t in (c.X, c.L1, c.L2, c.s, c.dY, c.T, c.base, c.base_x)] + list(c.lists()) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for st, (X, L1, L2, s, dY, T, base, base_x, off, order) in zip(streams, held):
            with torch.cuda.stream(st):
                got.append((nf4.adapters_fwd(X, L1, L2, s, off, order, base),
                            nf4.adapters_bwd(dY, X, T, L1, L2, s, off, order, base=base_x)))
        torch.cuda.synchronize()
        for c, a, b in zip(cs, got, want):
            some = ~c.none
            for u, v in zip(a[0] + (a[1][0],), b[0] + (b[1][0],)):
                assert np.array_equal(bits(u)[some], bits(v)[some])
            assert torch.equal(a[1][1], b[1][1]) and torch.equal(a[1][2], b[1][2])


def test_layer_around_a_shared_projection():
    """A run of them together: rows routed, the norm's two outputs, the 8-bit projection for all, the adapters beside
    it; back through the adapters from the norm's codes, the projection and the norm."""
    rng = np.random.default_rng(20)
    M, n, h, o, r = 150, 4, 272, 400, 16
    x, res = bf16_np(rows_of(rng, M, h)), bf16_np(rows_of(rng, M, h))
    w, b = bf16_np(1 + 0.1 * rng.standard_normal(h)), bf16_np(0.1 * rng.standard_normal(h))
    W = (0.05 * rng.standard_normal((o, h))).astype(np.float32)
    L1, L2 = bf16_np(rng.standard_normal((n, h, r)) * h ** -0.5), bf16_np(0.05 * rng.standard_normal((n, r, o)))
    s, ids = rng.random(n).astype(np.float32) + 0.5, rng.integers(-1, n, M).astype(np.int32)
    dY, dH = bf16_np(1e-2 * rows_of(rng, M, o)), bf16_np(1e-2 * rows_of(rng, M, h))
    ids[ids == 2] = 1  # an adapter without rows
    sd = on(torch.from_numpy(s))
    Wq, ws = nf4.fp8_quantize(on(torch.from_numpy(W)), 128)

    def layer(back=True):
        order, offsets = nf4.route(on(torch.from_numpy(ids)), n)
        y, hid, codes, sc, mean, rstd = nf4.layernorm_fwd(on(x), on(w), on(b), residual=on(res), want_fp8=True,
                                                          want_stats=True)
        Y = nf4.fp8_matmul(codes, sc, Wq, ws)
        nf4_Y, T = nf4.adapters_fwd(y, on(L1), on(L2), sd, offsets, order, base=Y, out=Y)
        assert nf4_Y is Y
        gq, gs = nf4.fp8_quantize(on(dY), 1, torch.float8_e5m2)
        dy = nf4.fp8_matmul(gq, gs, Wq, ws, True)
        _, dL1, dL2 = nf4.adapters_bwd(on(dY), codes, T, on(L1), on(L2), sd, offsets, order, x_scales=sc, base=dy,
                                       dX=dy)
        dx, dw, db = nf4.layernorm_bwd(dy, hid, on(w), mean, rstd, on(dH))
        return Y, T, dL1, dL2, dx, dw, db, (y, codes, sc, gq, gs, hid, mean, rstd)

    Y, T, dL1, dL2, dx, dw, db, (y, codes, sc, gq, gs, hid, mean, rstd) = layer()
    Wd = f64(nf4.fp8_dequantize(Wq, ws, 128))
    xq, gd = f64(nf4.fp8_dequantize(codes, sc)), f64(nf4.fp8_dequantize(gq, gs))
    order, offsets = around.route(ids, n)
    yb, t64, S, Q, R = around.adapters_fwd(f64(y), f64(L1), f64(L2), s, order, offsets, xq @ Wd.T)
    size = np.abs(xq) @ np.abs(Wd).T
    # the projection's own bounds (2^-11 of its terms, bf16), then the adapters'
    check_within("Y", Y, yb, 2.1 * BF16 * (np.abs(yb) + S) + size * 2.0 ** -11 + R * deep(h) * EPS32 + S * 2.0 ** -16)
    (dy64, Sx), (d1, S1), (d2, S2) = around.adapters_bwd(f64(dY), xq, f64(T) * (ids >= 0)[:, None], f64(L1), f64(L2), s,
                                                         order, offsets, gd @ Wd)
    check_within("dL1", dL1, d1, S1 * (deep(o) + deep(3 * M)) * EPS32)
    check_within("dL2", dL2, d2, S2 * deep(3 * M) * EPS32)
    assert torch.all(dL1[2] == 0) and torch.all(dL2[2] == 0)
    dx64, dw64, db64 = around.layernorm_grad(dy64, f64(hid), f64(w), f64(mean), f64(rstd), f64(dH))
    # dy is off by two bf16 roundings and the projection's bound; the norm's gradient is linear in it, with gains of
    # rstd |w| for a value and rstd (1 + |xhat|) for the means
    off = 2.1 * BF16 * (np.abs(dy64) + Sx) + (np.abs(gd) @ np.abs(Wd)) * 2.0 ** -11
    rs, xhat = f64(rstd)[:, None], np.abs(f64(hid) - f64(mean)[:, None]) * f64(rstd)[:, None]
    ow = off * np.abs(f64(w))
    gain = rs * (ow + ow.mean(1, keepdims=True) + xhat * (ow * xhat).mean(1, keepdims=True))
    check_within("dx", dx, dx64, gain * 1.01 + np.abs(dx64) * BF16 * (1 + BF16) + 1e-5 * (gain + np.abs(dx64)))
    check_within("dw", dw, dw64, (off * xhat).sum(0) * 1.01 + 1e-5 * np.abs(dy64 * xhat).sum(0))
    check_within("db", db, db64, off.sum(0) * 1.01 + 1e-5 * np.abs(dy64).sum(0))
    for a, c in zip(layer()[:7], (Y, T, dL1, dL2, dx, dw, db)):
        some = ids >= 0
        assert np.array_equal(bits(a)[some] if a.shape[0] == M else bits(a), bits(c)[some] if c.shape[0] == M else bits(c))
