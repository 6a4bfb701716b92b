"""The fp64 oracle of the operators around a shared projection against other forms of the same formulas (CPU)."""
import numpy as np
import pytest
import torch

from oracle import around


@pytest.mark.parametrize("M,n", [(0, 3), (1, 1), (50, 4), (200, 300)])
def test_route(M, n):
    ids = np.random.default_rng(M).integers(-1, n + 2, M).astype(np.int32)
    order, offsets = around.route(ids, n)
    key = np.where((ids >= 0) & (ids < n), ids, n)
    assert np.array_equal(order, np.argsort(key, kind="stable"))
    assert np.array_equal(offsets, np.searchsorted(np.sort(key), np.arange(n + 1)))


def test_layernorm_and_gradient():
    rng = np.random.default_rng(1)
    h, w, b, dy, dh = (torch.from_numpy(rng.standard_normal(s)) for s in ((7, 48), 48, 48, (7, 48), (7, 48)))
    h, w, b = (t.requires_grad_() for t in (h, w, b))
    y = torch.nn.functional.layer_norm(h, (48,), w, b, 1e-3)
    (torch.sum(y * dy) + torch.sum(h * dh)).backward()
    y64, mean, rstd = around.layernorm(h.detach(), w.detach(), b.detach(), 1e-3)
    dx, dw, db = around.layernorm_grad(dy, h.detach(), w.detach(), mean, rstd, dh)
    for got, want in ((y64, y.detach()), (dx, h.grad), (dw, w.grad), (db, b.grad)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("ordered", [False, True])
def test_adapters_and_gradients(ordered):
    rng = np.random.default_rng(2)
    M, n, h, r, o = 9, 3, 6, 4, 5
    ids = np.array([0, 0, 2, 2, 2, 2, -1, -1, -1] if not ordered else [2, -1, 0, 2, -1, 2, 0, 2, -1])
    order, offsets = around.route(ids, n)
    x, l1, l2, base, base_x, dy = (torch.from_numpy(rng.standard_normal(s)) for s in
                                   ((M, h), (n, h, r), (n, r, o), (M, o), (M, h), (M, o)))
    s = torch.from_numpy(rng.random(n) + 0.5)
    x, l1, l2 = (t.requires_grad_() for t in (x, l1, l2))
    y = base.clone()
    t = torch.zeros(M, r, dtype=torch.float64)
    for m, a in enumerate(ids):  # row by row
        if a >= 0:
            t[m] = (x[m] @ l1[a]).detach()
            y[m] = y[m] + s[a] * (x[m] @ l1[a] @ l2[a])
    (torch.sum(y * dy) + torch.sum(x * base_x)).backward()
    listed = order if ordered else None
    arrays = [v.detach().numpy() for v in (x, l1, l2, s)]
    y64, t64, S, Q, R = around.adapters_fwd(*arrays, listed, offsets, base.numpy())
    (dx, Sx), (dl1, S1), (dl2, S2) = around.adapters_bwd(dy, arrays[0], t64, *arrays[1:], listed, offsets, base_x.numpy())
    for got, want in ((y64, y.detach()), (t64, t), (dx, x.grad), (dl1, l1.grad), (dl2, l2.grad)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)
    # the sums of magnitudes bound the sums
    for big, small in ((S, y64 - base.numpy()), (Q, t64), (R, S), (Sx, dx - base_x.numpy()), (S1, dl1), (S2, dl2)):
        assert np.all(big >= np.abs(small) * (1 - 1e-12))
    # an adapter without rows learns nothing, a row without one is left alone
    assert not dl1[1].any() and not dl2[1].any() and np.array_equal(y64[ids < 0], base.numpy()[ids < 0])
