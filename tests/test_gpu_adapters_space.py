"""The adapters' gradients in a workspace of just the bytes they ask for, of pools that mix adapters of no row, of one item
and of several (needs an MI355X)."""
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

from tests.test_gpu_adapters import Case, on  # noqa: E402
from tests.test_gpu_fp8 import DEV, bits  # noqa: E402

POOLS = {"one among few": [3000], "every kind": [0, 1, 130, 0, 64, 65, 900, 2, 0, 129, 1500, 1],
         "big ones last": [2] * 100 + [0] * 40 + [700, 1300], "big ones first": [1300, 700] + [0] * 90 + [1] * 50,
         "no second item": [1] * 64 + [0] * 70, "just over": [65] * 40, "many": ([3, 0, 1] * 60 + [200]) * 5}


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("h,o,r", [(272, 144, 8), (1040, 528, 72)])
@pytest.mark.parametrize("pool", POOLS)
def test_gradients_in_just_their_workspace(pool, h, o, r, fmt):
    c = Case(51 + len(pool), POOLS[pool], 4, h, o, r, True, fmt)
    dX, dL1, dL2 = c.check_bwd()
    need = nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, c.M, o, h, c.n, r)
    room = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device=DEV)
    some = ~c.none
    got = c.bwd(ws=room[:need])
    assert np.array_equal(bits(got[0])[some], bits(dX)[some])
    assert torch.equal(got[1], dL1) and torch.equal(got[2], dL2)
    assert torch.all(room[need:] == 0xA5)


@pytest.mark.parametrize("pool", ["every kind", "big ones last", "many"])
def test_offsets_that_do_not_ascend_stay_in_the_workspace(pool):
    c = Case(52, POOLS[pool], 10, 272, 144, 16, True)
    M, n, big = c.M, c.n, 2 ** 31 - 1
    off, order = c.lists()
    need = nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, M, c.o, c.h, n, c.r)
    room = torch.full((need + (32 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    g1 = torch.full((n + 2, c.h, c.r), 0.375, device=DEV)
    g2 = torch.full((n + 2, c.r, c.o), 0.375, device=DEV)
    X, L1, L2, s, dY, T = (on(v) for v in (c.X, c.L1, c.L2, c.s, c.dY, c.T))
    end = off.tolist()
    for offs in (end[::-1], [0, M] * (n + 1), [big, -big] * (n + 1), [M // 2, M, 0] * (n + 1),
                 [0] * (n // 2) + [M, 0] * n):
        o = torch.tensor(offs[:n + 1], dtype=torch.int32, device=DEV)
        for orders in (order, None):
            nf4.adapters_bwd(dY, X, T, L1, L2, s, o, orders, dL1=g1[1:1 + n], dL2=g2[1:1 + n], ws=room[:need])
            torch.cuda.synchronize()
            assert torch.all(room[need:] == 0xA5)
            for g in (g1, g2):
                assert torch.all(g[0] == 0.375) and torch.all(g[-1] == 0.375)
