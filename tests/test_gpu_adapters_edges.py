"""The adapters at the end of fp32's range (needs an MI355X)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

try:
    import quantized_lora_fine_amd  # noqa: F401
except ImportError as exc:
    if torch.cuda.is_available():
        raise
    pytest.skip(f"libnf4lora.so not loaded: {exc}", allow_module_level=True)

from tests.test_gpu_adapters import Case  # noqa: E402

BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127
OVER = 1.5 * 2.0 ** 119  # BF16_MAX + OVER is an fp32 value that bf16 rounds to an infinity


@pytest.mark.parametrize("counts,r", [([1], 16), ([2, 1], 8), ([40], 16), ([300, 0, 200], 16), ([300, 200], 72),
                                      ([3000, 2000], 40)], ids=str)
def test_values_past_the_largest_bf16(counts, r):
    # T and G between the largest bf16 and the largest fp32, of either sign, and products with them that are in range
    c = Case(41, counts, 1, 528, 656, r, True)
    sign = torch.where(torch.arange(c.M) % 2 == 0, 1.0, -1.0)[:, None]
    tops = torch.tensor([BF16_MAX, OVER]) * sign
    c.L1 = (c.L1.float() * 2.0 ** -10).to(torch.bfloat16)
    c.L2 = (c.L2.float() * 2.0 ** -10).to(torch.bfloat16)
    c.s = c.s * 2.0 ** -20
    small = Case(41, counts, 1, 528, 656, r, True)
    # forward: T[m] = +-(BF16_MAX + OVER) in every place
    l1, x = c.L1.clone(), c.X.clone()
    c.L1 = torch.zeros_like(l1)
    c.L1[:, 3], c.L1[:, 300] = 1, 1
    c.X = torch.zeros_like(x)
    c.X[:, [3, 300]] = tops.to(torch.bfloat16)
    c.x64 = c.X.double().numpy()
    Y, T = c.check_fwd()
    listed = torch.from_numpy(~c.none)
    assert torch.all(T.cpu()[listed].abs() == BF16_MAX + OVER) and torch.isfinite(Y.cpu()[listed]).all()
    # backward: G[m] likewise; X and T small, so that the sums over rows are in range
    c.L1 = l1
    c.X = (small.X.float() * 2.0 ** -30).to(torch.bfloat16)
    c.x64 = c.X.double().numpy()
    c.T = small.T * 2.0 ** -30
    c.L2 = torch.zeros_like(c.L2)
    c.L2[:, :, 5], c.L2[:, :, 600] = 1, 1
    c.dY = torch.zeros_like(c.dY)
    c.dY[:, [5, 600]] = tops.to(torch.bfloat16)
    dX, dL1, dL2 = c.check_bwd()
    assert torch.isfinite(dX.cpu()[listed]).all() and torch.isfinite(dL1).all() and torch.isfinite(dL2).all()
