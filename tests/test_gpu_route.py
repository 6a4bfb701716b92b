"""Rows sorted by id against a plain sort: whole numbers, all equal (needs an MI355X)."""
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

DEV = "cuda"


def check(ids, n):
    order, offsets = nf4.route(torch.from_numpy(ids).to(DEV), n)
    want = around.route(ids, n)
    assert np.array_equal(offsets.cpu().numpy(), want[1])
    assert np.array_equal(order.cpu().numpy(), want[0])


ROWS = [0, 1, 2, 63, 64, 65, 511, 512, 513, 1536, 1537, 8191, 8192, 8193, 20000, 70001]


@pytest.mark.parametrize("n", [1, 2, 3, 31, 64, 255, 256, 1023, 1024, 4095, 4096])
@pytest.mark.parametrize("M", ROWS)
def test_route(M, n):
    rng = np.random.default_rng(M * 7 + n)
    check(rng.integers(0, n, M).astype(np.int32), n)


@pytest.mark.parametrize("M", [64, 1000, 30000])
def test_route_uneven(M):
    rng = np.random.default_rng(M)
    check(np.zeros(M, np.int32), 5)                                     # one id has them all
    check(np.full(M, 4, np.int32), 5)
    check(np.full(M, -1, np.int32), 5)                                  # none has an id
    check(np.repeat(np.arange(10, dtype=np.int32)[::-1], M // 10 + 1)[:M].copy(), 10)
    check(np.where(rng.random(M) < 0.9, 7, rng.integers(0, 300, M)).astype(np.int32), 300)
    ids = rng.integers(-3, 8, M).astype(np.int32)                       # rows without one, in between
    ids[rng.integers(0, M, 5)] = [2**31 - 1, -2**31, 8, 5, 6]
    check(ids, 5)


def test_route_many_rows():
    # runs longer than 512 rows, more of them than a wave reads at once
    rng = np.random.default_rng(3)
    M, n = 3_000_001, 700
    ids = rng.integers(-1, n + 1, M).astype(np.int32)
    order, offsets = nf4.route(torch.from_numpy(ids).to(DEV), n)
    key = np.where((ids < 0) | (ids >= n), n, ids)
    assert np.array_equal(order.cpu().numpy(), np.argsort(key, kind="stable").astype(np.int32))
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(n + 1)).astype(np.int32))


@pytest.mark.parametrize("M", [200, 20000])
def test_route_captured_and_replayed(M):
    rng = np.random.default_rng(M)
    n = 40
    ids = torch.from_numpy(rng.integers(0, n, M).astype(np.int32)).to(DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        nf4.route(ids, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        order, offsets = nf4.route(ids, n)
    for _ in range(3):
        new = rng.integers(-1, n, M).astype(np.int32)
        ids.copy_(torch.from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        want = around.route(new, n)
        assert np.array_equal(order.cpu().numpy(), want[0]) and np.array_equal(offsets.cpu().numpy(), want[1])


def test_route_for_the_grouped_product():
    # what it is for: rows sorted by expert, the product grouped by them, the results back in their places
    rng = np.random.default_rng(4)
    M, E, o, h = 90, 5, 144, 272
    ids = torch.from_numpy(rng.integers(0, E, M).astype(np.int32)).to(DEV)
    X = torch.from_numpy(rng.standard_normal((M, h)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    W = [nf4.fp8_quantize(torch.from_numpy(rng.standard_normal((o, h)).astype(np.float32)).to(DEV), 128)
         for _ in range(E)]
    order, offsets = nf4.route(ids, E)
    A, s = nf4.fp8_quantize(X[order.long()].contiguous())
    C = nf4.fp8_matmul_grouped(A, s, torch.stack([w.view(torch.uint8) for w, _ in W]).view(torch.float8_e4m3fn),
                               torch.stack([v for _, v in W]), offsets)
    for m in range(M):
        a, sa = nf4.fp8_quantize(X[order[m].long()][None].contiguous())
        e = int(ids[order[m].long()])
        one = nf4.fp8_dequantize(a, sa) @ nf4.fp8_dequantize(*W[e], 128).t()
        size = nf4.fp8_dequantize(a, sa).abs() @ nf4.fp8_dequantize(*W[e], 128).abs().t()
        # the 8-bit product's own bound: bf16, and 2^-13 of the largest of each 8 terms
        assert torch.all((C[m].float() - one[0]).abs() <= one[0].abs() * 2.0 ** -8 + size[0] * 2.0 ** -11)


def test_route_refuses():
    ids = torch.zeros(8, dtype=torch.int32, device=DEV)
    order, offsets = torch.empty_like(ids), torch.empty(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: nf4.route(ids.long(), 3), lambda: nf4.route(ids[None], 3), lambda: nf4.route(ids[::2], 3),
                lambda: nf4.route(ids, 3, outs=(order[:4], offsets)), lambda: nf4.route(ids, 4, outs=(order, offsets)),
                lambda: nf4.route(ids, 3, outs=(order.float(), offsets)), lambda: nf4.route(ids.cpu(), 3)):
        with pytest.raises(ValueError):
            bad()
    for n in (0, -1, 4097):
        with pytest.raises(nf4.NF4Error):
            nf4.route(ids, n)
    with pytest.raises(nf4.NF4Error):
        nf4.route(ids, 3, outs=(ids, offsets))
    with pytest.raises(nf4.NF4Error):
        nf4.route(torch.zeros(20000, dtype=torch.int32, device=DEV), 3,
                  ws=torch.empty(16, dtype=torch.uint8, device=DEV))
