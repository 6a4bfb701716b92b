"""What the adapters' gradients ask of their workspace (no GPU): sums of an adapter whose rows are one item go straight to
the results, so a pool of many adapters with few rows each costs its rows' own space alone."""
import os

import pytest

from tests.test_host_sanitized import COMMON, CSRC, GXX, HOST, ROCM, SAN, SAN_ENV, _run

nf4 = pytest.importorskip("quantized_lora_fine_amd", reason="libnf4lora.so not built")


def backward(M, n, o=4096, h=4096, r=16):
    return nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, M, o, h, n, r)


def own(M, o, r):
    """T and G in three bf16 parts (the rank in runs of 64), G, and G's sums in splits of 256 of the contraction."""
    runs = -(-r // 64)
    rp = 16 if r <= 16 else 32 if r <= 32 else 64
    return 512 + 2 * M * runs * 3 * rp * 2 + M * r * 4 * (1 + -(-o // 256))


@pytest.mark.parametrize("M,n", [(64, 512), (3, 4096), (64, 65), (1, 4096)])
def test_rows_that_are_one_item_need_no_sums(M, n):
    # an item is of 64 rows or more: none has a second one
    assert backward(M, n) <= own(M, 4096, 16)


@pytest.mark.parametrize("M,n,r", [(4096, 4096, 16), (1025, 512, 16), (2048, 1024, 64), (8192, 300, 128)])
def test_sums_go_by_the_rows(M, n, r):
    # less than 2 M / 64 items of adapters that have several, however many adapters there are
    sums = 2 * M // 64 * r * (4096 + 4096) * 4
    assert backward(M, n, r=r) <= own(M, 4096, r) + sums
    assert backward(M, 4096, r=r) <= own(M, 4096, r) + sums


@pytest.mark.skipif(GXX is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"),
                    reason="needs g++ and the HIP host runtime")
def test_space_units_sanitized(tmp_path):
    exe = str(tmp_path / "adapter_space_units")
    _run([GXX, *COMMON, *SAN, "-o", exe, os.path.join(HOST, "adapter_space_units.cpp"), os.path.join(CSRC, "plan.cpp")])
    assert "adapter space units: ok" in _run([exe], env={**os.environ, **SAN_ENV})
