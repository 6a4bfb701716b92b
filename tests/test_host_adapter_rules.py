"""The adapters' tile rules at sizes that were measured with both kinds of tile (no GPU)."""
import os

import pytest

from tests.test_host_sanitized import COMMON, CSRC, GXX, HOST, ROCM, SAN, SAN_ENV, _run


@pytest.mark.skipif(GXX is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"),
                    reason="needs g++ and the HIP host runtime")
def test_measured_sizes_get_the_faster_tiles(tmp_path):
    exe = str(tmp_path / "adapter_rule_units")
    _run([GXX, *COMMON, *SAN, "-o", exe, os.path.join(HOST, "adapter_rule_units.cpp"), os.path.join(CSRC, "plan.cpp")])
    assert "adapter rule units: ok" in _run([exe], env={**os.environ, **SAN_ENV})
