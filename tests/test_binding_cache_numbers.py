"""Numbers that are others once they are the library's (float32 and int64) are refused, not taken for what they become
(on the CPU, with stand-ins for device tensors)."""

import pytest

from quantized_prefill_gemm_amd import binding as B
from test_binding_cache import attend, pytestmark, run, tree  # noqa: F401


@pytest.mark.parametrize("call", [attend, tree])
def test_caps(run, call):  # noqa: F811
    for cap in (0, 0.0, 1e-30, 30, 30.0):
        assert run(lambda: call(cap=cap)) == "called", cap
    for cap in (1e-46, 5e-324, -1e-50):                    # 0 in float32, which means no cap
        assert run(lambda: call(cap=cap)) == B.QPG_EINVAL, cap


@pytest.mark.parametrize("call", [attend, tree])
def test_windows(run, call):  # noqa: F811
    for window in (0, 1, 1 << 30, (1 << 63) - 1):
        assert run(lambda: call(window=window)) == "called", window
    for window in (1 << 63, 1 << 64, (1 << 64) + 5, -(1 << 64) + 7):
        assert run(lambda: call(window=window)) == B.QPG_EINVAL, window
