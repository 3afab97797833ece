"""Caps so large that twice the cap, in powers of two, is no f32 are refused (no kernel is launched here): a score of
their size would become an infinity of the other sign."""
import pytest
import torch

from test_abi_cache import EDEVICE, EINVAL, NAMES, call, pytestmark as built

pytestmark = [built, pytest.mark.skipif(torch.cuda.device_count() > 0, reason="calls that pass would run on addresses that are none")]


@pytest.mark.parametrize("name", NAMES[1:])
def test_largest_caps(name):
    largest = 3.4028234e38 / 3
    for cap, status in ((1e30, EDEVICE), (0.999 * largest, EDEVICE), (1.001 * largest, EINVAL), (2e38, EINVAL)):
        assert call(name, scores={"cap": cap}) == status, cap
