"""The entry points that zero the rows no slot has refuse what their siblings refuse (no kernel is
launched here)."""
import os

import pytest

from quantized_prefill_gemm_amd import binding as B
from test_abi_mx import CALLS, EDEVICE

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libqpg.so not built")
SIBLINGS = [c for c in CALLS if c[0] in ("experts_gather", "experts_combine_grad")]


@pytest.mark.parametrize("name,args,bad", SIBLINGS, ids=[c[0] for c in SIBLINGS])
def test_refusals(name, args, bad):
    import torch
    f = getattr(B.lib(), name + "_zero")
    for at, value, status in bad:
        a = list(args)
        a[at] = value
        assert f(*a) == status, (at, value)
    if not torch.cuda.device_count():
        assert f(*args) == EDEVICE
