"""The largest launches of the attentions over a paged cache (no kernel is launched here): those of 2^32 threads and
more are refused by their arguments, whatever the size of the form's workgroups."""
import pytest
import torch

from quantized_prefill_gemm_amd import binding as B
from test_abi_cache import A, EDEVICE, EINVAL, call, pytestmark as built

pytestmark = [built, pytest.mark.skipif(torch.cuda.device_count() > 0, reason="calls that pass would run on addresses that are none")]

# T, heads, cache heads, dim, width, slots of 128, 64 and 32 columns less B, threads of a workgroup
CASES = [(32, 1024, 8, 128, 1, 32, 512),          # tiles of 128 columns, two groups of four waves
         (24, 1024, 8, 128, 1, 48, 512),          # of 64, four groups of two waves
         (8, 64, 8, 128, 1, 2, 256)]              # of 32, four groups of one


@pytest.mark.parametrize("T,heads,kv,dim,width,slots,threads", CASES)
def test_threads_of_a_launch(T, heads, kv, dim, width, slots, threads):
    cache = {"heads": kv, "dim": dim, "k_stride": kv * 16 * dim, "v_stride": kv * 16 * dim}
    most = min(2 ** 32 // threads, 2 ** 24) // kv             # slots that are one too many
    for more, status in ((-1, EDEVICE), (0, EINVAL), (1, EINVAL)):
        b = most + more - slots
        if b > 2 ** 20:                                       # refused by itself, or within all limits
            b, status = 2 ** 20, EDEVICE
        got = call("cache_attention", cache=cache, batch={"T": T, "B": b, "width": width}, args=[A, heads, A, 2, A, 0])
        assert got == status, (b, more)
        got = call("cache_attention_tree", cache=cache, batch={"T": T, "B": b, "width": width}, args=[A, heads, A, 2, A, A, 2, A, 0])
        assert got == status, (b, more)
