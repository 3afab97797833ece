"""Host-side checks of the MXFP4 and expert entry points (no kernel is launched here): sizes, and
the status of every kind of bad argument, before anything reaches a device."""
import ctypes
import os

import pytest

import mx_ref as R
from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libqpg.so not built")
EINVAL, EALIGN, EDEVICE = -1, -2, -4
A = 1 << 20                                   # a 16-byte aligned address that is never touched


def test_sizes():
    L = B.lib()
    assert L.qpg_mxfp4_bytes(1, 32) == 17 and L.qpg_mxfp4_bytes(7, 96) == 7 * 51
    assert L.qpg_mxfp4_bytes(512, 4096) == 512 * 4096 * 17 // 32
    assert L.qpg_mxfp4_bytes(2 ** 30 - 64, 32) == (2 ** 30 - 64) * 17
    for rows, K in ((0, 32), (-1, 32), (1, 0), (1, 16), (1, 48), (2 ** 31, 32), (1, 2 ** 24 + 32), (2 ** 15, 2 ** 20), (2 ** 30 - 63, 32),
                    (2 ** 30, 32)):
        assert L.qpg_mxfp4_bytes(rows, K) == 0, (rows, K)
    assert L.qpg_experts_sort_bytes(16, 8) == 0
    assert L.qpg_experts_sort_bytes(2 ** 20, 8) > 0
    assert L.qpg_experts_sort_bytes(2 ** 30, 1024) > 0
    for S, E in ((0, 8), (-1, 8), (2 ** 31, 8), (2 ** 30 + 1, 8), (16, 0), (16, 1025), (2 ** 20, 1025)):
        assert L.qpg_experts_sort_bytes(S, E) == 0
    assert len(R.pack(*R.encode(__import__("numpy").ones((7, 96))))) == B.mxfp4_bytes(7, 96)


# (function, valid arguments, [(position, bad value, status)]): every bad value alone must give its status
CALLS = [
    ("quantize_mxfp4", [A, 0, A, 4, 64, 0],
     [(0, 0, EINVAL), (2, 0, EINVAL), (1, 3, EINVAL), (1, -1, EINVAL), (3, 0, EINVAL), (3, 2 ** 31, EINVAL),
      (4, 48, EINVAL), (4, 0, EINVAL), (4, 2 ** 25, EINVAL), (0, A + 4, EALIGN), (2, A + 8, EALIGN)]),
    ("dequantize_mxfp4", [A, A, 1, 4, 64, 0],
     [(0, 0, EINVAL), (1, 0, EINVAL), (2, 7, EINVAL), (3, -4, EINVAL), (4, 33, EINVAL), (0, A + 1, EALIGN),
      (1, A + 2, EALIGN)]),
    ("mmq_mxfp4_mx", [A, A, A, 0, 4, 8, 64, 0],
     [(0, 0, EINVAL), (1, 0, EINVAL), (2, 0, EINVAL), (3, 9, EINVAL), (4, 0, EINVAL), (5, 0, EINVAL),
      (6, 40, EINVAL), (5, 2 ** 31, EINVAL), (0, A + 8, EALIGN), (1, A + 8, EALIGN), (2, A + 2, EALIGN)]),
    ("mmq_mxfp4_mx", [A, A, A, 2, 2 ** 28, 8, 64, 0], [(5, 2 ** 28, EINVAL), (4, 2 ** 30, EINVAL), (2, A + 1, EALIGN)]),
    ("mmq_mxfp4", [A, A, 2, A, 1, 4, 8, 64, A, 0],
     [(0, 0, EINVAL), (1, 0, EINVAL), (3, 0, EINVAL), (8, 0, EINVAL), (2, 5, EINVAL), (4, 5, EINVAL), (5, 0, EINVAL),
      (6, 0, EINVAL), (7, 31, EINVAL), (0, A + 4, EALIGN), (1, A + 4, EALIGN), (3, A + 1, EALIGN), (8, A + 4, EALIGN)]),
    ("experts_sort", [A, 8, 100, 8, A, A, A, 0, 0],
     [(0, 0, EINVAL), (1, 2, EINVAL), (2, 0, EINVAL), (2, 2 ** 31, EINVAL), (2, 2 ** 30 + 1, EINVAL), (3, 0, EINVAL), (3, 1025, EINVAL),
      (4, 0, EINVAL), (5, 0, EINVAL), (6, 0, EINVAL), (2, 2 ** 20, EINVAL), (0, A + 4, EALIGN), (4, A + 2, EALIGN),
      (5, A + 1, EALIGN), (6, A + 2, EALIGN), (7, A + 2, EALIGN)]),
    ("mmq_mxfp4_experts", [A, A, 4, A, A, 2, A, 0, 8, 3, 16, 64, 0],
     [(0, 0, EINVAL), (1, 0, EINVAL), (3, 0, EINVAL), (4, 0, EINVAL), (6, 0, EINVAL), (7, 4, EINVAL), (2, 0, EINVAL),
      (5, 0, EINVAL), (8, 0, EINVAL), (9, 0, EINVAL), (9, 1025, EINVAL), (10, 0, EINVAL), (11, 16, EINVAL),
      (10, 2 ** 30, EINVAL), (0, A + 4, EALIGN), (1, A + 4, EALIGN), (3, A + 2, EALIGN), (4, A + 2, EALIGN),
      (6, A + 2, EALIGN)]),
    # slots past 2^30 (a row and a tile's height past an int), and more tiles than an int counts
    ("mmq_mxfp4_experts", [A, A, 4, A, A, 2 ** 29, A, 0, 2 ** 30, 1, 16, 64, 0],
     [(8, 2 ** 30 + 1, EINVAL), (8, 2 ** 31 - 1, EINVAL), (9, 32, EINVAL)]),
    ("experts_gather", [A, 2, A, A, 4, 2, 64, 0],
     [(0, 0, EINVAL), (2, 0, EINVAL), (3, 0, EINVAL), (1, 3, EINVAL), (4, 0, EINVAL), (5, 0, EINVAL), (6, 0, EINVAL),
      (5, 2 ** 30, EINVAL), (5, 2 ** 28 + 1, EINVAL), (6, 2 ** 28, EINVAL), (4, 2 ** 24, EINVAL), (0, A + 1, EALIGN), (2, A + 2, EALIGN), (3, A + 1, EALIGN)]),
    ("experts_combine", [A, 0, A, A, A, 2, 4, 2, 64, 0],
     [(0, 0, EINVAL), (2, 0, EINVAL), (4, 0, EINVAL), (1, 3, EINVAL), (5, 3, EINVAL), (6, 0, EINVAL), (7, 0, EINVAL),
      (8, 0, EINVAL), (0, A + 2, EALIGN), (2, A + 1, EALIGN), (3, A + 2, EALIGN), (4, A + 1, EALIGN)]),
    ("experts_combine_grad", [A, 0, A, 2, A, A, A, A, 4, 2, 64, 0],
     [(0, 0, EINVAL), (2, 0, EINVAL), (4, 0, EINVAL), (5, 0, EINVAL), (6, 0, EINVAL), (7, 0, EINVAL), (1, 3, EINVAL),
      (3, 3, EINVAL), (8, 0, EINVAL), (9, 0, EINVAL), (10, 0, EINVAL), (0, A + 2, EALIGN), (2, A + 1, EALIGN),
      (6, A + 1, EALIGN), (5, A + 2, EALIGN), (7, A + 2, EALIGN)]),
]


@pytest.mark.parametrize("name,args,bad", CALLS, ids=[f"{c[0]}-{i}" for i, c in enumerate(CALLS)])
def test_bad_arguments(name, args, bad):
    f = getattr(B.lib(), name)
    for at, value, status in bad:
        a = list(args)
        a[at] = value
        assert f(*a) == status, (name, at, value)


@pytest.mark.parametrize("name,args,bad", CALLS, ids=[f"{c[0]}-{i}" for i, c in enumerate(CALLS)])
def test_valid_arguments_need_a_device(name, args, bad):
    import torch
    if torch.cuda.device_count():
        pytest.skip("a GPU is here: the call would run on addresses that are none")
    assert getattr(B.lib(), name)(*args) == EDEVICE


def test_binding_refuses_host_tensors():
    import torch
    x, ids = torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int64)
    u8, i32 = torch.zeros(4096, dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: B.quantize_mxfp4(x), lambda: B.dequantize_mxfp4(u8, 4, 64), lambda: B.mmq_mxfp4(u8, x, 8),
                 lambda: B.mmq_mxfp4_mx(u8, u8, 4, 8, 64), lambda: B.experts_sort(ids, 4),
                 lambda: B.mmq_mxfp4_experts(u8, u8, 4, i32, None, 1, 2, 8, 64), lambda: B.experts_gather(x, i32),
                 lambda: B.experts_gather_grad(x, i32), lambda: B.experts_combine(x, i32, x),
                 lambda: B.experts_combine_grad(x, x, i32, x)):
        with pytest.raises(B.QPGError) as e:
            call()
        assert e.value.status == EINVAL
