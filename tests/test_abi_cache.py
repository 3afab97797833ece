"""Host-side checks of the operators over a paged cache (no kernel is launched here): workspace sizes, and the
status of every kind of bad argument, before anything reaches a device."""
import ctypes
import math
import os

import pytest

from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libqpg.so not built")
EINVAL, EALIGN, EDEVICE = -1, -2, -4
A = 1 << 20                                   # a 16-byte aligned address that is never touched

CACHE = {"k": A, "v": A, "type": 1, "pages": 10, "heads": 2, "page": 16, "dim": 64, "k_stride": 2048, "v_stride": 2048}
BATCH = {"table": A, "lens": A, "offsets": A, "B": 3, "width": 4, "T": 5}
SCORES = {"scale": 0.125, "cap": 0.0, "slopes": 0, "window": 0, "prefix": 0}
APPEND = [A, A, A, 0, 512, 256, 256, 4, 0, A, 64, 1, A, A, 1e-6, A, 0]
ATTENTION = [A, 4, A, 2, A, 0]
TREE = [A, 4, A, 2, A, A, 2, A, 0]


def call(name, cache=None, batch=None, scores=None, args=None):
    c, b = B._Cache(**{**CACHE, **(cache or {})}), B._Batch(**{**BATCH, **(batch or {})})
    first = [ctypes.byref(c), ctypes.byref(b)]
    if name != "cache_append":
        first.append(ctypes.byref(B._Scores(**{**SCORES, **(scores or {})})))
    return getattr(B.lib(), name)(*first, *(args or {"cache_append": APPEND, "cache_attention": ATTENTION}.get(name, TREE)))


NAMES = ("cache_append", "cache_attention", "cache_attention_tree")
BAD_CACHE = [({"k": 0}, EINVAL), ({"v": 0}, EINVAL), ({"type": 0}, EINVAL), ({"type": 3}, EINVAL), ({"type": -1}, EINVAL),
             ({"pages": 0}, EINVAL), ({"pages": 2 ** 31}, EINVAL), ({"heads": 0}, EINVAL), ({"heads": 3}, EINVAL),
             ({"heads": 8192}, EINVAL), ({"page": 8}, EINVAL), ({"page": 48}, EINVAL), ({"page": 0}, EINVAL), ({"page": 512}, EINVAL),
             ({"dim": 0}, EINVAL), ({"dim": 12}, EINVAL), ({"dim": 264}, EINVAL), ({"dim": -8}, EINVAL), ({"k_stride": 2040}, EINVAL),
             ({"v_stride": 2040}, EINVAL), ({"k_stride": 2052}, EINVAL), ({"v_stride": 2 ** 41}, EINVAL), ({"k": A + 8}, EALIGN),
             ({"v": A + 2}, EALIGN)]
BAD_BATCH = [({"table": 0}, EINVAL), ({"lens": 0}, EINVAL), ({"offsets": 0}, EINVAL), ({"B": 0}, EINVAL), ({"B": 2 ** 20 + 1}, EINVAL),
             ({"width": 0}, EINVAL), ({"width": 2 ** 26 + 1}, EINVAL), ({"T": 0}, EINVAL), ({"T": 2 ** 24}, EINVAL),
             ({"table": A + 2}, EALIGN), ({"lens": A + 1}, EALIGN), ({"offsets": A + 2}, EALIGN)]
BAD_SCORES = [({"scale": 0.0}, EINVAL), ({"scale": -1.0}, EINVAL), ({"scale": math.nan}, EINVAL), ({"scale": math.inf}, EINVAL),
              ({"cap": -1.0}, EINVAL), ({"cap": math.nan}, EINVAL), ({"cap": math.inf}, EINVAL), ({"scale": 3e38}, EINVAL), ({"cap": 3e38}, EINVAL), ({"cap": 1e-39}, EINVAL),
              ({"scale": 1e20, "cap": 1e-20}, EINVAL), ({"window": -1}, EINVAL),
              ({"slopes": A + 2}, EALIGN)]


@pytest.mark.parametrize("name", NAMES)
def test_bad_caches_and_batches(name):
    for cache, status in BAD_CACHE:
        assert call(name, cache=cache) == status, cache
    for batch, status in BAD_BATCH:
        assert call(name, batch=batch) == status, batch
    f = getattr(B.lib(), name)
    rest = {"cache_append": APPEND, "cache_attention": ATTENTION}.get(name, TREE)
    c, b, s = (ctypes.byref(x) for x in (B._Cache(**CACHE), B._Batch(**BATCH), B._Scores(**SCORES)))
    mid = [] if name == "cache_append" else [s]
    assert f(None, b, *mid, *rest) == EINVAL and f(c, None, *mid, *rest) == EINVAL
    if mid:
        assert f(c, b, None, *rest) == EINVAL


@pytest.mark.parametrize("name", NAMES[1:])
def test_bad_scores(name):
    for scores, status in BAD_SCORES:
        assert call(name, scores=scores) == status, scores
    assert call(name, scores={"prefix": A + 2}) == (EALIGN if name == "cache_attention" else EINVAL)
    assert call("cache_attention_tree", scores={"prefix": A}) == EINVAL


# (function, arguments behind the structures, [(position, bad value, status)])
CALLS = [
    ("cache_append", APPEND,
     [(0, 0, EINVAL), (1, 0, EINVAL), (2, 0, EINVAL), (3, 3, EINVAL), (3, -1, EINVAL), (4, 248, EINVAL), (5, 120, EINVAL), (6, 127, EINVAL),
      (4, 2 ** 41, EINVAL), (5, -512, EINVAL), (7, 3, EINVAL), (7, 1, EINVAL), (7, -2, EINVAL), (7, 8192, EINVAL), (9, 0, EINVAL),
      (10, 72, EINVAL), (10, 12, EINVAL), (10, -8, EINVAL), (14, -1.0, EINVAL), (14, math.nan, EINVAL), (15, 0, EINVAL),
      (0, A + 2, EALIGN), (1, A + 1, EALIGN), (2, A + 2, EALIGN), (8, A + 2, EALIGN), (9, A + 2, EALIGN), (12, A + 1, EALIGN),
      (13, A + 2, EALIGN), (15, A + 8, EALIGN)]),
    ("cache_attention", ATTENTION,
     [(0, 0, EINVAL), (1, 0, EINVAL), (1, 3, EINVAL), (1, 1, EINVAL), (1, 8192, EINVAL), (2, 0, EINVAL), (3, 3, EINVAL), (0, A + 8, EALIGN),
      (2, A + 4, EALIGN), (4, A + 8, EALIGN)]),
    ("cache_attention_tree", TREE,
     [(0, 0, EINVAL), (1, 0, EINVAL), (2, 0, EINVAL), (3, 0, EINVAL), (3, 1025, EINVAL), (4, 0, EINVAL), (5, 0, EINVAL), (6, 7, EINVAL),
      (0, A + 8, EALIGN), (2, A + 4, EALIGN), (4, A + 2, EALIGN), (5, A + 8, EALIGN), (7, A + 4, EALIGN)]),
]


@pytest.mark.parametrize("name,args,bad", CALLS, ids=[c[0] for c in CALLS])
def test_bad_arguments(name, args, bad):
    for at, value, status in bad:
        a = list(args)
        a[at] = value
        assert call(name, args=a) == status, (name, at, value)


def test_launches_that_are_too_large():
    """2^24 workgroups and more (empty ones among them) are refused; a workspace that is needed has to be there."""
    many = {"heads": 4096, "k_stride": 2 ** 30, "v_stride": 2 ** 30}
    args = [A, 4096, A, 2, A, 0]
    assert call("cache_attention", cache=many, batch={"B": 4096}, args=args) == EINVAL
    assert call("cache_attention", batch={"T": 2 ** 24 - 1}, args=[A, 128, A, 2, A, 0]) == EINVAL         # T * heads >= 2^31
    assert call("cache_attention", batch={"T": 1, "B": 1, "width": 1024}, args=[A, 4, A, 2, 0, 0]) == EINVAL


def test_workspace_sizes():
    f = B.lib().qpg_cache_attention_bytes
    assert f(1, 1, 32, 32, 128, 1024) % (32 * (128 * 4 + 8)) == 0 and f(1, 1, 32, 32, 128, 1024) > 0
    assert f(8192, 1, 32, 8, 128, 8192) == 0                       # tiles enough without
    assert f(1, 1, 32, 32, 128, 100) == 0                          # keys too few to split
    for bad in ((0, 1, 4, 2, 64, 4096), (1, 0, 4, 2, 64, 4096), (1, 1, 3, 2, 64, 4096), (1, 1, 4, 0, 64, 4096), (1, 1, 4, 2, 60, 4096),
                (1, 1, 4, 2, 264, 4096), (1, 1, 4, 2, 64, 0), (1, 1, 4, 2, 64, 2 ** 31), (2 ** 24, 1, 4, 2, 64, 4096)):
        assert f(*bad) == 0, bad
    assert B.cache_attention_bytes(1, 1, 32, 32, 128, 1024) == f(1, 1, 32, 32, 128, 1024)


@pytest.mark.parametrize("name", NAMES)
def test_valid_arguments_need_a_device(name):
    import torch
    if torch.cuda.device_count():
        pytest.skip("a GPU is here: the call would run on addresses that are none")
    assert call(name) == EDEVICE
    if name == "cache_append":
        # keys and values alone; no rotation, no norms; one row of any stride
        args = list(APPEND)
        for at, value in ((0, 0), (7, 0), (15, 0), (9, 0), (10, 0), (12, 0), (13, 0)):
            args[at] = value
        assert call(name, args=args) == EDEVICE
        assert call(name, batch={"T": 1}, args=[A, A, A, 0, 0, 0, 0, *APPEND[7:]]) == EDEVICE
