"""Infinite values in the cache: a row that sees one is infinite there, of its sign, whatever its share; one that sees both
signs or a NaN is NaN; every other result is as if they were not there. In each form of the launch, with shares of one
piece and of several, shares that are 0 in 16 and in 32 bits, and maxima that leave them far behind."""
import math

import pytest
import torch

import cache_ref as R
from test_gpu_cache_forms_masks import FORMS, TYPES, compare, one_head

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("form", FORMS)
def test_every_form(form, value):
    for kind, y in TYPES:
        assert compare(form, kind, y, odd=((1, value), (40, value), (100, value), (299, -value))) > 0
    assert compare(form, "f16", "f32", odd=((9, value), (31, -value)), tree="mixed") > 0


def steep(new, lens, heads, kv, dim, page, kind, y, step, odd, window=0):
    """Scores that rise (or fall) by `step` from key to key; odd: {place: value} of value number place % dim."""
    batch = R.Batch(new, lens, kv, dim, page, kind, seed=dim)
    q = torch.zeros((batch.rows, heads, dim), dtype=batch.dtype)
    q[:, :, 0] = math.sqrt(dim)
    for b, n in enumerate(lens):
        for j in range(n):
            batch.k[batch.table[b, j // page], :, j % page, 0] = step * (j - n / 2)
        for j, value in odd.items():
            if j < n:
                batch.v[batch.table[b, j // page], :, j % page, j % dim] = value
    got = qpg.cache_attention(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), window=window, dtype=R.TYPES[y]).cpu().double()
    at = strange = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        here, there = torch.arange(length - n, length), torch.arange(length)
        far = here[:, None] - there[None, :]
        see = (far >= 0) & ((far < window) if window else torch.ones_like(far, dtype=torch.bool))
        keys, values = batch.keys(b, batch.k), batch.keys(b, batch.v)
        for h in (0, heads - 1):
            want, bound = one_head(q[at:at + n, h], keys[:, h * kv // heads], values[:, h * kv // heads], see, far, kind, y,
                                   1 / math.sqrt(dim), 0.0, 0.0)
            mine, fine = got[at:at + n, h], torch.isfinite(want)
            assert torch.equal(torch.isnan(mine), torch.isnan(want)) and torch.equal(mine[torch.isinf(want)], want[torch.isinf(want)])
            assert float(((mine - want).abs() - bound)[fine].max()) <= 0
            strange += int((~fine).sum())
        at += n
    assert strange > 0 or window                # a window may have passed all of them


ODD = {0: math.inf, 33: -math.inf, 70: math.nan, 71: math.inf, 40: math.inf, 168: -math.inf, 300: math.inf}
# tiles of 32, 64 and 128 columns, one sequence and more, keys in one piece and in several
SHAPES = [([40, 1], [200, 340], 4, 2, 64, 16), ([9, 1], [1500, 900], 8, 2, 128, 64), ([520], [540], 32, 4, 64, 64),
          ([1030], [1030], 32, 4, 64, 64), ([2100], [2100], 64, 2, 128, 64), ([700], [750], 16, 8, 192, 32), ([5, 1], [1500, 20], 4, 2, 256, 32)]


@pytest.mark.parametrize("kind,y", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{sum(s[0])}-{max(s[1])}-{s[4]}" for s in SHAPES])
def test_shares_that_are_nothing(shape, kind, y):
    """Shares of the infinite values down to e^-300 and less: 0 in f32, and the rest of the row's values are multiplied by 0
    when the maximum moves."""
    new, lens, heads, kv, dim, page = shape
    for step in (0.25, -0.25, 0.03125):
        steep(new, lens, heads, kv, dim, page, kind, y, step, ODD)
    steep(new, lens, heads, kv, dim, page, kind, y, 0.25, ODD, window=290)
    steep(new, lens, heads, kv, dim, page, kind, y, 0.25, {max(lens) - 9: math.inf, max(lens) - 280: -math.inf, 19: math.nan}, window=290)


def test_scores_that_are_no_numbers():
    """A key that is no number makes the rows that see it NaN, and no other; infinite values beside it change nothing of that."""
    for kind, y in TYPES:
        batch = R.Batch([60], [200], 1, 64, 16, kind, seed=2)
        q = batch.normal(60, 4, 64)
        want, bound, _ = R.attention(batch, q, y)
        for j, c in ((170, batch.k), (175, batch.v), (160, batch.v)):
            c[batch.table[0, j // 16], :, j % 16] = math.nan if j == 170 else math.inf
        got = qpg.cache_attention(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), dtype=R.TYPES[y]).cpu().double()
        assert float(((got - want).abs() - bound)[:20].max()) <= 0               # before token 160
        assert bool((got[20:30] == math.inf).all()) and bool(torch.isnan(got[30:]).all())


def test_graph_replays_over_values_that_come_and_go():
    batch = R.Batch([130], [400], 2, 128, 64, "bf16", seed=1)
    q = batch.normal(130, 16, 128)
    args = [t.to(DEV) for t in (q, batch.k, batch.v)]
    index = batch.index(DEV)
    y = torch.zeros((130, 16, 128), dtype=torch.float32, device=DEV)
    qpg.cache_attention(*args, *index, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qpg.cache_attention(*args, *index, y=y)
    clean = batch.v.clone()
    for value in (None, math.inf, None, math.nan, -math.inf, None):
        batch.v.copy_(clean)
        if value is not None:
            for j in (3, 290, 333):
                batch.v[batch.table[0, j // 64], :, j % 64, j % 128] = value
        args[2].copy_(batch.v)
        graph.replay()
        torch.cuda.synchronize()
        want, bound, _ = R.attention(batch, q, "f32")
        got, fine = y.cpu().double(), torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
        assert float(((got - want).abs() - bound)[fine].max()) <= 0
        assert bool(fine.all()) == (value is None)
