"""Every form of the attentions' launch under every kind of mask and score, against 64 bits: windows, prefixes with
windows, caps and distances, trees in any order under windows, values that are no numbers in rows that some columns see.
Some heads of each call are compared, whole."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"

# new tokens, lengths, heads, cache heads, dim, page, pages of the table behind the longest sequence's; the form: tiles of
# 32 * WC columns, WK groups of waves, p: in pieces
FORMS = {"64 4x1": ([2100], [2100], 64, 2, 64, 256, 0), "128 4x1": ([2100], [2150], 64, 2, 128, 64, 0),
         "64 4x2": ([1030], [1030], 32, 4, 64, 64, 0), "128 4x2": ([1100], [1200], 32, 8, 128, 128, 0),
         "128 4x2p": ([520], [8000], 16, 4, 128, 16, 0), "64 2x4": ([520, 3], [540, 700], 32, 4, 64, 64, 0),
         "128 2x4": ([520], [600], 32, 8, 128, 32, 0), "128 2x4p": ([130, 3, 40], [400, 4200, 60], 8, 2, 128, 64, 0),
         "64 1x4": ([40, 1], [300, 77], 4, 2, 64, 16, 0), "128 1x4p": ([9, 1], [1500, 900], 8, 2, 128, 64, 3),
         "256 4x1": ([2100], [2100], 32, 2, 256, 64, 0), "256 2x2": ([700], [750], 16, 8, 192, 32, 0),
         "256 2x2p": ([100], [500], 8, 1, 256, 256, 16), "256 1x2p": ([5, 1], [1500, 20], 4, 2, 256, 32, 0)}


def one_head(q, k, v, see, far, kind, y, scale, cap, slope):
    """(y, bound) of rows q [n][dim] over keys k, v [len][dim] by see and far [n][len], in 64 bits; the bound as in cache_ref."""
    dim, length, dtype, y_type = q.shape[1], k.shape[0], R.TYPES[kind], R.TYPES[y]
    u = R.half(dtype) if R.half(y_type) >= R.half(dtype) else 4 * R.STEP
    q, k, v = q.double(), k.double(), v.double()
    s, off = scale * (q @ k.T), (dim + 8) * R.STEP * scale * (q.abs() @ k.abs().T)
    if cap:
        s = cap * torch.tanh(s / cap)
        off = off + (16 * R.STEP * cap if u == R.half(dtype) and cap <= 128 else 16 * R.STEP * s.abs())
    if slope:
        bias = slope * far.abs().double()
        s = s - bias
        off = off + 8 * R.STEP * (bias + s.abs())
    off = off + 8 * R.STEP * s.abs()
    s = torch.where(see, s, -math.inf)
    top = s.amax(dim=1, keepdim=True)
    w = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = w.sum(dim=1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0)
    vs = torch.where(torch.isfinite(v), v, 0.0)
    up, down = (see.double() @ (torch.isnan(v) | (v == x)).double() > 0 for x in (math.inf, -math.inf))
    want = w @ vs + torch.where(up, math.inf, 0.0) - torch.where(down, math.inf, 0.0)
    size = w @ vs.abs()
    worst = torch.where(see, off, 0.0).amax(dim=1, keepdim=True)
    bound = (2 * torch.expm1(worst) + u + (2 * length + 64) * R.STEP) * size
    if kind == "f16":
        bound = bound + length * 2.0 ** -31 * vs.abs().max()
    tiny = 2.0 ** -25 if y == "f16" else 0.0
    return want, bound * (1 + R.half(y_type)) + R.half(y_type) * torch.nan_to_num(want, 0.0, 0.0, 0.0).abs() + tiny


def compare(form, kind, y, cap=0.0, bias=False, window=0, prefix=None, tree=None, odd=()):
    """odd: (distance before the end of its sequence, value) of what is put into the values there."""
    new, lens, heads, kv, dim, page, extra = FORMS[form]
    batch = R.Batch(new, lens, kv, dim, page, kind, seed=len(form) + window, extra_width=extra, pad=2)
    gen, group, scale = batch.gen, heads // kv, 1.0 / math.sqrt(dim)
    q = batch.normal(batch.rows, heads, dim)
    for back, value in odd:
        for b, length in enumerate(lens):
            j = max(length - back, 0)
            batch.v[batch.table[b, j // page], :, j % page, back % dim] = value
    kw = {"cap": cap, "window": window}
    if bias:
        kw["slopes"] = 2.0 ** (-8.0 * torch.arange(1, heads + 1, dtype=torch.float32) / heads)
    if prefix:
        kw["prefix"] = torch.tensor([min(prefix * (b + 1), 4000) for b in range(len(new))], dtype=torch.int32)
    sees, places = [], torch.zeros(batch.rows, dtype=torch.int32)
    words, at = -(-max(new) // 64), 0
    bits = torch.zeros((batch.rows, 64 * words), dtype=torch.bool)
    for n, length in zip(new, lens):
        here, there = torch.arange(length - n, length), torch.arange(length)
        see = there[None, :] <= here[:, None]
        if tree:
            kin, depth, order = torch.zeros((n, n), dtype=torch.bool), [0] * n, list(range(n))
            if tree == "leaf first":
                order.reverse()
            elif tree == "mixed":
                order = torch.randperm(n, generator=gen).tolist()
            ups = torch.randint(1, 4, (n,), generator=gen).tolist()
            for i in range(n):
                if i:
                    up = order[max(0, i - ups[i])]
                    kin[order[i]] = kin[up]
                    depth[order[i]] = depth[up] + 1
                kin[order[i], order[i]] = True
            bits[at:at + n, :n] = kin
            here = length - n + torch.tensor(depth)
            there = torch.cat([there[:length - n], here])
            places[at:at + n] = here.to(torch.int32)
            see = torch.cat([torch.ones((n, length - n), dtype=torch.bool), kin], dim=1)
        far = here[:, None] - there[None, :]
        if window:
            see = see & (far < window)
        if prefix:
            see = see | (torch.arange(length)[None, :] < int(kw["prefix"][len(sees)]))
        sees.append((see, far))
        at += n
    if tree:
        weights = torch.ones(64, dtype=torch.int64) << torch.arange(64)
        kw.update(tree=(bits.view(batch.rows, words, 64) * weights).sum(dim=2), positions=places)
    out = torch.full(q.shape, 777.0, dtype=R.TYPES[y], device=DEV)
    call = qpg.cache_attention_tree if tree else qpg.cache_attention
    call(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), y=out,
         **{n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in kw.items()})
    torch.cuda.synchronize()
    got, at = out.cpu().double(), 0
    assert bool((got[at + sum(new):] == float(torch.tensor(777.0).to(R.TYPES[y]))).all())
    strange = 0
    for b, (n, (see, far)) in enumerate(zip(new, sees)):
        keys, values = batch.keys(b, batch.k), batch.keys(b, batch.v)
        for h in sorted({0, heads // 2 + 1, heads - 1}):
            slope = float(kw["slopes"][h]) if bias else 0.0
            want, bound = one_head(q[at:at + n, h], keys[:, h // group], values[:, h // group], see, far, kind, y, scale, cap, slope)
            mine, fine = got[at:at + n, h], torch.isfinite(want)
            assert torch.equal(torch.isfinite(mine), fine)
            inf = torch.isinf(want)
            assert torch.equal(mine[inf], want[inf]) and bool(torch.isnan(mine[torch.isnan(want)]).all())
            over = ((mine - want).abs() - bound)[fine]
            assert float(over.max()) <= 0, (h, float(over.max()))
            strange += int((~fine).sum())
        at += n
    return strange


TYPES = [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")]


@pytest.mark.parametrize("form", FORMS)
def test_windows(form):
    for i, window in enumerate((1, 40, 333)):
        compare(form, *TYPES[i], window=window)


@pytest.mark.parametrize("form", FORMS)
def test_prefixes(form):
    for i, (prefix, window) in enumerate(((150, 70), (37, 0), (1, 500), (2000, 64))):
        compare(form, *TYPES[i], prefix=prefix, window=window)


@pytest.mark.parametrize("form", FORMS)
def test_caps_and_distances(form):
    compare(form, *TYPES[0], cap=20.0, bias=True)
    compare(form, *TYPES[1], cap=4.0, bias=True, window=200)
    compare(form, *TYPES[2], bias=True, prefix=90)
    compare(form, *TYPES[3], cap=300.0)


@pytest.mark.parametrize("order", ["root first", "leaf first", "mixed"])
@pytest.mark.parametrize("form", FORMS)
def test_trees(form, order):
    kind, y = TYPES[len(order) % 4]
    compare(form, kind, y, tree=order)
    compare(form, kind, y, tree=order, window=30)
    compare(form, kind, y, tree=order, window=9, bias=True, cap=15.0)


@pytest.mark.parametrize("form", FORMS)
def test_values_that_are_no_numbers(form):
    """In rows near the end, which some new tokens see and others do not."""
    odd = ((3, math.nan), (20, math.inf), (33, -math.inf), (64, math.nan))
    for i, kw in enumerate(({}, {"window": 50}, {"prefix": 60, "window": 20, "bias": True}, {"tree": "mixed", "window": 12}, {"tree": "root first"})):
        assert compare(form, *TYPES[i % 4], odd=odd, **kw) > 0


@pytest.mark.parametrize("seed", range(28))
def test_random_masks(seed):
    import random
    r = random.Random(seed)
    form, (kind, y) = sorted(FORMS)[seed % len(FORMS)], r.choice(TYPES)
    kw = {"cap": r.choice([0.0, 0.0, 6.0, 500.0]), "bias": r.random() < 0.4, "window": r.choice([0, 1, 17, 64, 100, 600])}
    if r.random() < 0.5:
        kw["tree"] = r.choice(["root first", "leaf first", "mixed"])
    elif r.random() < 0.5:
        kw["prefix"] = r.choice([1, 64, 333, 1500])
    if r.random() < 0.3:
        kw["odd"] = tuple((r.randint(1, 300), r.choice([math.nan, math.inf, -math.inf])) for _ in range(3))
    compare(form, kind, y, **kw)
