"""Appending to a paged cache against 64 bits: norms, rotations of both kinds and any part of a head, far positions,
types, row strides and alignments; tokens without a place; what is left alone; graph replays."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"


def freqs_of(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def run(batch, heads, x="f32", rot=0, adjacent=False, norm=False, positions=None, fused=False, shift=0, eps=1e-6, base=10000.0,
        weights_at=0):
    wide = [heads * batch.dim, batch.kv * batch.dim, batch.kv * batch.dim]
    q, k, v = (batch.normal(batch.rows, w, scale=2.0, kind=x) if w else None for w in wide)
    kw = {"adjacent": adjacent, "eps": eps, "freqs": freqs_of(rot, base) if rot else None,
          "positions": None if positions is None else torch.tensor(positions, dtype=torch.int32),
          "q_norm": 1 + 0.3 * batch.normal(batch.dim, kind="f32") if norm and heads else None,
          "k_norm": 1 + 0.3 * batch.normal(batch.dim, kind="f32") if norm else None}
    ((wq, bq), (wk, bk), (wv, bv)), where = R.append(batch, q, k, v, **kw)
    if fused:                                           # one buffer, rows `shift` values further apart
        whole = torch.zeros((batch.rows, sum(wide) + shift), dtype=R.TYPES[x], device=DEV)
        parts = whole[:, shift // 2:].split([*wide, shift - shift // 2], dim=1)
        for p, t in zip(parts, (q, k, v)):
            if t is not None:
                p.copy_(t)
        dq, dk, dv = (p if p.shape[1] else None for p in parts[:3])
    else:
        dq, dk, dv = (None if t is None else t.to(DEV) for t in (q, k, v))
    before = [batch.normal(*batch.k.shape), batch.normal(*batch.k.shape)]
    kc, vc = (t.to(DEV) for t in before)
    y = torch.full((batch.rows, heads, batch.dim), 777.0, dtype=batch.dtype, device=DEV) if heads else None
    kw = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in kw.items()}
    for n in ("q_norm", "k_norm"):                      # at any element of a buffer
        if kw[n] is not None:
            kw[n] = torch.cat([torch.zeros(weights_at, device=DEV), kw[n]])[weights_at:]
    got = qpg.cache_append(dq, dk, dv, kc, vc, *batch.index(DEV), y=y, **kw)
    torch.cuda.synchronize()
    lead, end = int(batch.offsets[0]), int(batch.offsets[-1])
    if heads:
        assert got is y
        got = got.cpu().double()
        assert float(((got - wq).abs() - bq)[lead:end].max()) <= 0, float(((got - wq).abs() / bq)[lead:end].max())
        left = float(torch.tensor(777.0).to(batch.dtype))
        assert bool((got[:lead] == left).all()) and bool((got[end:] == left).all())
    else:
        assert got is None
    for c, old, want, bound in ((kc, before[0], wk, bk), (vc, before[1], wv, bv)):
        expect, most = old.double(), torch.zeros(old.shape, dtype=torch.float64)
        for row, page, place in where:
            expect[page, :, place] = want[row]
            most[page, :, place] = bound[row]
        over = (c.cpu().double() - expect).abs() - most
        assert float(over.max()) <= 0, float(over.max())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_types(adjacent, norm, x, kind):
    run(R.Batch([3, 1, 20], [9, 40, 20], 2, 128, 16, kind, seed=1), 4, x, 128, adjacent, norm)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 8), (8, 0), (16, 8), (40, 24), (64, 64), (72, 72), (80, 32), (96, 96), (128, 64), (136, 8),
                                     (192, 192), (256, 256), (256, 128), (248, 240)])
def test_head_sizes_and_rotated_parts(dim, rot, adjacent):
    run(R.Batch([3, 1, 20], [9, 40, 20], 2, dim, 16, "f16", seed=dim + rot), 6, "f32", rot, adjacent, True)
    run(R.Batch([7], [9], 1, dim, 32, "bf16", seed=dim + rot), 1, "bf16", rot, adjacent, False)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (32, 8), (64, 1), (9, 3), (0, 4), (128, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_head_layouts(heads, kv, page):
    run(R.Batch([2, 5], [300, 5], kv, 64, page, "bf16", seed=heads), heads, "f32", 64, True, True)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 8, 2, 1, 7])
def test_slices_of_one_product(shift, x):
    """Rows at any distance, and beginning at any element."""
    run(R.Batch([2, 5], [30, 5], 3, 40, 16, "bf16", seed=shift), 6, x, 40, False, True, fused=True, shift=shift)


@pytest.mark.parametrize("weights_at", [1, 2, 3])
def test_norm_weights_at_any_element(weights_at):
    run(R.Batch([2, 5], [30, 5], 3, 40, 16, "bf16", seed=3), 6, "f32", 40, True, True, weights_at=weights_at)


def test_tokens_by_the_thousand():
    run(R.Batch([1000, 1, 1500], [1000, 70, 1600], 2, 64, 64, "f16", seed=7, lead=3, pad=5), 4, "bf16", 64, True, True)
    run(R.Batch([1] * 300, [1 + i % 90 for i in range(300)], 1, 64, 16, "f16", seed=8, pad=9), 2, "f32", 32, False, False)


@pytest.mark.parametrize("adjacent", [False, True])
def test_far_positions(adjacent):
    """Angles of up to 2^31 turns of the fastest pair."""
    positions = [0, 1, 1000, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -5]
    run(R.Batch([8], [8], 1, 64, 16, "f16", seed=2), 2, "f32", 64, adjacent, positions=positions)
    run(R.Batch([8], [8], 1, 64, 16, "f16", seed=2), 2, "f32", 64, adjacent, positions=positions, base=1e6, norm=True)


def test_tokens_without_a_place():
    """More new tokens than the length says; entries of the table that are no page; empty sequences; wrong arrays."""
    run(R.Batch([50, 3, 0, 2], [20, 0, 30, 17], 2, 64, 16, "bf16", seed=1), 2, rot=64)
    batch = R.Batch([5, 3], [20, 40], 2, 64, 16, "bf16", seed=1)
    batch.table[0, 1] = -1
    batch.table[1, 2] = batch.pool
    run(batch, 2, rot=64)
    # a length behind the table: clamped to it
    batch = R.Batch([5, 3], [32, 48], 1, 64, 16, "f16", seed=1)
    batch.lens = torch.tensor([32, 1 << 30], dtype=torch.int32)
    run(batch, 2)


def test_zeros_and_large_values_in_a_norm():
    batch = R.Batch([4], [4], 1, 64, 16, "bf16", seed=1)
    x = torch.zeros((4, 64))
    x[1], x[2, 5], x[3] = 1e18, 3e-20, 1e-30
    kc = torch.zeros(batch.k.shape, dtype=torch.bfloat16, device=DEV)
    got = qpg.cache_append(x.to(DEV), x.to(DEV), x.to(DEV), kc, kc.clone(), *batch.index(DEV), q_norm=torch.ones(64, device=DEV),
                           k_norm=torch.ones(64, device=DEV)).cpu().double()[:, 0]
    assert bool((got[0] == 0).all())
    want = x.double() / torch.sqrt((x.double() ** 2).mean(dim=1, keepdim=True) + 1e-6)
    assert float((got - want).abs().max()) <= 2.0 ** -8


def test_strided_pages():
    batch = R.Batch([3, 5], [40, 60], 2, 80, 16, "bf16", seed=9)
    pool = torch.zeros((batch.pool, 2, 2, 16, 80), dtype=torch.bfloat16, device=DEV)
    k, v = (batch.normal(8, 160, kind="f32") for _ in range(2))
    assert qpg.cache_append(None, k.to(DEV), v.to(DEV), pool[:, 0], pool[:, 1], *batch.index(DEV)) is None
    (_, (wk, bk), (wv, bv)), where = R.append(batch, None, k, v)
    want, most = torch.zeros((2, *pool.shape), dtype=torch.float64)
    for row, page, place in where:
        for side, (w, b) in enumerate(((wk, bk), (wv, bv))):
            want[page, side, :, place], most[page, side, :, place] = w[row], b[row]
    assert float(((pool.cpu().double() - want).abs() - most).max()) <= 0


def test_pages_past_32_bits():
    page, kv, dim = 256, 8, 128
    pool = (5 << 30) // (page * kv * dim * 2)
    batch = R.Batch([2, 1], [700, 300], kv, dim, page, "bf16", seed=4, spare=0)
    k, v = (batch.normal(3, kv * dim, kind="f32") for _ in range(2))
    (_, (wk, bk), (wv, bv)), where = R.append(batch, None, k, v)
    kc, vc = (torch.zeros((pool, kv, page, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moved = torch.tensor([0, pool - 1, pool // 2, pool - 2, 3])
    table, lens, offsets = batch.index("cpu")
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()].to(torch.int32), table)
    qpg.cache_append(None, k.to(DEV), v.to(DEV), kc, vc, table.to(DEV), lens.to(DEV), offsets.to(DEV))
    for row, p, place in where:
        for c, w, b in ((kc, wk, bk), (vc, wv, bv)):
            assert float(((c[int(moved[p]), :, place].cpu().double() - w[row]).abs() - b[row]).max()) <= 0
    assert all(int((c != 0).any(dim=3).sum()) == 3 * kv for c in (kc, vc))


def test_graph_replays_and_streams():
    cases = [R.Batch(new, lens, 2, 64, 16, "f16", seed=i, pad=6 - sum(new), spare=60 - sum(-(-n // 16) for n in lens),
                     extra_width=40 - max(-(-n // 16) for n in lens))
             for i, (new, lens) in enumerate([([1, 1, 1], [640, 1, 77]), ([2, 0, 3], [500, 0, 9]), ([0, 6, 0], [0, 300, 5])])]
    inputs = [[b.normal(6, w, kind="f32") for w in (256, 128, 128)] for b in cases]
    freqs = freqs_of(64).to(DEV)
    b = cases[0]
    table, lens, offsets = b.index(DEV)
    q, k, v = (t.to(DEV) for t in inputs[0])
    kc, vc = (torch.zeros(b.k.shape, dtype=torch.float16, device=DEV) for _ in range(2))
    y = torch.zeros((6, 4, 64), dtype=torch.float16, device=DEV)
    step = lambda s=None: qpg.cache_append(q, k, v, kc, vc, table, lens, offsets, freqs=freqs, y=y, stream=s)  # noqa: E731
    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 2, 1):
        b = cases[i]
        for to, src in ((table, b.table), (lens, b.lens), (offsets, b.offsets), (q, inputs[i][0]), (k, inputs[i][1]), (v, inputs[i][2])):
            to.copy_(src)
        results = []
        for how in (graph.replay, step, lambda: step(side)):
            for t in (kc, vc, y):
                t.fill_(9.0)
            torch.cuda.synchronize()
            how()
            torch.cuda.synchronize()
            results.append([t.clone() for t in (kc, vc, y)])
        assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))
        ((wq, bq), (wk, bk), _), where = R.append(b, *inputs[i], freqs=freqs.cpu())
        n = int(b.offsets[-1])
        assert float(((results[0][2].cpu().double() - wq).abs() - bq)[:n].max()) <= 0 and bool((results[0][2][n:] == 9.0).all())
        for row, page, place in where:
            assert float(((results[0][0][page, :, place].cpu().double() - wk[row]).abs() - bk[row]).max()) <= 0


def draw(seed):
    """A random call: sequences, heads, types, rotated part, slices."""
    import random
    r = random.Random(seed)
    dim = 8 * r.choice([1, 2, 5, 8, 8, 10, 16, 16, 17, 24, 32])
    kv, B = r.choice([1, 2, 3, 8]), r.choice([1, 2, 3, 70])
    new = [r.randint(0, r.choice([1, 3, 60] if B < 5 else [1, 2])) for _ in range(B)]
    new[r.randrange(B)] += 1
    lens = [max(0, n + r.randint(0, 200) - r.choice([0, 0, 0, 3])) for n in new]
    batch = R.Batch(new, lens, kv, dim, r.choice([16, 32, 64, 128, 256]), r.choice(["f16", "bf16"]), seed=seed, lead=r.choice([0, 2]),
                    pad=r.choice([0, 3]), extra_width=r.choice([0, 2]))
    kw = {"x": r.choice(["f32", "f16", "bf16"]), "rot": r.choice([0, dim, 8 * r.randint(0, dim // 8)]), "adjacent": r.random() < 0.5,
          "norm": r.random() < 0.5, "fused": r.random() < 0.5, "shift": r.choice([0, 0, 8, 3]), "eps": r.choice([1e-6, 1e-5, 0.0]),
          "weights_at": r.choice([0, 0, 1])}
    if r.random() < 0.3:
        kw["positions"] = [r.randint(0, 200000) for _ in range(batch.rows)]
    return batch, kv * r.choice([0, 1, 2, 3, 7]), kw


@pytest.mark.parametrize("seed", range(30))
def test_random_calls(seed):
    batch, heads, kw = draw(seed)
    run(batch, heads, **kw)
