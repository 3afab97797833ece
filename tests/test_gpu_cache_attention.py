"""Attention over a paged cache against 64 bits: head layouts, types, lengths, pages, masks, caps, distances, trees;
what is in masked places; rows in no sequence; refused and wrong arrays; streams and graph replays."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"


def run(batch, heads, y="same", scale=None, cap=0.0, bias=False, window=0, prefix=None, tree=0, q_scale=1.0, give=True,
        change=None, small=False):
    """The call and its check. tree: branches of random trees; change: edits (batch, q) before the call, and what it sees;
    small: shares may be too small for the cache's type."""
    y = batch.kind if y == "same" else y
    q = batch.normal(batch.rows, heads, batch.dim, scale=q_scale)
    kw = {"cap": cap, "window": window}
    if scale is not None:
        kw["scale"] = scale
    if bias:
        kw["slopes"] = 2.0 ** (-8.0 * torch.arange(1, heads + 1, dtype=torch.float32) / heads)
    if prefix is not None:
        kw["prefix"] = torch.tensor(prefix, dtype=torch.int32)
    if tree:
        lead = int(batch.offsets[0])
        bits, depths = R.tree_of(batch.gen, batch.new, tree)
        words = -(-max(batch.new) // 64)
        kw["tree"] = R.words_of(bits, batch.rows, lead, words)
        kw["positions"] = torch.zeros(batch.rows, dtype=torch.int32)
        at = 0
        for n, length in zip(batch.new, batch.lens_list):
            for i in range(n):
                kw["positions"][lead + at + i] = length - n + depths[at + i]
            at += n
    if change:
        change(batch, q)
    want, bound, mine = R.attention(batch, q, y, **kw)
    out = torch.full(q.shape, 777.0, dtype=R.TYPES[y], device=DEV) if give else None
    kw = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    call = qpg.cache_attention_tree if tree else qpg.cache_attention
    got = call(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), y=out, dtype=R.TYPES[y], **kw)
    torch.cuda.synchronize()
    assert got.shape == q.shape and got.dtype == R.TYPES[y]
    got = got.cpu().double()
    check(got[mine], want[mine], bound[mine], pieces=small or R.half(R.TYPES[y]) < R.half(batch.dtype))
    if give:
        assert bool((got[~mine] == float(torch.tensor(777.0).to(R.TYPES[y]))).all())
    return got, want, mine


def check(got, want, bound, pieces=False):
    """pieces: shares in several pieces, some of which may be 0 or below, or shares that may round to 0: with an infinite
    value they make NaN."""
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    odd = torch.isinf(want) & ~(torch.isnan(got) if pieces else torch.zeros_like(got, dtype=torch.bool))
    assert torch.equal(got[odd], want[odd])
    assert bool(torch.isnan(got[torch.isnan(want)]).all())
    fine = torch.isfinite(want)
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (float(over.max()), float((got - want).abs()[fine].max()))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 128, 136, 192, 256])
def test_head_sizes(dim, kind):
    run(R.Batch([5, 1, 70], [9, 40, 70], 2, dim, 16, kind, seed=dim), 4)


@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 6), (6, 2), (5, 1), (32, 2), (64, 1), (40, 1)])
def test_head_layouts_and_types(heads, kv, kind, y):
    run(R.Batch([3, 33], [130, 77], kv, 64, 32, kind, seed=heads), heads, y)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1000])
def test_single_tokens(length, page):
    run(R.Batch([1, 1], [length, 1], 2, 128, page, "bf16", seed=length), 4, "f32")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 300])
def test_prompts(new, dim):
    run(R.Batch([new], [new], 1, dim, 16, "f16", seed=new), 1)
    run(R.Batch([new], [new + 37], 1, dim, 32, "bf16", seed=new), 3, "f32")


@pytest.mark.parametrize("B", [3, 64, 65, 200])
def test_many_sequences(B):
    new = [(i * 7) % 4 for i in range(B)]
    run(R.Batch(new, [n + (i * 37) % 150 for i, n in enumerate(new)], 1, 64, 16, "bf16", seed=B, lead=2, pad=3), 2)


def test_long_sequences_in_pieces():
    run(R.Batch([1], [8191], 1, 128, 64, "f16", seed=1), 4, "f32")
    run(R.Batch([1, 1, 1], [3000, 5, 4097], 2, 128, 64, "bf16", seed=2), 4)
    run(R.Batch([40, 9], [5000, 2100], 1, 64, 64, "bf16", seed=3), 4, "f32")
    run(R.Batch([300], [3300], 1, 256, 128, "f16", seed=4), 1)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 63, 64, 65, 100, 5000])
def test_windows(window):
    run(R.Batch([130, 1, 7], [300, 200, 7], 1, 64, 16, "f16", seed=window), 2, window=window)
    run(R.Batch([1, 1], [1500, 64], 2, 128, 16, "bf16", seed=window), 4, window=window)


@pytest.mark.parametrize("prefix", [[0, 0, 0], [1, 300, 3], [64, 65, 7], [1000, 128, 0], [129, 20, -5]])
@pytest.mark.parametrize("window", [0, 10, 70])
def test_prefixes(prefix, window):
    run(R.Batch([130, 290, 7], [300, 290, 7], 1, 64, 16, "bf16", seed=prefix[0]), 3, window=window, prefix=prefix)
    run(R.Batch([1, 2, 7], [300, 1290, 7], 1, 128, 16, "bf16", seed=prefix[0]), 3, window=window, prefix=prefix)


@pytest.mark.parametrize("y", ["f32", "f16"])
@pytest.mark.parametrize("cap", [0.5, 3.0, 50.0, 128.0, 129.0, 1e6])
def test_caps(cap, y):
    run(R.Batch([70, 1], [100, 33], 2, 80, 16, "f16", seed=3), 2, y, cap=cap, q_scale=8.0)


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("scale", [None, 1.0, 0.01, 3e-6])
def test_scales_and_distances(scale, cap):
    run(R.Batch([70, 1], [200, 333], 2, 72, 16, "bf16", seed=3), 6, scale=scale, cap=cap, bias=True)
    run(R.Batch([70, 1], [200, 333], 2, 72, 16, "bf16", seed=4), 6, "f32", scale=scale, cap=cap, bias=True, prefix=[150, 400], window=40)


def test_steep_scores():
    """A maximum that moves by much from key to key, both ways."""
    def ramp(sign):
        def change(batch, q):
            q[:] = 1.0
            for b, n in enumerate(batch.lens_list):
                for j in range(n):
                    batch.k[batch.table[b, j // 16], :, j % 16] = sign * (j - n / 2) / 2
        return change
    for sign in (1, -1):
        for y in ("f16", "f32"):
            run(R.Batch([90, 1], [200, 700], 1, 64, 16, "f16", seed=5), 2, y, change=ramp(sign))


@pytest.mark.parametrize("branch", [1, 3, 200])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([26], [26]), ([5, 64, 1], [205, 64, 100]), ([65, 128, 33], [300, 129, 1033]),
                                      ([200], [777])])
def test_trees(new, lens, branch):
    run(R.Batch(new, lens, 2, 64, 16, "bf16", seed=branch, lead=1, pad=2), 8, tree=branch)
    run(R.Batch(new, lens, 1, 128, 32, "f16", seed=branch), 3, "f32", tree=branch, window=19, bias=True, cap=10.0)


def test_tree_with_too_few_words():
    """Nodes that no bit stands for are seen by none."""
    batch = R.Batch([70], [100], 1, 64, 16, "f16", seed=3)
    q = batch.normal(70, 2, 64)
    bits, depths = R.tree_of(batch.gen, [70], 2)
    tree = R.words_of(bits, 70, 0, 1)
    positions = torch.tensor([30 + d for d in depths], dtype=torch.int32)
    want, bound, _ = R.attention(batch, q, "f16", tree=tree, positions=positions)
    got = qpg.cache_attention_tree(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), tree.to(DEV), positions.to(DEV))
    check(got.cpu().double(), want, bound)


def test_more_new_tokens_than_the_length_says():
    """The first ones have no place: they see nothing (zeros), or the prefix."""
    got, want, _ = run(R.Batch([50, 3], [20, 0], 1, 64, 16, "bf16", seed=1), 2)
    assert bool((got[:30] == 0).all()) and bool((got[50:53] == 0).all()) and bool((got[31:50] != 0).any())
    run(R.Batch([50, 3], [20, 0], 1, 64, 16, "bf16", seed=1), 2, prefix=[5, 9])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_values_of_later_tokens_touch_nothing(what, dim):
    """Keys and values that are no numbers: rows that see them have them, the others are as if they were not there."""
    for kind, y in (("bf16", "bf16"), ("f16", "f32")):
        for new, lens, heads, kw in (([100], [150], 1, {}), ([9, 40], [90, 40], 4, {"window": 20}), ([33], [70], 2, {"tree": 2})):
            def change(batch, q):
                n, length = batch.new[0], batch.lens_list[0]
                j = length - n // 2                      # seen by the later half of the new tokens
                batch.v[batch.table[0, j // 16], :, j % 16, 3] = what
                j = length - 2
                batch.v[batch.table[0, j // 16], :, j % 16, : dim // 2] = -what
            got, want, _ = run(R.Batch(new, lens, 1, dim, 16, kind, seed=dim), heads, y, change=change, **kw)
            assert bool(torch.isfinite(want).any()) and not bool(torch.isfinite(want).all())

    def key(batch, q):
        batch.k[batch.table[0, 149 // 16], :, 149 % 16] = what
    # the last key is seen by the last token alone; its score is no number, or of either sign by the query's
    batch = R.Batch([100], [150], 1, dim, 16, "bf16", seed=dim)
    q = batch.normal(100, 1, dim)
    before, bound, _ = R.attention(batch, q, "bf16")
    key(batch, q)
    got = qpg.cache_attention(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV)).cpu().double()
    check(got[:99], before[:99], bound[:99])
    assert bool(torch.isnan(got[99]).all())


def test_lengths_and_tables_that_point_outside():
    """Clamped: rows may be wrong, nothing outside is touched, and the other sequences are right."""
    batch = R.Batch([3, 5], [40, 60], 2, 64, 16, "f16", seed=9, spare=0)
    q = batch.normal(8, 2, 64)
    want, bound, _ = R.attention(batch, q, "f16")
    k, v = batch.k.to(DEV), batch.v.to(DEV)
    for at, value in (("table", 1 << 30), ("table", -7), ("lens", 1 << 30), ("lens", -3), ("offsets", -9)):
        table, lens, offsets = batch.index(DEV)
        {"table": table[0], "lens": lens[:1], "offsets": offsets[:1]}[at][:1] = value
        got = qpg.cache_attention(q.to(DEV), k, v, table, lens, offsets).cpu().double()
        check(got[3:], want[3:], bound[3:])


def test_strided_pages():
    """Keys and values side by side in one pool, pages that other layers' lie between."""
    batch = R.Batch([3, 50], [40, 60], 2, 80, 16, "bf16", seed=9)
    q = batch.normal(53, 4, 80)
    want, bound, _ = R.attention(batch, q, "bf16")
    pool = torch.full((batch.pool, 3, 2, 2, 16, 80), math.nan, dtype=torch.bfloat16, device=DEV)
    k, v = pool[:, 1, 0], pool[:, 1, 1]
    k.copy_(batch.k)
    v.copy_(batch.v)
    got = qpg.cache_attention(q.to(DEV), k, v, *batch.index(DEV)).cpu().double()
    check(got, want, bound)


def test_pages_past_32_bits():
    """A pool of 9 GiB whose used pages lie at its ends."""
    page, kv, dim = 256, 8, 128
    pool = (9 << 30) // (page * kv * dim * 2)
    batch = R.Batch([2, 1], [700, 300], kv, dim, page, "bf16", seed=4, spare=0)
    q = batch.normal(3, 8, dim)
    want, bound, _ = R.attention(batch, q, "bf16")
    k, v = (torch.empty((pool, kv, page, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moved = torch.tensor([0, pool - 1, pool // 2, pool - 2, 3])
    for c, src in ((k, batch.k), (v, batch.v)):
        for i, to in enumerate(moved.tolist()):
            c[to].copy_(src[i])
    table, lens, offsets = batch.index("cpu")
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()].to(torch.int32), table)
    got = qpg.cache_attention(q.to(DEV), k, v, table.to(DEV), lens.to(DEV), offsets.to(DEV)).cpu().double()
    check(got, want, bound)


def test_same_result_every_time_and_in_any_workspace():
    batch = R.Batch([1, 30], [5000, 3000], 2, 128, 64, "bf16", seed=4)
    q = batch.normal(31, 8, 128).to(DEV)
    args = (q, batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV))
    size = qpg.cache_attention_bytes(31, 2, 8, 2, 128, batch.width * 64)
    assert size > 0
    first = qpg.cache_attention(*args)
    for fill in (0, 255):
        ws = torch.full((size + 512,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(qpg.cache_attention(*args, ws=ws[:size]), first)
        assert bool((ws[size:] == fill).all())
        assert torch.equal(qpg.cache_attention(*args), first)


def test_streams():
    batches = [R.Batch([1, 30], [5000, 3000 + i], 2, 128, 64, "bf16", seed=i) for i in range(2)]
    qs = [b.normal(31, 8, 128).to(DEV) for b in batches]
    args = [(q, b.k.to(DEV), b.v.to(DEV), *b.index(DEV)) for q, b in zip(qs, batches)]
    want = [qpg.cache_attention(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(qpg.cache_attention(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


def test_graph_replays_with_other_contents():
    """One captured step for lengths up to the table's: other lengths, pages and rows on every replay."""
    cases = [R.Batch(new, lens, 2, 64, 16, "f16", seed=i, pad=6 - sum(new), spare=60 - sum(-(-n // 16) for n in lens),
                     extra_width=40 - max(-(-n // 16) for n in lens))
             for i, (new, lens) in enumerate([([1, 1, 1], [640, 1, 77]), ([2, 0, 3], [500, 0, 9]), ([0, 6, 0], [0, 300, 5]), ([1, 1, 4], [16, 16, 16])])]
    qs = [b.normal(6, 4, 64) for b in cases]
    b = cases[0]
    q, k, v, table, lens, offsets = (t.to(DEV) for t in (qs[0], b.k, b.v, b.table, b.lens, b.offsets))
    y = torch.full((6, 4, 64), 777.0, dtype=torch.float32, device=DEV)
    size = qpg.cache_attention_bytes(6, 3, 4, 2, 64, 640)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    step = lambda: qpg.cache_attention(q, k, v, table, lens, offsets, y=y, ws=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 2, 3, 1, 0):
        b = cases[i]
        for to, src in ((q, qs[i]), (k, b.k), (v, b.v), (table, b.table), (lens, b.lens), (offsets, b.offsets)):
            to.copy_(src)
        y.fill_(777.0)
        graph.replay()
        torch.cuda.synchronize()
        want, bound, mine = R.attention(b, qs[i], "f32")
        got = y.cpu().double()
        check(got[mine], want[mine], bound[mine])
        assert bool((got[~mine] == 777.0).all())
        assert torch.equal(qpg.cache_attention(q, k, v, table, lens, offsets, dtype=torch.float32)[mine.to(DEV)], y[mine.to(DEV)])


# Shapes that take each form of the launch (tiles of 32, 64 and 128 columns, one and two groups of waves, one and more
# pieces): new tokens, lengths, heads, cache heads, dim, page
FORMS = [([256], [256], 32, 32, 64, 16), ([520], [520], 32, 32, 64, 64), ([520], [600], 32, 8, 128, 64), ([1030], [1030], 32, 32, 64, 64),
         ([1100], [1100], 32, 8, 128, 128), ([2100], [2100], 64, 64, 64, 256), ([130, 3, 40], [5000, 4200, 60], 16, 4, 128, 64),
         ([300], [5000], 16, 4, 128, 16), ([520], [4500], 8, 8, 256, 64), ([700], [700], 16, 8, 192, 32), ([2100], [2100], 32, 32, 256, 64),
         ([1] * 40, [4200] + [i * 3 + 1 for i in range(39)], 16, 4, 128, 64)]


@pytest.mark.parametrize("kind,y", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("case", FORMS, ids=[f"{sum(c[0])}-{max(c[1])}-{c[2]}-{c[3]}-{c[4]}" for c in FORMS])
def test_forms(case, kind, y):
    """Rows here and there of large calls against 64 bits."""
    new, lens, heads, kv, dim, page = case
    batch = R.Batch(new, lens, kv, dim, page, kind, seed=len(new))
    q = batch.normal(batch.rows, heads, dim)
    got = qpg.cache_attention(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), dtype=R.TYPES[y]).cpu().double()
    group, at = heads // kv, 0
    for b, (n, length) in enumerate(zip(new, lens)):
        for h in sorted({0, heads - 1, heads // 2}):
            one = R.Batch([n], [length], 1, dim, page, kind, seed=0)
            for c, src in ((one.k, batch.k), (one.v, batch.v)):
                for p in range(-(-length // page)):
                    c[one.table[0, p], 0] = src[batch.table[b, p], h // group]
            want, bound, _ = R.attention(one, q[at:at + n, h:h + 1], y)
            check(got[at:at + n, h:h + 1], want, bound)
        at += n


def test_the_longest_sequence():
    """2^29 tokens and a few: the pieces cover all of them. Keys are alike but for some, so the shares are known."""
    page, dim = 256, 8
    length = (1 << 29) + 300
    pages = -(-length // page)
    k = torch.zeros((pages, 1, page, dim), dtype=torch.float16, device=DEV)
    v = torch.zeros((pages, 1, page, dim), dtype=torch.float16, device=DEV)
    rows = k.view(-1, dim)
    at = torch.tensor([0, 1 << 20, (1 << 24) + 7, (1 << 28) + 5, (1 << 29) - 1, 1 << 29, length - 1], device=DEV)
    rows[:, 0] = -30.0                                 # shares of e^-60 of the others': together 2^29 e^-60, below 2^-50
    rows[at, 0] = 30.0
    v.view(-1, dim)[at, 1] = torch.arange(1, len(at) + 1, dtype=torch.float16, device=DEV)
    q = torch.zeros((1, 1, dim), dtype=torch.float16, device=DEV)
    q[0, 0, 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    lens, offsets = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([length], [0, 1]))
    for window in (0, 1 << 28, length - 1):
        seen = int((length - 1 - at < (window or length)).sum())
        y = qpg.cache_attention(q, k, v, table, lens, offsets, scale=1.0, window=window, dtype=torch.float32)[0, 0].cpu().double()
        values = torch.arange(len(at) - seen + 1, len(at) + 1, dtype=torch.float64)
        # shares are powers of exactly equal scores: equal; sums of a few terms
        assert abs(float(y[1]) - float(values.mean())) <= 64 * 2.0 ** -24 * 7 and float(y[0]) == 0 and bool((y[2:] == 0).all())


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream, with eager work between: each call writes all of the workspace that it reads."""
    made = []
    batches = [R.Batch([1, 1], [5000, 900], 2, 128, 64, "bf16", seed=1), R.Batch([30], [3000], 1, 64, 64, "bf16", seed=2)]
    sizes = [qpg.cache_attention_bytes(2, 2, 8, 2, 128, batches[0].width * 64), qpg.cache_attention_bytes(30, 1, 4, 1, 64, batches[1].width * 64)]
    assert min(sizes) > 0
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    for b, heads in zip(batches, (8, 4)):
        args = (b.normal(b.rows, heads, b.dim).to(DEV), b.k.to(DEV), b.v.to(DEV), *b.index(DEV))
        want = qpg.cache_attention(*args)
        y = torch.zeros_like(want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            qpg.cache_attention(*args, y=y, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qpg.cache_attention(*args, y=y, ws=ws)
        made.append((graph, args, y, want))
    for turn in (0, 1, 1, 0, 1, 0):
        graph, args, y, want = made[turn]
        y.zero_()
        graph.replay()
        again = qpg.cache_attention(*args)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(again, want)


def draw(seed):
    """A random call: sequences, heads, masks and all; values that are no numbers in one of four."""
    import random
    r = random.Random(seed)
    kind = r.choice(["f16", "bf16"])
    kv = r.choice([1, 1, 2, 3, 8])
    group = r.choice([1, 1, 2, 3, 4, 7, 8])
    dim = 8 * r.choice([1, 2, 5, 8, 8, 10, 12, 16, 16, 17, 24, 32])
    tree = r.choice([0, 0, 1, 3])
    B = r.choice([1, 2, 3, 5, 66])
    most = 3 if B > 5 else r.choice([1, 2, 9, 40, 150])
    new = [r.randint(0, most) for _ in range(B)]
    new[r.randrange(B)] = most
    far = r.choice([0, 5, 70, 300] if B > 5 else [0, 5, 70, 700, 2500])
    lens = [max(0, n + r.randint(0, far) - (r.choice([0, 0, 0, 4]) if not tree else 0)) for n in new]
    batch = R.Batch(new, lens, kv, dim, r.choice([16, 32, 64, 128, 256]), kind, seed=seed, lead=r.choice([0, 0, 2]), pad=r.choice([0, 0, 3]),
                    extra_width=r.choice([0, 0, 1, 40]))
    kw = {"y": r.choice(["same", "f32", "f16", "bf16"]), "cap": r.choice([0.0, 0.0, 5.0, 40.0, 1000.0]), "bias": r.random() < 0.3,
          "window": r.choice([0, 0, 1, 17, 64, 300]), "tree": tree, "q_scale": r.choice([0.3, 1.0, 4.0]), "small": True}
    if not tree and r.random() < 0.3:
        kw["prefix"] = [r.randint(0, 400) for _ in range(B)]
    if r.random() < 0.25:
        def change(b, q):
            for _ in range(3):
                s = r.randrange(B)
                if lens[s]:
                    j = r.randrange(lens[s])
                    b.v[b.table[s, j // b.page], :, j % b.page, r.randrange(dim)] = r.choice([math.nan, math.inf, -math.inf])
        kw["change"] = change
    return batch, kv * group, kw


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    batch, heads, kw = draw(seed)
    run(batch, heads, **kw)
