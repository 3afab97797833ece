"""Trees of drafts whose nodes are stored in any order, parents before their children or behind them, under windows: which
nodes a node sees goes by the bits and the positions, not by where the nodes lie."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"


def tree_in_order(gen, new, branch, order):
    """Random trees (parents at most `branch` nodes back), their nodes stored root first, leaf first or in no order: rows of
    bits as Python ints, and depths."""
    bits, depths = [], []
    for n in new:
        at = {"root first": torch.arange(n), "leaf first": torch.arange(n - 1, -1, -1), "mixed": torch.randperm(n, generator=gen)}[order].tolist()
        mine, deep = [0] * n, [0] * n
        for i in range(n):
            up = at[max(0, i - int(torch.randint(1, branch + 1, (1,), generator=gen)))] if i else None
            mine[at[i]] = (1 << at[i]) | (mine[up] if i else 0)
            deep[at[i]] = deep[up] + 1 if i else 0
        bits += mine
        depths += deep
    return bits, depths


def compare(batch, heads, y, order, branch=1, ahead=0, **kw):
    q = batch.normal(batch.rows, heads, batch.dim)
    lead = int(batch.offsets[0])
    bits, depths = tree_in_order(batch.gen, batch.new, branch, order)
    tree = R.words_of(bits, batch.rows, lead, -(-max(batch.new) // 64))
    positions = torch.zeros(batch.rows, dtype=torch.int32)
    starts = [length - n for n, length in zip(batch.new, batch.lens_list) for _ in range(n)]
    positions[lead:lead + len(bits)] = torch.tensor([s + d + ahead for s, d in zip(starts, depths)], dtype=torch.int32)
    want, bound, mine = R.attention(batch, q, y, tree=tree, positions=positions, **kw)
    kw = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    got = qpg.cache_attention_tree(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), tree.to(DEV), positions.to(DEV),
                                   dtype=R.TYPES[y], **kw).cpu().double()
    over = ((got - want).abs() - bound)[mine]
    assert float(over.max()) <= 0, float(over.max())
    assert bool((want[mine] != 0).any(dim=2).all())           # every node sees itself


# new nodes, lengths, cache heads, heads, dim, page, pages of the table behind the longest sequence's: tiles of 32, 64 and
# 128 columns
SHAPES = [([64], [160], 1, 8, 64, 32, 0), ([64, 5, 33], [2000, 5, 90], 2, 8, 64, 16, 0), ([70, 64], [300, 1700], 1, 8, 128, 256, 14),
          ([64, 130], [200, 400], 1, 8, 64, 256, 1024), ([64], [160], 1, 8, 256, 32, 0), ([100], [500], 1, 8, 256, 256, 16)]


@pytest.mark.parametrize("window", [1, 8, 19, 70])
@pytest.mark.parametrize("order", ["root first", "leaf first", "mixed"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s[0]}-{s[4]}-{s[6]}" for s in SHAPES])
def test_chains(shape, order, window):
    """Every node has one child, so that the deepest lie far behind, or far before, where their position is."""
    new, lens, kv, heads, dim, page, extra = shape
    batch = R.Batch(new, lens, kv, dim, page, "bf16", seed=window, extra_width=extra)
    compare(batch, heads, "bf16", order, window=window)


@pytest.mark.parametrize("order", ["leaf first", "mixed"])
@pytest.mark.parametrize("branch", [2, 9])
def test_trees(branch, order):
    for window in (0, 5, 33):
        batch = R.Batch([64, 1, 128, 33], [300, 1, 129, 1033], 2, 64, 16, "f16", seed=branch, lead=1, pad=2)
        compare(batch, 8, "f32", order, branch, window=window, cap=10.0, slopes=2.0 ** (-torch.arange(1, 9, dtype=torch.float32)))


@pytest.mark.parametrize("order", ["root first", "leaf first"])
@pytest.mark.parametrize("ahead", [40, 5000])
def test_positions_behind_the_length(ahead, order):
    """Nodes whose positions are past every place of the sequence: the window goes by the positions."""
    batch = R.Batch([64, 7], [200, 100], 1, 64, 16, "bf16", seed=ahead)
    compare(batch, 8, "bf16", order, ahead=ahead, window=30)


@pytest.mark.parametrize("order", ["root first", "leaf first", "mixed"])
def test_values_that_are_no_numbers(order):
    """In places that some nodes see and others do not: the nodes that do not are as if they were not there, also where
    the keys are gone through one by one."""
    batch = R.Batch([64], [160], 1, 64, 32, "bf16", seed=3)
    q = batch.normal(64, 8, 64)
    bits, depths = tree_in_order(batch.gen, [64], 1, order)
    tree = R.words_of(bits, 64, 0, 1)
    positions = torch.tensor([96 + d for d in depths], dtype=torch.int32)
    row = 96 + depths.index(40)                             # of the node at depth 40, which later ones see
    batch.v[batch.table[0, row // 32], :, row % 32, 5] = math.nan
    want, bound, _ = R.attention(batch, q, "bf16", tree=tree, positions=positions, window=8)
    got = qpg.cache_attention_tree(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), *batch.index(DEV), tree.to(DEV), positions.to(DEV),
                                   window=8).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and int(torch.isnan(want).any(dim=2).all(dim=1).sum()) == 8
    fine = ~torch.isnan(want)
    assert float(((got - want).abs() - bound)[fine].max()) <= 0


@pytest.mark.parametrize("window", [0, 9])
def test_more_nodes_than_the_length_says(window):
    """The first nodes have no place; the others are a tree of their own."""
    n, length = 40, 26
    batch = R.Batch([length], [length], 2, 64, 16, "f16", seed=window)
    q = batch.normal(n, 4, 64)
    bits, depths = tree_in_order(batch.gen, [length], 2, "mixed")
    tree = torch.zeros((n, 1), dtype=torch.int64)
    tree[n - length:] = R.words_of([x << (n - length) for x in bits], length, 0, 1)
    positions = torch.zeros(n, dtype=torch.int32)
    positions[n - length:] = torch.tensor(depths, dtype=torch.int32)
    want, bound, _ = R.attention(batch, q[n - length:], "f16", tree=R.words_of(bits, length, 0, 1), positions=positions[n - length:],
                                 window=window)
    offsets = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    got = qpg.cache_attention_tree(q.to(DEV), batch.k.to(DEV), batch.v.to(DEV), batch.table.to(DEV), batch.lens.to(DEV), offsets,
                                   tree.to(DEV), positions.to(DEV), window=window).cpu().double()
    assert bool((got[:n - length] == 0).all())
    assert float(((got[n - length:] - want).abs() - bound).max()) <= 0
