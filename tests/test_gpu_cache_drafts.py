"""A step of drafting over a paged cache, as a user runs it: a prompt, a tree of drafts appended at the positions that
its nodes would have (the length before plus the depth) and attended to, then the accepted branch appended again. Every
node's queries, keys and attention are those of its branch appended as ordinary tokens."""
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"
HEADS, KV, DIM, PAGE = 8, 2, 64, 16


def index(table, lens, new):
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    return [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (table, lens, offsets)]


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("before", [1, 37])
def test_a_tree_is_its_branches(before, adjacent):
    gen = torch.Generator().manual_seed(before)
    parents = [-1, 0, 0, 1, 2, 2, 3, 6, 7]
    depth, path = [0] * 9, []
    for i, p in enumerate(parents):
        path.append((path[p] if i else []) + [i])
        depth[i] = len(path[i]) - 1
    x = [torch.randn((before + 9, n * DIM), generator=gen).to(DEV) for n in (HEADS, KV, KV)]
    kw = {"freqs": (10000.0 ** (-torch.arange(0, DIM, 2) / DIM)).to(DEV), "adjacent": adjacent}
    table = [[2, 0, 5]]
    prompt, drafts = [t[:before] for t in x], [t[before:] for t in x]

    def fresh():
        pair = [torch.zeros((6, KV, PAGE, DIM), dtype=torch.float16, device=DEV) for _ in range(2)]
        qpg.cache_append(*prompt, *pair, *index(table, [before], [before]), **kw)
        return pair

    tree = torch.tensor([sum(1 << m for m in p) for p in path], dtype=torch.int64, device=DEV).view(9, 1)
    positions = torch.tensor([before + d for d in depth], dtype=torch.int32, device=DEV)         # lens[b] - new[b] + depth
    kc, vc = fresh()
    at = index(table, [before + 9], [9])
    q = qpg.cache_append(*drafts, kc, vc, *at, positions=positions, **kw)
    y = {w: qpg.cache_attention_tree(q, kc, vc, *at, tree, positions, window=w, dtype=torch.float32) for w in (0, 3)}
    for i, p in enumerate(path):
        alone = fresh()
        at = index(table, [before + len(p)], [len(p)])
        qa = qpg.cache_append(*(t[p].contiguous() for t in drafts), *alone, *at, **kw)
        assert torch.equal(qa[-1], q[i])
        place, node = before + len(p) - 1, before + i
        for c, a in ((kc, alone[0]), (vc, alone[1])):
            assert torch.equal(c[table[0][node // PAGE], :, node % PAGE], a[table[0][place // PAGE], :, place % PAGE])
        for w in (0, 3):
            batch = R.Batch([len(p)], [before + len(p)], KV, DIM, PAGE, "f16")
            batch.table, batch.k, batch.v = torch.tensor(table, dtype=torch.int32), alone[0].cpu(), alone[1].cpu()
            want, bound, _ = R.attention(batch, qa.cpu(), "f32", window=w)
            ya = qpg.cache_attention(qa, *alone, *at, window=w, dtype=torch.float32).cpu().double()
            assert float(((ya - want).abs() - bound).max()) <= 0
            assert float(((y[w][i].cpu().double() - want[-1]).abs() - bound[-1]).max()) <= 0
    # the branch to node 8 is accepted: appended again, at its places, the cache is as if the others had never been
    best = path[8]
    at = index(table, [before + len(best)], [len(best)])
    qb = qpg.cache_append(*(t[best].contiguous() for t in drafts), kc, vc, *at, **kw)
    alone = fresh()
    assert torch.equal(qpg.cache_append(*(t[best].contiguous() for t in drafts), *alone, *at, **kw), qb)
    assert torch.equal(qpg.cache_attention(qb, kc, vc, *at), qpg.cache_attention(qb, *alone, *at))
