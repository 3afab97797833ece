"""The paged cache's operators over many sequences and many rows: batches whose sequence is found in three rounds of loads
and more, and as many rows as a call takes."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
qpg = pytest.importorskip("quantized_prefill_gemm_amd")
DEV = "cuda"
PAGE, DIM = 16, 8


def sequences(gen, B, most):
    """One page to a sequence, pages in no order; some sequences without new tokens; a row of none before and three behind."""
    lens = torch.randint(1, PAGE + 1, (B,), generator=gen, device=DEV)
    new = torch.minimum(torch.randint(0, most + 1, (B,), generator=gen, device=DEV), lens)
    offsets = torch.cat([torch.ones(1, dtype=torch.int64, device=DEV), 1 + torch.cumsum(new, 0)])
    table = torch.randperm(B, generator=gen, device=DEV)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), new)
    place = lens[seq] - new[seq] + torch.arange(len(seq), device=DEV) + 1 - offsets[seq]
    return table, lens, offsets, seq, place


@pytest.mark.parametrize("most", [1, 5])
@pytest.mark.parametrize("B", [63, 64, 4096, 4097, 70000, 300000])
def test_many_sequences(B, most):
    gen = torch.Generator(device=DEV).manual_seed(B)
    table, lens, offsets, seq, place = sequences(gen, B, most)
    n = len(seq)
    index = [t.to(torch.int32) for t in (table.view(B, 1), lens, offsets)]
    pools = [torch.randn((B, 1, PAGE, DIM), generator=gen, device=DEV).half() for _ in range(2)]
    k, v = (torch.randn((n + 4, DIM), generator=gen, device=DEV).half() for _ in range(2))
    q = torch.randn((n + 4, 2 * DIM), generator=gen, device=DEV).half()
    want = [p.clone() for p in pools]
    for w, x in zip(want, (k, v)):
        w[table[seq], 0, place] = x[1:1 + n]
    y = torch.full((n + 4, 2, DIM), 777.0, dtype=torch.float16, device=DEV)
    assert qpg.cache_append(q, k, v, *pools, *index, y=y) is y
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])               # copies: no norm, no rotation
    assert torch.equal(y[1:1 + n], q.view(-1, 2, DIM)[1:1 + n]) and bool((y[0] == 777).all()) and bool((y[1 + n:] == 777).all())
    out = torch.full((n + 4, 2, DIM), 777.0, device=DEV)
    qpg.cache_attention(y, *pools, *index, y=out)
    keys, values = (p[table[seq], 0].double() for p in pools)                              # [rows][page][dim]
    see = torch.arange(PAGE, device=DEV)[None, :] <= place[:, None]
    for h in range(2):
        qh = y[1:1 + n, h].double()
        s = (keys * qh[:, None, :]).sum(dim=2) / math.sqrt(DIM)
        off = (DIM + 16) * R.STEP * (keys.abs() * qh.abs()[:, None, :]).sum(dim=2) / math.sqrt(DIM)
        w = torch.softmax(torch.where(see, s, -math.inf), dim=1)
        exact, size = ((w[:, :, None] * x).sum(dim=1) for x in (values, values.abs()))
        worst = torch.where(see, off, 0.0).amax(dim=1, keepdim=True)
        bound = (2 * torch.expm1(worst) + (4 + 2 * PAGE + 64) * R.STEP) * size + PAGE * 2.0 ** -31 * values.abs().max() + R.STEP * exact.abs()
        assert float(((out[1:1 + n, h].double() - exact).abs() - bound).max()) <= 0
    assert bool((out[0] == 777).all()) and bool((out[1 + n:] == 777).all())


def test_as_many_rows_as_a_call_takes():
    """2^24 - 1 new tokens of 2^20 sequences. With queries of zeros a token's result is the mean of what it sees, and the values
    are their places in the sequence."""
    T, B = (1 << 24) - 1, 1 << 20
    offsets = torch.minimum(torch.arange(B + 1, device=DEV) * 16, torch.tensor(T, device=DEV)).to(torch.int32)
    lens = offsets[1:] - offsets[:-1]
    table = torch.arange(B - 1, -1, -1, dtype=torch.int32, device=DEV).view(B, 1)
    kc, vc = (torch.full((B, 1, PAGE, DIM), 9.0, dtype=torch.float16, device=DEV) for _ in range(2))
    place = (torch.arange(T, device=DEV) % 16).half()
    x = place[:, None].expand(T, DIM).contiguous()
    zeros = torch.zeros((T, DIM), dtype=torch.float16, device=DEV)
    q = qpg.cache_append(zeros, x, x, kc, vc, table, lens, offsets)
    want = torch.arange(16, device=DEV).half()[None, :].repeat(B, 1)
    want[0, 15] = 9.0                                       # the last sequence, of 15 tokens, has page 0
    assert all(bool((c[:, 0] == want[:, :, None]).all()) for c in (kc, vc)) and bool((q == 0).all())
    y = qpg.cache_attention(q, kc, vc, table, lens, offsets, dtype=torch.float32).view(T, DIM)
    # equal shares: sums of whole numbers, and one division
    assert float((y - place.float()[:, None] / 2).abs().max()) <= 2 * 2.0 ** -24 * 7.5
