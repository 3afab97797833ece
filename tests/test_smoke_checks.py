"""What smoke() compares the paged cache's results with refuses every wrong one, a NaN among them (on the CPU, with results
of plain torch in the kernels' place)."""
import math

import pytest
import torch

import __graft_entry__ as entry


def results():
    gen = torch.Generator().manual_seed(1)
    heads, kv, dim, page, lens, new = 4, 2, 16, 8, [5, 19], [5, 1]
    table = torch.tensor([[5, 0, 3], [1, 2, 4]], dtype=torch.int32)
    kc, vc = torch.randn((2, 6, kv, page, dim), generator=gen).half()
    q = torch.randn((6, heads * dim), generator=gen)
    freqs = 10000.0 ** (-torch.arange(0, dim, 2) / dim)
    at = torch.tensor([0, 1, 2, 3, 4, 18])
    a, b = q.view(6, heads, -1, 2).unbind(dim=3)
    cos, sin = (f(at[:, None, None] * freqs) for f in (torch.cos, torch.sin))
    qr = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=3).reshape(6, heads, dim).half()
    y = torch.zeros((6, heads, dim))
    for row, (s, n) in enumerate([(0, 1), (0, 2), (0, 3), (0, 4), (0, 5), (1, 19)]):
        spot = torch.arange(n)
        keys, values = (c[table[s].long()[spot // page], :, spot % page].float() for c in (kc, vc))
        for h in range(heads):
            y[row, h] = torch.softmax(keys[:, h // 2] @ qr[row, h].float() / math.sqrt(dim), 0) @ values[:, h // 2]
    return [q, freqs, table, lens, new, kc, vc, qr, y]


def test_right_results_pass():
    assert entry.cache_error(*results()) <= 0


@pytest.mark.parametrize("what", [math.nan, math.inf, 7.0])
@pytest.mark.parametrize("at", ["queries", "outputs"])
@pytest.mark.parametrize("row", [0, 3, 5])
def test_wrong_results_do_not(row, at, what):
    args = results()
    args[7 if at == "queries" else 8][row, 2, 7] = what
    assert not entry.cache_error(*args) <= 0


def test_no_result_at_all():
    args = results()
    args[8][:] = math.nan
    assert not entry.cache_error(*args) <= 0
