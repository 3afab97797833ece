"""The MXFP4 product where workgroups walk from tile to tile, and scale bytes of NaN in every form
of the experts' product, against 64 bits (torch on the GPU, from the formulas of mx_ref)."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import mx_ref as R
from mx_walks import DENSE, EVERY, EXPERTS
from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
KINDS = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def random_mx(rows, K, gen, low=116, high=122):
    """Any codes, scale bytes of [low, high)."""
    b = torch.randint(0, 256, (B.mxfp4_bytes(rows, K),), dtype=torch.uint8, device=DEV, generator=gen)
    b[rows * K // 2:] = torch.randint(low, high, (rows * K // 32,), device=DEV, generator=gen).to(torch.uint8)
    return b


def values(buf, rows, K):
    """mx_ref.values on the GPU."""
    p = buf[:rows * K // 2].view(rows, K // 2).long()
    codes = torch.stack([p & 15, p >> 4], dim=2).view(rows, K)
    grid = torch.from_numpy(np.concatenate([R.GRID, -R.GRID])).to(DEV)
    power = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [float("nan")], dtype=torch.float64, device=DEV)
    return grid[codes] * power[buf[rows * K // 2:rows * K // 2 + rows * K // 32].view(rows, K // 32).long()].repeat_interleave(32, 1)


def check(y, x, w, kind, where):
    """y against x w^T within mx_ref.product_bound; NaN exactly where that has it."""
    exact = x @ w.T
    rel, least = R.HALF[kind]
    bound = (x.shape[1] / 64 + 9) * 2.0 ** -23 * (x.abs() @ w.abs().T) + 1.0001 * (exact.abs() * rel + least)
    lost = torch.isnan(exact)
    assert torch.equal(torch.isnan(y), lost), where
    assert bool(((y.double() - exact).abs() <= bound)[~lost].all()), where


def layout(counts, dropped, top_k, gen):
    """ids [T, top_k] in which expert e is chosen counts[e] times and `dropped` choices are -1."""
    ids = torch.cat([torch.full((c,), e) for e, c in enumerate(counts)] + [torch.full((dropped,), -1)])
    return ids[torch.randperm(ids.numel(), generator=gen)].view(-1, top_k)


def run_experts(case, kinds, spoil=False):
    form, counts, dropped, top_k, N, K = case
    say(f"[experts {form} {counts} + {dropped}, {N} x {K}]")
    gen = torch.Generator(device=DEV).manual_seed(N + K)
    ids = layout(counts, dropped, top_k, torch.Generator().manual_seed(K))
    T, E, S = ids.shape[0], len(counts), ids.numel()
    offsets, order, _ = (torch.from_numpy(a).to(DEV) for a in R.sort(ids.numpy(), E))
    n = int(offsets[-1])
    w, x = random_mx(E * N, K, gen), random_mx(T, K, gen)
    if spoil:
        # the last row of every second expert, its last block; the first row of one expert's matrix and the
        # last of another's: what a tile's padding and the neighbouring expert have beside them
        xs, ws = x[T * K // 2:].view(T, K // 32), w[E * N * K // 2:].view(E, N, K // 32)
        last = [int(offsets[e + 1]) - 1 for e in range(0, E, 2) if counts[e]]
        xs[order[last].long() // top_k, -1] = 255
        ws[1, 0, 0] = 255
        ws[E - 2, N - 1, K // 32 - 1] = 255
    xv = values(x, T, K)
    # activations in sorted order: the same rows
    at = (order.clamp(min=0) // top_k).long()
    codes, scales = x[:T * K // 2].view(T, -1), x[T * K // 2:].view(T, -1)
    xsorted = torch.cat([codes[at].reshape(-1), scales[at].reshape(-1)])
    wc, wsc = w[:E * N * K // 2].view(E, -1), w[E * N * K // 2:].view(E, -1)
    wv = [values(torch.cat([wc[e], wsc[e]]), N, K) for e in range(E)]
    for kind in kinds:
        room = torch.full((S + 2, N), 5.0, dtype=KINDS[kind], device=DEV)
        y = B.mmq_mxfp4_experts(w, x, T, offsets, order, top_k, E, N, K, y=room[1:-1])
        assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all()) and bool((y[n:] == 5.0).all()), kind
        for e in range(E):
            rows = slice(int(offsets[e]), int(offsets[e + 1]))
            check(y[rows], xv[at[rows]], wv[e], kind, (kind, e))
        ys = B.mmq_mxfp4_experts(w, xsorted, S, offsets, None, 1, E, N, K, y=torch.full_like(y, 5.0))
        assert torch.equal(torch.nan_to_num(ys, nan=7.0), torch.nan_to_num(y, nan=7.0)), kind


@pytest.mark.parametrize("form,M,N,K", DENSE)
def test_dense_walks(form, M, N, K):
    say(f"[{form} {M} x {N} x {K}]")
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    w, x = random_mx(N, K, gen), random_mx(M, K, gen)
    xv, wv = values(x, M, K), values(w, N, K)
    for kind, t in KINDS.items():
        room = torch.full((M + 2, N), 5.0, dtype=t, device=DEV)
        y = B.mmq_mxfp4_mx(w, x, M, N, K, y=room[1:-1])
        assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all()), kind
        check(y, xv, wv, kind, kind)


@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: f"{c[0]}-{c[4]}-{c[5]}")
def test_experts_walks(case):
    run_experts(case, list(KINDS))


@pytest.mark.parametrize("case", EVERY, ids=lambda c: c[0])
def test_nan_scales_of_experts(case):
    run_experts(case, ["float32", "bfloat16"], spoil=True)
