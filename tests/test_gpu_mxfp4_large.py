"""Products with more tiles than one row of a grid holds: activations of 2^32 bytes of codes for
experts, outputs of more than 2^33 values, one token against more than 2^29 rows. Every value is a
power of two that differs from row to row, so every sum is exact and the outputs are compared for
equality."""
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def powers(rows, step):
    """Exponents in [-11, 11], neighbouring rows apart."""
    return (torch.arange(rows, device=DEV) * step % 23 - 11).int()


def ones(rows, K, step):
    """Rows of 2^powers, as MXFP4 and in f32."""
    power = powers(rows, step)
    b = torch.full((B.mxfp4_bytes(rows, K),), 0x22, dtype=torch.uint8, device=DEV)
    b[rows * K // 2:].view(rows, K // 32).copy_((power + 127).to(torch.uint8)[:, None].expand(rows, K // 32))
    return b, torch.ldexp(torch.ones(rows, device=DEV), power)


@pytest.mark.parametrize("gathered", [True, False])
def test_experts_activations_of_4_gib(gathered):
    T, E, N, K = 2 ** 23, 8, 1024, 1024
    say(f"[experts {T} of {E}, {N} x {K}, gathered {gathered}]")
    gen = torch.Generator(device=DEV).manual_seed(4)
    ids = torch.randint(0, E, (T, 1), generator=gen, device=DEV)
    offsets, order, _ = B.experts_sort(ids, E)
    w, wp = ones(E * N, K, 7)
    x, xp = ones(T, K, 5)
    wp = wp.view(E, N)
    y = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    B.mmq_mxfp4_experts(w, x, T, offsets, order if gathered else None, 1, E, N, K, y=y)
    row = order.long() if gathered else torch.arange(T, device=DEV)
    expert = ids.view(-1)[order.long()]
    for at in range(0, T, 2 ** 18):
        part = slice(at, at + 2 ** 18)
        assert bool((y[part].float() == xp[row[part], None] * wp[expert[part]] * K).all()), at


def test_many_tokens_of_a_very_wide_matrix():
    M, N, K = 520, 2 ** 24 + 40, 32
    say(f"[product {M} x {N} x {K}]")
    w, wp = ones(N, K, 7)
    xp = torch.ldexp(torch.ones(M, device=DEV), powers(M, 5))
    x = xp[:, None].expand(M, K).contiguous()
    ws = torch.empty(B.mxfp4_bytes(M, K), dtype=torch.uint8, device=DEV)
    y = B.mmq_mxfp4(w, x, N, xm_ws=ws, dtype=torch.bfloat16)
    assert torch.equal(ws, B.quantize_mxfp4(x))
    for at in range(0, M, 40):
        assert bool((y[at:at + 40].float() == xp[at:at + 40, None] * (wp * K)[None]).all()), at


def test_one_token_against_very_many_rows():
    N, K = 2 ** 29 + 48, 32
    say(f"[product 1 x {N} x {K}]")
    w, wp = ones(N, K, 7)
    x, xp = ones(1, K, 5)
    assert bool((B.mmq_mxfp4_mx(w, x, 1, N, K)[0] == wp * (xp * K)).all())
