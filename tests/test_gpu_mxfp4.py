"""MXFP4 quantisation and product on the GPU against their definition in 64 bits.

Codes and scale bytes are compared bit for bit (the scale is a power of two, the rounding rule
leaves no choice); products within the bound of mx_ref.product_bound.
"""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import mx_ref as R
from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
KINDS = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def values_of(which, rows, K, rng):
    x = rng.standard_normal((rows, K))
    if which == "wide":                      # every block its own magnitude, over most of f32
        x = x * np.exp2(rng.integers(-100, 100, (rows, K // 32)).repeat(32, axis=1).astype(np.float64))
    elif which == "tiny":                    # around and below the smallest normal f32
        x = x * np.exp2(rng.integers(-150, -118, (rows, K // 32)).repeat(32, axis=1).astype(np.float64))
    elif which == "halfway":                 # the points between two codes, and their neighbours
        pts = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 1.5, 3.0])
        x = rng.choice(pts, (rows, K)) * rng.choice([-1.0, 1.0], (rows, K))
        x[:, ::32] = 4.0                     # the block's exponent is 2: the scale is 1
        x = x * (1 + rng.integers(-1, 2, (rows, K)) * 2.0 ** -7)
    elif which == "zeros":
        x[:, : 32 * ((K // 32 + 1) // 2)] = 0.0
        x[0, 0] = -0.0
    elif which == "nonfinite":
        x[0, 5] = np.nan
        x[-1, K - 1] = np.inf
        x[rows // 2, K // 2] = -np.inf
    return x


@pytest.mark.parametrize("which", ["normal", "wide", "tiny", "halfway", "zeros", "nonfinite"])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 1056), (130, 2912), (33, 4096)])
def test_quantize_bits(which, kind, rows, K):
    rng = np.random.default_rng([rows, K, len(which)])
    with np.errstate(over="ignore"):
        x = torch.from_numpy(values_of(which, rows, K, rng).astype(np.float32)).to(KINDS[kind])
    if which != "nonfinite":
        x = torch.where(torch.isfinite(x), x, torch.ones_like(x))     # what overflowed in f16
    buf = B.quantize_mxfp4(x.to(DEV))
    want = R.pack(*R.encode(f64(x)))
    got = buf.cpu().numpy()
    assert got.shape == want.shape
    assert np.array_equal(got, want), np.flatnonzero(got != want)[:8]
    for out in KINDS:
        y = B.dequantize_mxfp4(buf, rows, K, dtype=KINDS[out]).cpu()
        exact = torch.from_numpy(R.values(want, rows, K))
        same = exact.to(KINDS[out])            # f64 -> the type: one rounding
        assert torch.equal(torch.nan_to_num(y.double(), nan=7e30), torch.nan_to_num(same.double(), nan=7e30)), out


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    buf = R.pack(codes, scales)
    exact = torch.from_numpy(R.values(buf, 256, 32))
    for kind, t in KINDS.items():
        y = B.dequantize_mxfp4(torch.from_numpy(buf).to(DEV), 256, 32, dtype=t).cpu()
        # the value is formed in f32 first: it is exact there up to 2^128, beyond it infinite
        want = exact.float().to(t)
        assert torch.equal(torch.nan_to_num(y.double(), nan=7e300), torch.nan_to_num(want.double(), nan=7e300)), kind


def product_case(M, N, K, seed, kind="float32", scale=0.02):
    rng = np.random.default_rng([seed, M, N, K])
    w = R.weights(N, K, rng, scale)
    x = rng.standard_normal((M, K)) * rng.uniform(0.25, 4.0, (M, 1))
    return w, torch.from_numpy(x.astype(np.float32)).to(KINDS[kind])


# Every form and its edges: rows around 16, 32, 64, 128 and 256, odd widths, K with whole and
# partial units, one block alone; one tile to a workgroup, and several (the last four).
SHAPES = [(1, 1, 32), (1, 4096, 4096), (2, 7, 96), (15, 100, 544), (16, 256, 512), (17, 33, 480), (31, 130, 1024),
          (33, 64, 1056), (48, 1000, 2912), (64, 512, 2048), (65, 129, 64), (100, 260, 992), (127, 384, 768),
          (129, 255, 1280), (200, 640, 2080), (257, 513, 1312), (512, 256, 256), (300, 1030, 4096), (700, 900, 2912),
          (200, 1500, 544), (190, 1600, 640), (200, 1501, 800), (513, 2050, 1024), (600, 2100, 288), (300, 40000, 320),
          (200, 1500, 32), (300, 1300, 96), (600, 2100, 64), (600, 2100, 256), (10, 20000, 288), (30, 40000, 480),
          (3000, 3100, 768), (4200, 4200, 544), (2600, 4097, 640), (2600, 4100, 128), (1100, 2101, 544), (2000, 2900, 1056),
          (1900, 2100, 32), (1100, 9000, 288), (4360, 4352, 288)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    say(f"[product {M} x {N} x {K}]")
    w, x = product_case(M, N, K, 1)
    wd = torch.from_numpy(w).to(DEV)
    xv, wv = R.decode(*R.encode(f64(x))), R.values(w, N, K)
    exact = xv @ wv.T
    for kind, t in KINDS.items():
        ws = torch.empty(B.mxfp4_bytes(M, K), dtype=torch.uint8, device=DEV)
        y = B.mmq_mxfp4(wd, x.to(DEV), N, xm_ws=ws, dtype=t)
        assert y.shape == (M, N) and y.dtype == t
        assert np.array_equal(ws.cpu().numpy(), R.pack(*R.encode(f64(x))))
        off = np.abs(f64(y) - exact) - R.product_bound(xv, wv, exact, kind)
        assert off.max() <= 0, (kind, off.max())
        again = B.mmq_mxfp4_mx(wd, ws, M, N, K, dtype=t)
        assert torch.equal(again, y), kind


@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (14, 60, 96), (40, 130, 512), (260, 258, 1056)])
def test_product_from_narrow_activations(M, N, K, kind):
    w, x = product_case(M, N, K, 2, kind)
    xv, wv = R.decode(*R.encode(f64(x))), R.values(w, N, K)
    exact = xv @ wv.T
    y = B.mmq_mxfp4(torch.from_numpy(w).to(DEV), x.to(DEV), N)
    assert (np.abs(f64(y) - exact) <= R.product_bound(xv, wv, exact, "float32")).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 1120), (40, 72, 1120), (200, 300, 1120), (250, 1400, 1120), (250, 1400, 896),
                                   (600, 2100, 1120), (3000, 3100, 640), (1100, 2100, 1120)])
def test_scales_of_any_size_and_nan(M, N, K):
    """Scale bytes over the whole range a product stays finite in, and NaN scales: a NaN block
    of x makes its row of y NaN, one of w its column, and nothing else."""
    rng = np.random.default_rng([7, M])
    xc, wc = rng.integers(0, 16, (M, K), dtype=np.uint8), rng.integers(0, 16, (N, K), dtype=np.uint8)
    xs, ws = rng.integers(80, 175, (M, K // 32), dtype=np.uint8), rng.integers(80, 175, (N, K // 32), dtype=np.uint8)
    xs[M - 1, K // 32 - 1] = 255
    xc[M - 1, -32:] = 0
    ws[N // 2, 0] = 255
    xb, wb = R.pack(xc, xs), R.pack(wc, ws)
    xv, wv = R.decode(xc, xs), R.decode(wc, ws)
    exact = xv @ wv.T
    y = f64(B.mmq_mxfp4_mx(torch.from_numpy(wb).to(DEV), torch.from_numpy(xb).to(DEV), M, N, K))
    assert np.isnan(exact[M - 1]).all() and np.isnan(exact[:, N // 2]).all()
    assert np.array_equal(np.isnan(y), np.isnan(exact))
    ok = ~np.isnan(exact)
    bound = R.product_bound(xv, wv, exact, "float32")
    assert (np.abs(y - exact)[ok] <= bound[ok]).all()


@pytest.mark.parametrize("M,N,K", [(5, 37, 160), (70, 131, 1056), (300, 257, 544), (300, 1301, 544), (601, 2100, 544),
                                   (3001, 3100, 544), (1101, 2100, 544), (4201, 4203, 160)])
def test_nothing_outside_the_outputs_is_written(M, N, K):
    w, x = product_case(M, N, K, 3)
    wd, xd = torch.from_numpy(w).to(DEV), x.to(DEV)
    for t in KINDS.values():
        room = torch.full((M * N + 512,), 5.0, dtype=t, device=DEV)
        y = room[257:257 + M * N].view(M, N)              # aligned to its element only
        B.mmq_mxfp4(wd, xd, N, y=y)
        assert torch.equal(y, B.mmq_mxfp4(wd, xd, N, dtype=t))
        assert bool((room[:257] == 5.0).all()) and bool((room[257 + M * N:] == 5.0).all())
    nb = B.mxfp4_bytes(M, K)
    room = torch.full((nb + 64,), 77, dtype=torch.uint8, device=DEV)
    B.quantize_mxfp4(xd, room[16:16 + nb])
    assert bool((room[:16] == 77).all()) and bool((room[16 + nb:] == 77).all())
    room = torch.full((M * K + 64,), 5.0, device=DEV)
    B.dequantize_mxfp4(B.quantize_mxfp4(xd), M, K, room[32:32 + M * K].view(M, K))
    assert bool((room[:32] == 5.0).all()) and bool((room[32 + M * K:] == 5.0).all())


@pytest.mark.parametrize("M,N,K", [(21, 50, 1056), (250, 1400, 1056), (250, 1400, 1152), (600, 2100, 1056), (1100, 2100, 1056),
                                   (2600, 4100, 1056)])
def test_operand_at_the_end_of_its_buffer(M, N, K):
    """The last rows' partial units: the result does not depend on what follows the operands
    (scale bytes of NaN right behind both planes)."""
    w, x = product_case(M, N, K, 4)
    wd, xd = torch.from_numpy(w).to(DEV), x.to(DEV)
    y = B.mmq_mxfp4(wd, xd, N)
    room = torch.full((w.size + 256,), 255, dtype=torch.uint8, device=DEV)
    room[: w.size] = wd
    xm = B.quantize_mxfp4(xd)
    roomx = torch.full((xm.numel() + 256,), 255, dtype=torch.uint8, device=DEV)
    roomx[: xm.numel()] = xm
    assert torch.equal(B.mmq_mxfp4_mx(room, roomx, M, N, K), y)


@pytest.mark.parametrize("M,N,K", [(1, 40, 1056), (4, 300, 480), (16, 33, 992), (16, 1000, 1024), (14, 2000, 1120)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_few_tokens_with_nan_and_infinity(M, N, K, kind):
    """From floats, a block with a NaN or an infinity makes its token's outputs NaN and no other's."""
    w, x = product_case(M, N, K, 8, kind)
    x[M - 1, K - 1] = float("inf")
    if M > 3:
        x[2, 33] = float("nan")
        x[0, :32] = 0
    wd, xd = torch.from_numpy(w).to(DEV), x.to(DEV)
    ws = torch.empty(B.mxfp4_bytes(M, K), dtype=torch.uint8, device=DEV)
    y = B.mmq_mxfp4(wd, xd, N, xm_ws=ws)
    assert torch.equal(ws, B.quantize_mxfp4(xd))
    lost = [m for m in range(M) if m == M - 1 or (M > 3 and m == 2)]
    kept = [m for m in range(M) if m not in lost]
    assert bool(torch.isnan(y[lost]).all()) and not bool(torch.isnan(y[kept]).any())
    assert torch.equal(y[kept], B.mmq_mxfp4_mx(wd, ws, M, N, K)[kept])


# Ones times powers of two: every sum is a multiple of the power below 2^24 times it, exact in f32.
@pytest.mark.parametrize("M,N,K", [(1, 40, 2 ** 24), (140, 2040, 2 ** 24), (1, 2 ** 24 + 40, 64), (20, 2 ** 24 + 40, 32),
                                   (2 ** 20 + 3, 520, 32)])
def test_longest_rows_and_widest_outputs(M, N, K):
    say(f"[product {M} x {N} x {K}]")
    def ones(rows):
        b = torch.full((B.mxfp4_bytes(rows, K),), 0x22, dtype=torch.uint8, device=DEV)
        power = torch.arange(rows, device=DEV) % 5
        b[rows * K // 2:].view(rows, K // 32).copy_((125 + power).to(torch.uint8)[:, None].expand(rows, K // 32))
        return b, torch.ldexp(torch.ones(rows, device=DEV), power.int() - 2)
    w, wp = ones(N)
    x, xp = ones(M)
    y = B.mmq_mxfp4_mx(w, x, M, N, K)
    assert bool((y == xp[:, None] * (wp * K)[None]).all())


def test_rows_past_32_bit_offsets():
    """Weights of more than 2^32 bytes."""
    N, K, M = 1_060_000, 8192, 2
    rng = np.random.default_rng(5)
    w = torch.empty(B.mxfp4_bytes(N, K), dtype=torch.uint8, device=DEV)
    w[: N * K // 2].random_(0, 256)
    w[N * K // 2:].random_(110, 130)
    assert N * K // 2 > 2 ** 32
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DEV)
    y = B.mmq_mxfp4(w, x, N)
    xv = R.decode(*R.encode(f64(x)))
    for at in (0, 1_048_570, N - 16):                           # rows before, around and behind 2^32 bytes
        rows = torch.cat([w[at * K // 2:(at + 16) * K // 2], w[N * K // 2 + at * K // 32:N * K // 2 + (at + 16) * K // 32]])
        wv = R.values(rows.cpu().numpy(), 16, K)
        exact = xv @ wv.T
        assert (np.abs(f64(y[:, at:at + 16]) - exact) <= R.product_bound(xv, wv, exact, "float32")).all(), at


def test_refusals():
    x = torch.zeros((4, 64), device=DEV)
    w = torch.zeros(B.mxfp4_bytes(8, 64), dtype=torch.uint8, device=DEV)
    for bad in (lambda: B.quantize_mxfp4(torch.zeros((4, 48), device=DEV)),
                lambda: B.quantize_mxfp4(torch.zeros((0, 64), device=DEV)),
                lambda: B.quantize_mxfp4(x.double()),
                lambda: B.quantize_mxfp4(x.cpu()),
                lambda: B.quantize_mxfp4(x.t()),
                lambda: B.quantize_mxfp4(x[:, :32]),
                lambda: B.quantize_mxfp4(x, torch.empty(8, dtype=torch.uint8, device=DEV)),
                lambda: B.dequantize_mxfp4(w, 9, 64),
                lambda: B.dequantize_mxfp4(w, 8, 64, dtype=torch.int32),
                lambda: B.mmq_mxfp4(w, x, 9),
                lambda: B.mmq_mxfp4(w, x, 8, y=torch.empty((4, 7), device=DEV)),
                lambda: B.mmq_mxfp4(w, x, 8, dtype=torch.float64),
                lambda: B.mmq_mxfp4(w.cpu(), x, 8),
                lambda: B.mmq_mxfp4(w, x, 8, xm_ws=torch.empty(8, dtype=torch.uint8, device=DEV)),
                lambda: B.mmq_mxfp4_mx(w, w, 9, 8, 64)):
        with pytest.raises(B.QPGError):
            bad()
    with pytest.raises(B.QPGError) as e:                        # 4-byte aligned activations
        B.quantize_mxfp4(torch.zeros(4 * 64 + 1, device=DEV)[1:].view(4, 64))
    assert e.value.status == B.QPG_EALIGN


def test_streams_and_graph():
    """The same product on the current stream, on two other streams at once, and captured and
    replayed with new activations between the replays."""
    cases = [product_case(m, n, k, 6) for m, n, k in ((3, 1024, 2048), (150, 700, 1056))]
    dev = [(torch.from_numpy(w).to(DEV), x.to(DEV), n) for (w, x), n in zip(cases, (1024, 700))]
    want = [B.mmq_mxfp4(w, x, n) for w, x, n in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        got = [B.mmq_mxfp4(w, x, n, stream=streams[(i + rep) % 2]) for i, (w, x, n) in enumerate(dev)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for w, x, n in dev:
        xin, y = x.clone(), torch.empty((x.shape[0], n), device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.mmq_mxfp4(w, xin, n, y=y)
        for rep in range(3):
            xin.copy_(x * (rep + 1.5))
            y.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, B.mmq_mxfp4(w, xin, n)), rep
