"""Sort by expert, gather, the experts' product, the weighted sum and the gradients on the GPU
against their definitions in 64 bits. Index arrays and moved rows are compared for equality."""
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


def routing(T, top_k, E, rng, how="uniform"):
    if how == "one":
        return np.full((T, top_k), E - 1)
    if how == "none":
        return np.full((T, top_k), -1)
    ids = rng.integers(0, E, (T, top_k))
    if how == "skew":
        ids = np.minimum(ids, rng.integers(0, E, (T, top_k)) // 3)
    if how == "drop":
        ids = np.where(rng.random((T, top_k)) < 0.3, rng.choice([-1, E, -7, E + 1000], (T, top_k)), ids)
    return ids


@pytest.mark.parametrize("T,top_k,E,how", [
    (1, 1, 1, "uniform"), (1, 8, 3, "uniform"), (7, 3, 61, "drop"), (64, 1, 64, "uniform"), (65, 2, 128, "skew"),
    (500, 4, 129, "drop"), (1024, 8, 1024, "uniform"), (1025, 8, 1000, "drop"), (4097, 2, 8, "skew"), (30, 5, 9, "none"),
    (3000, 3, 256, "one"), (40_000, 8, 257, "skew"), (100_001, 3, 1024, "drop")])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, top_k, E, how, dtype):
    rng = np.random.default_rng([T, top_k, E])
    ids = routing(T, top_k, E, rng, how)
    got = B.experts_sort(torch.from_numpy(ids).to(dtype).to(DEV), E)
    for name, g, w in zip(("offsets", "order", "slots"), got, R.sort(ids, E)):
        assert g.dtype == torch.int32 and tuple(g.shape) == w.shape
        assert np.array_equal(g.cpu().numpy(), w), name


def test_sort_of_far_ids():
    """int64 ids whose low 32 bits are an expert's number are no expert of the call."""
    ids = np.array([[2 ** 32 + 1, 1], [-2 ** 32, 0], [2 ** 62, -2 ** 63]])
    got = B.experts_sort(torch.from_numpy(ids).to(DEV), 4)
    for g, w in zip(got, R.sort(ids, 4)):
        assert np.array_equal(g.cpu().numpy(), w)


ROWS = [(1, 1, 1, 1, "uniform"), (1, 4, 8, 4096, "uniform"), (7, 3, 61, 2050, "drop"), (5, 2, 4, 33, "skew"),
        (130, 8, 16, 1032, "drop"), (300, 1, 7, 520, "uniform"), (40, 9, 12, 4096, "drop"), (12, 2, 3, 100, "none"),
        (64, 4, 32, 7168, "skew")]


@pytest.mark.parametrize("T,top_k,E,H,how", ROWS)
@pytest.mark.parametrize("kind", list(KINDS))
def test_gather_and_gradient(T, top_k, E, H, how, kind):
    rng = np.random.default_rng([T, H])
    ids = routing(T, top_k, E, rng, how)
    _, order, slots = R.sort(ids, E)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(KINDS[kind])
    sd = torch.from_numpy(slots).to(DEV)
    room = torch.full((T * top_k * H + 64,), 5.0, dtype=KINDS[kind], device=DEV)
    xs = room[32:32 + T * top_k * H].view(T * top_k, H)
    assert B.experts_gather(x.to(DEV), sd, xs) is xs
    n = int((order >= 0).sum())
    assert torch.equal(xs[:n].cpu(), x[torch.from_numpy(order[:n].astype(np.int64) // top_k)])
    assert bool((xs[n:] == 5.0).all()) and bool((room[:32] == 5.0).all()) and bool((room[-32:] == 5.0).all())

    dxs = rng.standard_normal((T * top_k, H)).astype(np.float32)
    dxs[n:] = np.nan                                             # rows of no slot are not read
    d = torch.from_numpy(dxs).to(KINDS[kind])
    dx = B.experts_gather_grad(d.to(DEV), sd)
    v = np.where(slots[:, :, None] >= 0, f64(d)[np.maximum(slots, 0)], 0.0)
    exact, mag = v.sum(axis=1), np.abs(v).sum(axis=1)
    assert dx.dtype == KINDS[kind]
    assert (np.abs(f64(dx) - exact) <= top_k * 2.0 ** -24 * mag + 1.0001 * R.rounding(exact, kind) + 2.0 ** -140).all()


@pytest.mark.parametrize("T,top_k,E,H,how", ROWS)
@pytest.mark.parametrize("ys_kind,y_kind", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                            ("float16", "float32"), ("bfloat16", "float16")])
def test_combine_and_gradients(T, top_k, E, H, how, ys_kind, y_kind):
    """Bounds: the weighted sum adds top_k f32 products, one rounding each for product and sum
    (2 * top_k * 2^-24 of the magnitudes); a dot over H takes, in each of 256 threads, at most
    ceil(H / 256) + 8 of them in turn, and 8 more join lanes and waves."""
    rng = np.random.default_rng([T, H, 1])
    ids = routing(T, top_k, E, rng, how)
    _, order, slots = R.sort(ids, E)
    n = int((order >= 0).sum())
    ys = rng.standard_normal((T * top_k, H)).astype(np.float32)
    ys[n:] = np.nan
    ys = torch.from_numpy(ys).to(KINDS[ys_kind])
    w = rng.standard_normal((T, top_k)).astype(np.float32)
    dy = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(KINDS[y_kind])
    sd, wd = torch.from_numpy(slots).to(DEV), torch.from_numpy(w).to(DEV)
    y = B.experts_combine(ys.to(DEV), sd, wd, dtype=KINDS[y_kind])
    assert y.dtype == KINDS[y_kind]
    on = slots[:, :, None] >= 0
    v = np.where(on, f64(ys)[np.maximum(slots, 0)], 0.0)
    terms = v * w.astype(np.float64)[:, :, None]
    exact, mag = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    bound = top_k * 2.0 ** -23 * mag
    assert (np.abs(f64(y) - exact) <= bound + 1.001 * R.rounding(exact, y_kind) + 2.0 ** -140).all()

    room = torch.full((T * top_k + 2, H), 5.0, dtype=KINDS[ys_kind], device=DEV)
    dys, dw = B.experts_combine_grad(dy.to(DEV), ys.to(DEV), sd, wd, dys=room[1:-1])
    assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all()) and bool((dys[n:] == 5.0).all())
    g = f64(dy)
    want = g[order[:n] // top_k] * w.astype(np.float64).reshape(-1)[order[:n]][:, None]
    # one f32 rounding of the product, then the stored type's
    assert (np.abs(f64(dys[:n]) - want) <= 2.0 ** -24 * np.abs(want) + 1.001 * R.rounding(want, ys_kind) + 2.0 ** -140).all()
    dots = v * g[:, None, :]
    exact, mag = dots.sum(axis=2), np.abs(dots).sum(axis=2)
    steps = -(-H // 256) + 16
    assert (np.abs(f64(dw) - exact) <= steps * 2.0 ** -23 * mag + 2.0 ** -140).all()
    assert (f64(dw)[slots < 0] == 0).all()


def test_gradients_against_differences():
    """<dy, combine(ys + h u, w + h v) - combine(ys - h u, w - h v)> / 2h is the gradients' product
    with (u, v): the sum is bilinear, so in 64 bits the difference is exact for h = 1; the kernel's
    gradients are within their f32 roundings of it."""
    rng = np.random.default_rng(11)
    T, top_k, E, H = 9, 3, 5, 264
    ids = routing(T, top_k, E, rng, "drop")
    _, order, slots = R.sort(ids, E)
    ys, u = rng.standard_normal((2, T * top_k, H)).astype(np.float32)
    w, v = rng.standard_normal((2, T, top_k)).astype(np.float32)
    dy = rng.standard_normal((T, H)).astype(np.float32)

    def combine(a, b):
        rows = np.where(slots[:, :, None] >= 0, a.astype(np.float64)[np.maximum(slots, 0)], 0.0)
        return (rows * b.astype(np.float64)[:, :, None]).sum(axis=1)

    u64, v64 = u.astype(np.float64), v.astype(np.float64)
    diff = (dy * (combine(ys + u64, w + v64) - combine(ys - u64, w - v64))).sum() / 2
    dev = [torch.from_numpy(a).to(DEV) for a in (dy, ys, slots, w)]
    dys, dw = B.experts_combine_grad(*dev, dys=torch.zeros((T * top_k, H), device=DEV))
    got = (f64(dys) * u).sum() + (f64(dw) * v).sum()
    size = np.abs(f64(dys) * u).sum() + (np.abs(v) * 18 * np.abs(dy).sum(axis=1)[:, None] * np.abs(ys).max()).sum()
    assert abs(got - diff) <= 2.0 ** -23 * size

    x, p = rng.standard_normal((2, T, H)).astype(np.float32)
    g = rng.standard_normal((T * top_k, H)).astype(np.float32)
    n = int((order >= 0).sum())
    g[n:] = 0
    move = np.zeros((T * top_k, H))
    move[:n] = p[order[:n] // top_k]
    dx = B.experts_gather_grad(torch.from_numpy(g).to(DEV), dev[2])
    assert abs((f64(dx) * p).sum() - (g * move).sum()) <= 2.0 ** -22 * np.abs(g[:n] * move[:n]).sum()


PRODUCTS = [(1, 1, 1, 1, 32, "uniform"), (4, 4, 32, 300, 1056, "uniform"), (3, 2, 8, 17, 96, "drop"),
            (40, 2, 3, 130, 544, "skew"), (64, 1, 4, 64, 512, "one"), (200, 2, 4, 260, 992, "drop"), (9, 3, 5, 50, 64, "none"),
            (700, 2, 5, 200, 1312, "skew"), (600, 1, 2, 513, 768, "drop"), (100, 4, 200, 48, 160, "uniform"),
            (1500, 1, 4, 1400, 544, "skew"), (3000, 2, 3, 2100, 768, "drop"), (2500, 2, 3, 2500, 640, "skew"),
            (300, 2, 40, 300, 800, "uniform"), (4, 4, 32, 1100, 1056, "drop"), (200, 2, 12, 3000, 288, "uniform"),
            (3000, 2, 3, 4200, 544, "drop"), (2300, 2, 7, 2304, 160, "uniform")]


@pytest.mark.parametrize("T,top_k,E,N,K,how", PRODUCTS)
def test_experts_product(T, top_k, E, N, K, how):
    say(f"[experts {T} x {top_k} of {E}, {N} x {K}, {how}]")
    rng = np.random.default_rng([T, E, N])
    ids = routing(T, top_k, E, rng, how)
    offsets, order, slots = R.sort(ids, E)
    n, S = int(offsets[-1]), T * top_k
    w = R.weights(E * N, K, rng)
    x = rng.standard_normal((T, K)).astype(np.float32)
    xv, wv = R.decode(*R.encode(x)), R.values(w, E * N, K).reshape(E, N, K)
    xm = torch.from_numpy(R.pack(*R.encode(x))).to(DEV)
    expert = np.repeat(np.arange(E), np.diff(offsets))
    wd = torch.from_numpy(w).to(DEV)
    od, rd = torch.from_numpy(offsets).to(DEV), torch.from_numpy(order).to(DEV)
    exact = np.zeros((S, N))
    bound = {k: np.zeros((S, N)) for k in KINDS}
    for e in range(E):
        rows = np.flatnonzero(expert == e)
        if rows.size:
            xe = xv[order[rows] // top_k]
            exact[rows] = xe @ wv[e].T
            for k in KINDS:
                bound[k][rows] = R.product_bound(xe, wv[e], exact[rows], k)
    for kind, t in KINDS.items():
        room = torch.full((S + 2, N), 5.0, dtype=t, device=DEV)
        y = B.mmq_mxfp4_experts(wd, xm, T, od, rd, top_k, E, N, K, y=room[1:-1])
        assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all()) and bool((y[n:] == 5.0).all())
        assert (np.abs(f64(y[:n]) - exact[:n]) <= bound[kind][:n]).all(), kind
        # activations already in sorted order
        xs = np.zeros((S, K), dtype=np.float32)
        xs[:n] = x[order[:n] // top_k]
        ys = torch.full((S, N), 5.0, dtype=t, device=DEV)
        B.mmq_mxfp4_experts(wd, B.quantize_mxfp4(torch.from_numpy(xs).to(DEV)), S, od, None, 1, E, N, K, y=ys)
        assert torch.equal(ys, y), kind


def test_wrong_arrays_stay_inside_the_buffers():
    """Index arrays that are none: the kernels clamp or drop what they read, so nothing outside
    the outputs is written and the call ends; the rows themselves are unspecified."""
    rng = np.random.default_rng(3)
    T, top_k, E, N, K, H = 20, 2, 6, 40, 96, 64
    S = T * top_k
    wild = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (S,)).astype(np.int32)).to(DEV)
    w = torch.from_numpy(R.weights(E * N, K, rng)).to(DEV)
    xm = torch.from_numpy(R.weights(T, K, rng)).to(DEV)
    for off in ([0, 5, 3, 100, -4, 60, 2 ** 31 - 1], [-2 ** 31] * 7, [2 ** 31 - 1] * 7, [40, 30, 20, 10, 0, 0, 40]):
        offsets = torch.tensor(off, dtype=torch.int64).to(torch.int32).to(DEV)
        room = torch.full((S + 2, N), 5.0, device=DEV)
        B.mmq_mxfp4_experts(w, xm, T, offsets, wild, top_k, E, N, K, y=room[1:-1])
        torch.cuda.synchronize()
        assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all())
    # ranges of experts that overlap, in the tiled forms: more tiles than rows stand for
    for T2, N2 in ((700, 600), (1500, 1400), (2500, 2500)):
        S2 = T2 * 2
        w2 = torch.from_numpy(R.weights(4 * N2, K, rng)).to(DEV)
        xm2 = torch.from_numpy(R.weights(T2, K, rng)).to(DEV)
        order = torch.arange(S2 - 1, -1, -1, dtype=torch.int32, device=DEV)
        for off in ([0, S2, 0, S2, 0], [5, 2 ** 31 - 1, -9, S2, S2]):
            room = torch.full((S2 + 2, N2), 5.0, device=DEV)
            B.mmq_mxfp4_experts(w2, xm2, T2, torch.tensor(off, dtype=torch.int32, device=DEV), order, 2, 4, N2, K,
                                y=room[1:-1])
            torch.cuda.synchronize()
            assert bool((room[0] == 5.0).all()) and bool((room[-1] == 5.0).all())
    # slots: out of range counts as no row
    slots = torch.full((T, top_k), -1, dtype=torch.int32, device=DEV)
    slots[0, 0], slots[1, 1], slots[2, 0] = S, 2 ** 31 - 1, -2 ** 31
    x, ws = torch.ones((T, H), device=DEV), torch.ones((T, top_k), device=DEV)
    room = torch.full((S + 2, H), 5.0, device=DEV)
    B.experts_gather(x, slots, room[1:-1])
    ys = torch.full((S, H), float("nan"), device=DEV)
    assert bool((B.experts_combine(ys, slots, ws) == 0).all())
    dys, dw = B.experts_combine_grad(x, ys, slots, ws, dys=room[1:-1])
    assert bool((room == 5.0).all()) and bool((dw == 0).all())


def layer(ids, x, w, wts, E, N, K, dtype):
    """The operators as a layer uses them."""
    offsets, order, slots = B.experts_sort(ids, E)
    ys = B.mmq_mxfp4_experts(w, B.quantize_mxfp4(x), x.shape[0], offsets, order, ids.shape[1], E, N, K)
    return B.experts_combine(ys, slots, wts, dtype=dtype)


@pytest.mark.parametrize("T,top_k,E,N,K,how", [(5, 2, 8, 96, 256, "drop"), (150, 3, 6, 200, 480, "skew"),
                                               (400, 2, 4, 700, 1056, "drop")])
def test_operators_together_and_in_a_graph(T, top_k, E, N, K, how):
    """Sort, quantise, product and weighted sum in one run against 64 bits; on two streams at
    once; captured, and replayed with other routings and activations, eager work in between."""
    rng = np.random.default_rng([T, 5])
    w = R.weights(E * N, K, rng)
    wv = R.values(w, E * N, K).reshape(E, N, K)
    wd = torch.from_numpy(w).to(DEV)

    def inputs():
        return (torch.from_numpy(routing(T, top_k, E, rng, how)).to(DEV),
                torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(DEV),
                torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV))

    ids, x, wts = inputs()
    y = layer(ids, x, wd, wts, E, N, K, torch.float32)
    xv = R.decode(*R.encode(f64(x)))
    exact, bound = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(top_k):
            e = int(ids[t, j])
            if 0 <= e < E:
                one = xv[t:t + 1] @ wv[e].T
                exact[t] += float(wts[t, j]) * one[0]
                bound[t] += abs(float(wts[t, j])) * (R.product_bound(xv[t:t + 1], wv[e], one, "float32")[0]
                                                     + (top_k + 1) * 2.0 ** -23 * np.abs(one[0]))
    assert (np.abs(f64(y) - exact) <= bound + R.rounding(exact, "float32")).all()

    other = inputs()
    want = [y, layer(other[0], other[1], wd, other[2], E, N, K, torch.float32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, (i, a, b) in zip(streams, ((ids, x, wts), other)):
        with torch.cuda.stream(s):
            got.append(layer(i, a, wd, b, E, N, K, torch.float32))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    si, sx, sw = ids.clone(), x.clone(), wts.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(si, sx, wd, sw, E, N, K, torch.float32)
    for rep in range(4):
        i, a, b = inputs()
        si.copy_(i); sx.copy_(a); sw.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer(i, a, wd, b, E, N, K, torch.float32)), rep


@pytest.mark.parametrize("T,top_k,E,H,kind", [(3, 2, 4, 40, "float32"), (2100, 3, 40, 520, "bfloat16"),
                                              (700, 9, 8, 1001, "float16")])
def test_training_operators_in_a_graph_and_on_a_stream(T, top_k, E, H, kind):
    """Sort (with its workspace), gather, weighted sum and all gradients: on two streams at once, and
    captured and replayed with other routings and values, against the calls one by one."""
    rng = np.random.default_rng([T, 6])

    def inputs():
        return (torch.from_numpy(routing(T, top_k, E, rng, "drop")).to(DEV),
                torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(KINDS[kind]).to(DEV),
                torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV))

    def chain(ids, x, wts, ws, stream=None):
        with torch.cuda.stream(stream):                          # rows that no choice has: zeros
            xs, dys = torch.zeros((2, T * top_k, H), dtype=x.dtype, device=DEV)
        offsets, order, slots = B.experts_sort(ids, E, ws=ws, stream=stream)
        B.experts_gather(x, slots, xs, stream=stream)
        y = B.experts_combine(xs, slots, wts, stream=stream)
        _, dw = B.experts_combine_grad(y, xs, slots, wts, dys=dys, stream=stream)
        dx = B.experts_gather_grad(dys, slots, stream=stream)
        return [offsets, order, slots, xs, y, dys, dw, dx]

    def workspace():
        return torch.empty(B.experts_sort_bytes(T * top_k, E) + 4, dtype=torch.uint8, device=DEV)

    pair = [inputs(), inputs()]
    want = [chain(*a, workspace()) for a in pair]
    spaces = [workspace(), workspace()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for rep in range(3):
        got = [chain(*a, ws, stream=streams[(i + rep) % 2]) for i, (a, ws) in enumerate(zip(pair, spaces))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b)), rep

    held, ws = [t.clone() for t in pair[0]], workspace()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(*held, ws)
    for rep in range(4):
        new = inputs()
        for t, n in zip(held, new):
            t.copy_(n)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, chain(*new, workspace()))), rep


@pytest.mark.parametrize("T,top_k,E,H,kind", [(2 ** 24 - 1, 1, 1024, 1, "float32"), (1, 2, 3, 2 ** 26 + 1, "float16"),
                                              (2, 300, 5, 70_001, "bfloat16")])
def test_many_tokens_long_rows_and_many_choices(T, top_k, E, H, kind):
    """Small whole numbers: every product and sum is exact (f32 holds those below 2^24, the 16-bit
    types those below 2^8)."""
    say(f"[rows {T} x {top_k} of {E}, H {H}]")
    gen = torch.Generator(device=DEV).manual_seed(T)
    def whole(shape, below, dtype):
        return torch.randint(-below, below + 1, shape, generator=gen, device=DEV).to(dtype)
    ids = torch.randint(-1, E, (T, top_k), generator=gen, device=DEV)
    offsets, order, slots = B.experts_sort(ids, E)
    n, S = int(offsets[-1]), T * top_k
    assert n == int((ids >= 0).sum())
    at = order[:n].long()
    sorted_ids = ids.view(-1)[at]
    assert bool((slots.view(-1)[at] == torch.arange(n, device=DEV)).all()) and bool((sorted_ids.diff() >= 0).all())
    assert bool((at.diff()[sorted_ids.diff() == 0] > 0).all()) and bool((order[n:] == -1).all())
    x = whole((T, H), 100, KINDS[kind])
    xs = torch.zeros((S, H), dtype=x.dtype, device=DEV)
    B.experts_gather(x, slots, xs)
    assert torch.equal(xs[:n], x[at // top_k]) and not bool(xs[n:].any())
    ys, wts, dy = whole((S, H), 1, x.dtype), whole((T, top_k), 1, torch.float32), whole((T, H), 1, x.dtype)
    # torch adds in another order: of whole numbers that is the same
    scaled = ys[:n].float() * wts.view(-1)[at][:, None]
    y = torch.zeros((T, H), device=DEV).index_add_(0, at // top_k, scaled)
    assert torch.equal(B.experts_combine(ys, slots, wts, dtype=torch.float32), y)
    dys, dw = B.experts_combine_grad(dy, ys, slots, wts, dys=torch.zeros_like(ys))
    assert torch.equal(dys[:n].float(), wts.view(-1)[at][:, None] * dy[at // top_k].float())
    dots = torch.zeros(S, device=DEV)
    dots[at] = (dy[at // top_k].double() * ys[:n].double()).sum(dim=1).float()
    assert torch.equal(dw.view(-1), dots)


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    offsets, order, slots = B.experts_sort(ids, 3)
    x = torch.zeros((4, 64), device=DEV)
    ys = torch.zeros((8, 64), device=DEV)
    wt = torch.zeros((4, 2), device=DEV)
    w = torch.zeros(B.mxfp4_bytes(3 * 16, 64), dtype=torch.uint8, device=DEV)
    xm = B.quantize_mxfp4(x)
    for bad in (lambda: B.experts_sort(ids.float(), 3), lambda: B.experts_sort(ids.view(-1), 3),
                lambda: B.experts_sort(ids, 0), lambda: B.experts_sort(ids, 1025), lambda: B.experts_sort(ids.cpu(), 3),
                lambda: B.experts_sort(ids.t(), 3), lambda: B.experts_sort(ids[:0], 3),
                lambda: B.experts_sort(ids, 3, offsets=order),
                lambda: B.mmq_mxfp4_experts(w, xm, 4, offsets, order, 2, 4, 16, 64),
                lambda: B.mmq_mxfp4_experts(w, xm, 4, offsets, order, 0, 3, 16, 64),
                lambda: B.mmq_mxfp4_experts(w, xm, 5, offsets, order, 2, 3, 16, 64),
                lambda: B.mmq_mxfp4_experts(w, xm, 4, offsets, slots, 2, 3, 16, 64),
                lambda: B.mmq_mxfp4_experts(w, xm, 4, offsets, order, 2, 3, 16, 64, y=ys),
                lambda: B.experts_gather(x[:3], slots), lambda: B.experts_gather(x, slots.long()),
                lambda: B.experts_gather(x, slots, x), lambda: B.experts_gather(x.double(), slots),
                lambda: B.experts_combine(x, slots, wt), lambda: B.experts_combine(ys, slots, wt.half()),
                lambda: B.experts_combine(ys, slots, None), lambda: B.experts_combine(ys, slots, wt, dtype=torch.int8),
                lambda: B.experts_combine(ys.t(), slots, wt),
                lambda: B.experts_combine_grad(x[:2], ys, slots, wt),
                lambda: B.experts_combine_grad(x, ys, slots, wt, dys=x)):
        with pytest.raises(B.QPGError):
            bad()
