"""A layer of experts as a model runs it -- sort, gate and up through the order, the activation, down on
rows that are in sorted order already, the weighted sum -- with dropped choices, whose rows hold
whatever the memory did: each product against 64 bits of the activations it was given, and the
layer in a graph replayed with other routings, the memory full of NaN in between."""
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


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def layer(ids, x, gains, gate, up, down, E, H, F, dtype):
    T, top_k = ids.shape
    offsets, order, slots = B.experts_sort(ids, E)
    xm = B.quantize_mxfp4(x)
    g = B.mmq_mxfp4_experts(gate, xm, T, offsets, order, top_k, E, F, H, dtype=dtype)
    u = B.mmq_mxfp4_experts(up, xm, T, offsets, order, top_k, E, F, H, dtype=dtype)
    a = torch.nn.functional.silu(g) * u
    ys = B.mmq_mxfp4_experts(down, B.quantize_mxfp4(a), T * top_k, offsets, None, 1, E, H, F, dtype=dtype)
    return g, u, a, ys, B.experts_combine(ys, slots, gains, dtype=torch.float32)


@pytest.mark.parametrize("T,top_k,E,H,F", [(1, 2, 4, 256, 352), (5, 3, 8, 96, 544), (130, 2, 6, 416, 1056), (700, 2, 4, 1024, 1120)])
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_layer(T, top_k, E, H, F, kind):
    say(f"[layer {T} x {top_k} of {E}, {F} x {H}, {kind}]")
    rng = np.random.default_rng([T, E, H])
    dtype = getattr(torch, kind)
    host = [R.weights(E * N, K, rng, 0.1) for N, K in ((F, H), (F, H), (H, F))]
    gate, up, down = (torch.from_numpy(w).to(DEV) for w in host)

    def inputs():
        ids = rng.integers(0, E, (T, top_k))
        ids[rng.random((T, top_k)) < 0.3] = -1
        return (torch.from_numpy(ids).to(DEV), torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype).to(DEV),
                torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV))

    def spoil():
        held = [torch.full(s, float("nan"), dtype=dtype, device=DEV) for s in ((T * top_k, F),) * 3 + ((T * top_k, H),) * 2]
        torch.cuda.synchronize()
        del held

    ids, x, gains = inputs()
    spoil()
    g, u, a, ys, y = layer(ids, x, gains, gate, up, down, E, H, F, dtype)
    offsets, order, slots = R.sort(ids.cpu().numpy(), E)
    wg, wu, wd = (R.values(w, E * N, K).reshape(E, N, K) for w, (N, K) in zip(host, ((F, H), (F, H), (H, F))))
    xv = R.decode(*R.encode(f64(x)))
    n = int(offsets[-1])
    av = R.decode(*R.encode(f64(a)[:n])) if n else np.zeros((0, F))
    for e in range(E):
        rows = slice(offsets[e], offsets[e + 1])
        at = order[rows] // top_k
        for got, act, w in ((g, xv[at], wg[e]), (u, xv[at], wu[e]), (ys, av[rows], wd[e])):
            exact = act @ w.T
            assert (np.abs(f64(got)[rows] - exact) <= R.product_bound(act, w, exact, kind)).all(), e
    # the weighted sum of the products' own rows: one rounding for each product and each sum
    v = np.where(slots[:, :, None] >= 0, f64(ys)[np.maximum(slots, 0)], 0.0) * f64(gains)[:, :, None]
    assert (np.abs(f64(y) - v.sum(axis=1)) <= top_k * 2.0 ** -23 * np.abs(v).sum(axis=1) + 2.0 ** -140).all()

    si, sx, sg = ids.clone(), x.clone(), gains.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(si, sx, sg, gate, up, down, E, H, F, dtype)
    for rep in range(4):
        i, b, c = inputs()
        for t, new in ((si, i), (sx, b), (sg, c)):
            t.copy_(new)
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        spoil()
        want = layer(i, b, c, gate, up, down, E, H, F, dtype)
        rows = int((i >= 0).sum())
        for k, (p, q) in enumerate(zip(out, want)):
            assert torch.equal(p[:rows] if k < 4 else p, q[:rows] if k < 4 else q), (rep, k)
