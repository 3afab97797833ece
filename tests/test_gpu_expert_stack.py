"""The stack whose FFN is MXFP4 experts (quantized_prefill_gemm_amd.stack.ExpertStack), captured as
one graph and replayed with other inputs and routings: sampled output columns of every expert
product against 64 bits, the attention projections against the plain stack's calls."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import mx_ref as R
from quantized_prefill_gemm_amd import binding as B
from quantized_prefill_gemm_amd import inputs
from quantized_prefill_gemm_amd.stack import ExpertStack

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
L, M, E, TOP = 2, 48, 4, 2


def f64(t):
    return t.detach().cpu().double().numpy()


def columns(w, rows, N, K, pick):
    """Rows `pick` of every expert's matrix, in 64 bits: [E][len(pick)][K]."""
    codes, scales = R.unpack(w, rows, K)
    at = (np.arange(E)[:, None] * N + pick).reshape(-1)
    return R.decode(codes[at], scales[at]).reshape(E, len(pick), K)


def test_expert_stack_in_a_graph():
    rng = np.random.default_rng(77)
    weights = [[torch.from_numpy(inputs.make_stack_matrix(layer, i)[4].reshape(-1)).to(DEV) for i in range(4)]
               for layer in range(L)]
    host = []
    for layer in range(L):
        row = []
        for _, _, N, K in inputs.STACK_LAYER[4:]:
            codes = rng.integers(0, 256, E * N * K // 2, dtype=np.uint8)
            row.append(np.concatenate([codes, rng.integers(116, 122, E * N * K // 32, dtype=np.uint8)]))
        host.append(row)
    st = ExpertStack(weights, [[torch.from_numpy(w).to(DEV) for w in row] for row in host], M, E, TOP, per_layer=True)
    graph = st.capture("shared")
    for rep in range(2):
        x, ids, gains = {}, [], []
        for layer in range(L):
            for src in (0, 3, 4, 6):
                x[layer, src] = rng.standard_normal(tuple(st.x[layer][src].shape)).astype(np.float32)
                st.set_input(layer, src, torch.from_numpy(x[layer, src]).to(DEV))
            ids.append(rng.integers(-1, E, (M, TOP)))
            gains.append(rng.random((M, TOP)).astype(np.float32))
            st.set_routing(layer, torch.from_numpy(ids[-1]).to(DEV), torch.from_numpy(gains[-1]).to(DEV))
            for i in range(7):
                st.output(layer, i).fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for layer in range(L):
            for i, (_, wtype, N, K) in enumerate(inputs.STACK_LAYER[:4]):
                src = (0, 0, 0, 3)[i]
                xq = B.quantize_q8_1(torch.from_numpy(x[layer, src]).to(DEV))
                w = weights[layer][i]
                y = B.mmq_q4K_q8(w, xq, M, N, K) if wtype == "q4_K" else B.mmq_q6K_exp_q8(B.q6K_expand(w, N, K), xq, M, N, K)
                assert torch.equal(st.output(layer, i), y), (rep, layer, i)
            offsets, order, slots = R.sort(ids[layer], E)
            n = int(offsets[-1])
            expert = np.repeat(np.arange(E), np.diff(offsets))
            for i in (4, 5, 6):
                _, _, N, K = inputs.STACK_LAYER[i]
                pick = np.sort(rng.choice(N, 24, replace=False))
                wv = columns(host[layer][i - 4], E * N, N, K, pick)
                xv = R.decode(*R.encode(x[layer, 4 if i < 6 else 6]))
                rows = xv[order[:n] // TOP] if i < 6 else xv[:n]
                exact, bound = np.zeros((n, 24)), np.zeros((n, 24))
                for p in range(n):
                    exact[p] = wv[expert[p]] @ rows[p]
                    bound[p] = R.product_bound(rows[p:p + 1], wv[expert[p]], exact[p:p + 1], "float32")[0]
                if i == 6:                                # the weighted sum of a token's rows
                    on = slots >= 0
                    g = np.where(on, gains[layer], 0.0).astype(np.float64)
                    pick_rows = np.maximum(slots, 0)
                    magnitude = (g[:, :, None] * (np.abs(exact) + bound)[pick_rows]).sum(axis=1)
                    bound = (g[:, :, None] * bound[pick_rows]).sum(axis=1) + TOP * 2.0 ** -23 * magnitude
                    exact = (g[:, :, None] * exact[pick_rows]).sum(axis=1)
                    got = f64(st.output(layer, 6))[:, pick]
                    bound = bound + R.rounding(exact, "float32")
                else:
                    got = f64(st.output(layer, i))
                    assert np.isnan(got[n:]).all()        # rows behind the last stay as they were
                    got = got[:n, pick]
                assert (np.abs(got - exact) <= bound).all(), (rep, layer, i)
        # the eager pass with a quantisation before each product gives the same
        want = [[st.output(layer, i).clone() for i in range(7)] for layer in range(L)]
        st.run("all")
        torch.cuda.synchronize()
        for layer in range(L):
            for i in range(7):
                assert torch.equal(torch.nan_to_num(st.output(layer, i), nan=7e30),
                                   torch.nan_to_num(want[layer][i], nan=7e30)), (layer, i)


def test_refusals():
    with pytest.raises(ValueError):
        ExpertStack([[]], [], M, E, TOP)
    with pytest.raises(ValueError):
        ExpertStack([[]], [[]], M, E, E + 1)
