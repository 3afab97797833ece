"""The stack with attention over paged caches (quantized_prefill_gemm_amd.stack.AttentionStack), captured as one
graph and replayed: a prompt into an empty cache, then decoding beside another prompt, then trees of drafts. Every row's
attention against 64 bits of what the pass left in its own buffers, the projections against the plain stack's calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cache_ref as R
from quantized_prefill_gemm_amd import binding as B
from quantized_prefill_gemm_amd import inputs
from quantized_prefill_gemm_amd.stack import AttentionStack

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
L, M, SEQ, PAGE, WIDTH = 2, 24, 3, 16, 5
H, D = 32, 128


@pytest.fixture(scope="module")
def weights():
    return [[torch.from_numpy(inputs.make_stack_matrix(layer, i)[4].reshape(-1)).to(DEV) for i in range(7)] for layer in range(L)]


def batch_of(new, lens, table):
    """A Batch of the tests' reference whose pages are the stack's."""
    b = R.Batch(new, lens, H, D, PAGE, "f16", pad=M - sum(new))
    b.table = table
    b.width, b.pool = WIDTH, SEQ * WIDTH
    return b


def compare(st, b, tree=None, positions=None):
    for layer in range(L):
        io = st.io(layer)
        q, k, v = (st.y[io][i].cpu() for i in range(3))
        ((wq, bq), (wk, bk), (wv, bv)), where = R.append(b, q, k, v, st.freqs.cpu(), positions, adjacent=True)
        n = int(b.offsets[-1])
        b.k, b.v = st.k_cache[layer].cpu(), st.v_cache[layer].cpu()
        for row, page, place in where:
            for c, w, e in ((b.k, wk, bk), (b.v, wv, bv)):
                assert float(((c[page, :, place].double() - w[row]).abs() - e[row]).max()) <= 0
        if layer == L - 1:                            # one buffer for all layers
            assert float(((st.q.cpu().double() - wq).abs() - bq)[:n].max()) <= 0
        # the queries as the kernel rounded them, again through its own call (the caches hold the keys already)
        qr = B.cache_append(st.y[io][0], st.y[io][1], st.y[io][2], st.k_cache[layer].clone(), st.v_cache[layer].clone(), st.table,
                            st.lens, st.offsets, freqs=st.freqs, positions=st.positions, adjacent=True).cpu()
        want, bound, mine = R.attention(b, qr, "f32", tree=tree, positions=positions)
        got = st.x[io][3].view(M, H, D).cpu().double()
        assert float(((got - want).abs() - bound)[mine].max()) <= 0
        for idx, (_, wtype, N, K) in enumerate(inputs.STACK_LAYER):
            f = B.mmq_q4K if wtype == "q4_K" else B.mmq_q6K_exp_q8
            x = st.x[io][(0, 0, 0, 3, 4, 4, 6)[idx]]
            again = f(st.mats[layer][idx], x, N) if wtype == "q4_K" else f(st.mats[layer][idx], B.quantize_q8_1(x), M, N, K)
            assert torch.equal(st.output(layer, idx), again)


def give(st, gen):
    for layer in range(L):
        for src in (0, 4, 6):
            st.set_input(layer, src, torch.randn(st.x[0][src].shape, generator=gen).to(DEV))


def test_prompts_and_decoding_in_one_graph(weights):
    gen = torch.Generator().manual_seed(5)
    st = AttentionStack(weights, M, SEQ, WIDTH, SEQ * WIDTH, PAGE, per_layer=True)
    table = torch.randperm(SEQ * WIDTH, generator=gen).view(SEQ, WIDTH).to(torch.int32)
    give(st, gen)
    graph = st.capture()
    for new, lens in (([20, 0, 3], [20, 0, 3]), ([1, 17, 1], [21, 17, 4]), ([1, 1, 22], [22, 18, 26]), ([1, 1, 1], [23, 19, 27])):
        give(st, gen)
        b = batch_of(new, lens, table)
        st.set_batch(table, b.lens, b.offsets)
        graph.replay()
        torch.cuda.synchronize()
        compare(st, b)


def test_trees_in_a_graph(weights):
    gen = torch.Generator().manual_seed(6)
    st = AttentionStack(weights, M, SEQ, WIDTH, SEQ * WIDTH, PAGE, per_layer=True, words=1)
    table = torch.randperm(SEQ * WIDTH, generator=gen).view(SEQ, WIDTH).to(torch.int32)
    for c in (*st.k_cache, *st.v_cache):
        c.copy_(torch.randn(c.shape, generator=gen))
    give(st, gen)
    graph = st.capture()
    for new, lens in (([8, 8, 8], [30, 60, 9]), ([1, 16, 7], [31, 76, 7])):
        give(st, gen)
        b = batch_of(new, lens, table)
        bits, depths = R.tree_of(gen, new, 3)
        tree = R.words_of(bits, M, 0, 1)
        starts = np.repeat([n - k for n, k in zip(lens, new)], new)
        positions = torch.zeros(M, dtype=torch.int32)
        positions[:sum(new)] = torch.tensor([int(s) + d for s, d in zip(starts, depths)], dtype=torch.int32)
        st.set_batch(table, b.lens, b.offsets)
        st.set_tree(tree, positions)
        graph.replay()
        torch.cuda.synchronize()
        compare(st, b, tree, positions)


def test_arguments():
    for bad in ({"sequences": 0}, {"sequences": 30}, {"width": 0}, {"pages": 0}, {"words": -1}, {"q6": "raw "}):
        with pytest.raises(ValueError):
            AttentionStack([None], **{**{"M": M, "sequences": SEQ, "width": WIDTH, "pages": 4}, **bad})
