"""Rows that no choice has, in buffers that experts_gather and experts_combine_grad allocate: zeros,
whatever the memory held before -- eagerly, on another stream, and in a graph replayed with other
routings."""
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
# T, top_k, H, E: single and odd rows, rows of several segments, and from 2^14 choices on rows that are
# zeroed beside the others (long ones) and ahead of them (short ones)
CASES = [(1, 1, 1, 3), (7, 3, 33, 5), (130, 8, 1032, 16), (2100, 2, 520, 9), (5, 2, 20_001, 4), (9, 300, 17_000, 4),
         (8192, 2, 3, 9), (8193, 2, 3, 9), (5000, 4, 17, 6), (20_000, 4, 1000, 33), (65_537, 2, 40, 9), (43_691, 3, 17, 200)]


def routing(T, top_k, E, rng):
    ids = rng.integers(0, E, (T, top_k))
    ids[rng.random((T, top_k)) < 0.4] = -1
    ids[0, 0] = E                              # one choice at least has no row
    return ids


def spoil(shape, dtype):
    """Memory that the allocator hands out next, full of NaN."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("T,top_k,H,E", CASES)
@pytest.mark.parametrize("kind", list(KINDS))
def test_rows_of_no_choice_are_zeros(T, top_k, H, E, kind):
    rng = np.random.default_rng([T, H])
    dtype = KINDS[kind]
    _, order, slots = R.sort(routing(T, top_k, E, rng), E)
    n = int((order >= 0).sum())
    x, dy = (torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype).to(DEV) for _ in range(2))
    ys = torch.from_numpy(rng.standard_normal((T * top_k, H)).astype(np.float32)).to(dtype).to(DEV)
    sd, w = torch.from_numpy(slots).to(DEV), torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV)
    given = torch.zeros((2, T * top_k, H), dtype=dtype, device=DEV)
    B.experts_gather(x, sd, given[0])
    B.experts_combine_grad(dy, ys, sd, w, dys=given[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        with torch.cuda.stream(stream):
            spoil((T * top_k, H), dtype)
        xs = B.experts_gather(x, sd, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(xs, given[0]) and not bool(xs[n:].any())
        del xs
        with torch.cuda.stream(stream):
            spoil((T * top_k, H), dtype)
        dys, _ = B.experts_combine_grad(dy, ys, sd, w, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(dys, given[1]) and not bool(dys[n:].any())
        # rows that no choice has anywhere, not behind the last alone: every other row
        some = torch.where(sd % 2 == 0, sd, torch.full_like(sd, -1))
        del dys
        with torch.cuda.stream(stream):
            spoil((T * top_k, H), dtype)
        xs = B.experts_gather(x, some, stream=stream)
        torch.cuda.synchronize()
        assert not bool(xs[1::2].any()) and torch.equal(xs[:n:2], given[0][:n:2])
        del xs


@pytest.mark.parametrize("kind", list(KINDS))
def test_nothing_else_is_written(kind):
    """The entry points that zero rows, on rows within a larger buffer that is aligned to its element."""
    L, dtype = B.lib(), KINDS[kind]
    code, s = B._type(dtype, "x"), torch.cuda.current_stream().cuda_stream
    for T, top_k, H, E in CASES[:4] + CASES[6:]:
        rng = np.random.default_rng([T, H, 3])
        _, order, slots = R.sort(routing(T, top_k, E, rng), E)
        n, S = int((order >= 0).sum()), T * top_k
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype).to(DEV)
        ys = torch.from_numpy(rng.standard_normal((S, H)).astype(np.float32)).to(dtype).to(DEV)
        sd, w = torch.from_numpy(slots).to(DEV), torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV)
        dw = torch.empty((T, top_k), device=DEV)
        for lead in (8, 9):
            room = torch.full((S * H + 64,), 5.0, dtype=dtype, device=DEV)
            rows = room[lead:lead + S * H].view(S, H)
            assert L.experts_gather_zero(x.data_ptr(), code, sd.data_ptr(), rows.data_ptr(), T, top_k, H, s) == B.QPG_OK
            assert torch.equal(rows[:n].cpu(), x.cpu()[torch.from_numpy(order[:n].astype(np.int64) // top_k)])
            assert not bool(rows[n:].any()) and bool((room[:lead] == 5.0).all()) and bool((room[lead + S * H:] == 5.0).all())
            room.fill_(5.0)
            assert L.experts_combine_grad_zero(x.data_ptr(), code, ys.data_ptr(), code, sd.data_ptr(), w.data_ptr(),
                                               rows.data_ptr(), dw.data_ptr(), T, top_k, H, s) == B.QPG_OK
            # at the same place in memory: the alignment decides which thread adds which products of a dot
            zeros = torch.zeros(S * H + 64, dtype=dtype, device=DEV)[lead:lead + S * H].view(S, H)
            want, want_dw = B.experts_combine_grad(x, ys, sd, w, dys=zeros)
            assert torch.equal(rows, want) and torch.equal(dw, want_dw)
            assert bool((room[:lead] == 5.0).all()) and bool((room[lead + S * H:] == 5.0).all())


def test_slots_that_name_no_row():
    """Entries outside [0, S) name none, wherever they would fall: all rows become zeros."""
    T, top_k, H = 300, 2, 24
    slots = torch.full((T, top_k), -1, dtype=torch.int32, device=DEV)
    slots.view(-1)[:6] = torch.tensor([T * top_k, T * top_k + 1, 2 ** 31 - 1, -2 ** 31, 768, -256], dtype=torch.int32)
    spoil((T * top_k, H), torch.float32)
    xs = B.experts_gather(torch.ones((T, H), device=DEV), slots)
    assert xs.shape == (T * top_k, H) and not bool(xs.any())


@pytest.mark.parametrize("T,top_k,H,E", CASES)
def test_and_in_a_graph(T, top_k, H, E):
    rng = np.random.default_rng([T, H, 2])

    def inputs():
        return (torch.from_numpy(routing(T, top_k, E, rng)).to(DEV),
                torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DEV),
                torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).to(DEV))

    def chain(ids, x, w):
        _, _, slots = B.experts_sort(ids, E)
        xs = B.experts_gather(x, slots)
        dys, dw = B.experts_combine_grad(x, xs, slots, w)
        return [slots, xs, dys, dw]
    held = list(inputs())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(*held)
    for rep in range(4):
        new = inputs()
        for t, v in zip(held, new):
            t.copy_(v)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        slots, xs, dys, dw = out
        n = int((slots >= 0).sum())
        assert not bool(xs[n:].any()) and not bool(dys[n:].any()), rep
        assert all(torch.equal(a, b) for a, b in zip(out, chain(*new))), rep
