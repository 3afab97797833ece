"""What the binding of the operators over a paged cache refuses by itself, before the library is called (on the
CPU, with stand-ins that have a device tensor's type, shape, strides and place)."""
import os

import pytest
import torch

from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libqpg.so not built")
F16, BF16, F32, I32, I64 = torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64


class Fake:
    """A tensor on a device, without memory."""

    def __init__(self, *shape, dtype=F32, strides=None, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device, self.is_cuda = torch.device("cuda", index), True
        plain = [1]
        for n in reversed(shape[1:]):
            plain.insert(0, plain[0] * n)
        self.plain, self.strides = tuple(plain), tuple(strides or plain)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.strides == self.plain

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


class Called(Exception):
    pass


@pytest.fixture
def run(monkeypatch):
    """The status of a call's refusal; "called" where the checks let it pass."""
    def stop(t, stream, call):
        raise Called
    monkeypatch.setattr(B, "_run", stop)

    def status(call):
        try:
            call()
        except B.QPGError as e:
            return e.status
        except Called:
            return "called"
    return status


def base():
    return {"k_cache": Fake(10, 2, 16, 64, dtype=F16), "v_cache": Fake(10, 2, 16, 64, dtype=F16), "table": Fake(3, 4, dtype=I32),
            "lens": Fake(3, dtype=I32), "offsets": Fake(4, dtype=I32)}


def append(**more):
    return B.cache_append(**{"q": Fake(5, 256), "k": Fake(5, 128), "v": Fake(5, 128), **base(), **more})


def attend(**more):
    return B.cache_attention(**{"q": Fake(5, 4, 64, dtype=F16), **base(), **more})


def tree(**more):
    return B.cache_attention_tree(**{"q": Fake(5, 4, 64, dtype=F16), **base(), "tree": Fake(5, 2, dtype=I64),
                                     "positions": Fake(5, dtype=I32), **more})


GOOD_CACHE = [{}, {"k_cache": Fake(10, 2, 16, 64, dtype=F16, strides=(4096, 1024, 64, 1)), "v_cache": Fake(10, 2, 16, 64, dtype=F16)}]
BAD_BASE = [{"k_cache": Fake(10, 2, 16, 64)}, {"v_cache": Fake(10, 2, 16, 64, dtype=BF16)}, {"v_cache": Fake(9, 2, 16, 64, dtype=F16)},
            {"k_cache": Fake(10, 2, 1024, dtype=F16)}, {"v_cache": Fake(10, 2, 16, 64, dtype=F16, index=1)},
            {"k_cache": Fake(10, 2, 16, 64, dtype=F16, strides=(2048, 64, 128, 1))},
            {"v_cache": Fake(10, 2, 16, 64, dtype=F16, strides=(1024, 1024, 64, 1))},
            {"v_cache": Fake(10, 2, 16, 64, dtype=F16, strides=(4096, 2048, 64, 2))},
            {"k_cache": Fake(0, 2, 16, 64, dtype=F16), "v_cache": Fake(0, 2, 16, 64, dtype=F16)},
            {"table": Fake(3, 4, dtype=I64)}, {"table": Fake(12, dtype=I32)}, {"table": Fake(3, 4, dtype=I32, strides=(8, 1))},
            {"lens": Fake(4, dtype=I32)}, {"lens": Fake(3)}, {"offsets": Fake(3, dtype=I32)}, {"offsets": Fake(4, dtype=I64)},
            {"offsets": Fake(4, dtype=I32, index=1)}]


@pytest.mark.parametrize("call", [append, attend, tree])
def test_caches_and_batches(run, call):
    for more in GOOD_CACHE:
        assert run(lambda: call(**more)) == "called"
    for more in BAD_BASE:
        assert run(lambda: call(**more)) == B.QPG_EINVAL, {n: (t.shape, t.dtype) for n, t in more.items()}


def test_append(run):
    for more in ({"q": None}, {"q": Fake(5, 256, strides=(600, 1)), "k": Fake(5, 128, strides=(600, 1))}, {"freqs": Fake(32)},
                 {"positions": Fake(5, dtype=I32)}, {"q_norm": Fake(64), "k_norm": Fake(64)}, {"y": Fake(5, 4, 64, dtype=F16)},
                 {n: Fake(5, w, dtype=BF16) for n, w in (("q", 128), ("k", 128), ("v", 128))}):
        assert run(lambda: append(**more)) == "called", more
    for more in ({"q": Fake(5, 250)}, {"q": Fake(5, 192)}, {"q": Fake(5, 0)}, {"q": Fake(4, 256)}, {"q": Fake(5, 256, dtype=F16)}, {"q": Fake(5, 4, 64)},
                 {"q": Fake(5, 256, strides=(1, 5))}, {"q": Fake(5, 256, strides=(0, 1))}, {"q": Fake(5, 256, strides=(200, 1))},
                 {"k": Fake(5, 64)}, {"v": Fake(5, 256)}, {"v": Fake(6, 128)}, {"k": Fake(5, 128, index=1)}, {"k": Fake(5, 128, dtype=torch.float64)},
                 {"freqs": Fake(32, dtype=F16)}, {"freqs": Fake(32, 1)}, {"positions": Fake(5, dtype=I64)}, {"positions": Fake(4, dtype=I32)},
                 {"q_norm": Fake(32)}, {"k_norm": Fake(64, dtype=F16)}, {"y": Fake(5, 4, 64)}, {"y": Fake(5, 256, dtype=F16)},
                 {"q": None, "y": Fake(5, 4, 64, dtype=F16)}):
        assert run(lambda: append(**more)) == B.QPG_EINVAL, {n: t and (t.shape, t.dtype) for n, t in more.items()}


@pytest.mark.parametrize("call", [attend, tree])
def test_attention(run, call):
    for more in ({"q": Fake(5, 2, 64, dtype=F16)}, {"slopes": Fake(4)}, {"y": Fake(5, 4, 64)}, {"dtype": F32}, {"dtype": BF16},
                 {"ws": Fake(1 << 24, dtype=torch.uint8)}):
        assert run(lambda: call(**more)) == "called", more
    for more in ({"q": Fake(5, 4, 64)}, {"q": Fake(5, 256, dtype=F16)}, {"q": Fake(5, 3, 64, dtype=F16)}, {"q": Fake(5, 4, 32, dtype=F16)},
                 {"q": Fake(5, 4, 64, dtype=F16, strides=(512, 64, 1))}, {"q": Fake(5, 4, 64, dtype=F16, index=1)}, {"slopes": Fake(2)},
                 {"slopes": Fake(4, dtype=F16)}, {"y": Fake(5, 4, 32)}, {"y": Fake(5, 4, 64, dtype=I32)}, {"dtype": torch.float64},
                 {"ws": Fake(1 << 24)}):
        assert run(lambda: call(**more)) == B.QPG_EINVAL, {n: getattr(t, "shape", t) for n, t in more.items()}
    one = {"q": Fake(1, 4, 64, dtype=F16), "table": Fake(1, 512, dtype=I32), "lens": Fake(1, dtype=I32), "offsets": Fake(2, dtype=I32)}
    if call is attend:
        size = B.cache_attention_bytes(1, 1, 4, 2, 64, 512 * 16)
        assert size > 0 and run(lambda: call(**one, ws=Fake(size, dtype=torch.uint8))) == "called"
        assert run(lambda: call(**one, ws=Fake(size - 1, dtype=torch.uint8))) == B.QPG_EINVAL


def test_masks(run):
    assert run(lambda: attend(prefix=Fake(3, dtype=I32))) == "called"
    for more in ({"prefix": Fake(4, dtype=I32)}, {"prefix": Fake(3, dtype=I64)}, {"prefix": Fake(3, dtype=I32, index=1)}):
        assert run(lambda: attend(**more)) == B.QPG_EINVAL
    for more in ({"tree": None}, {"positions": None}, {"tree": Fake(5, 2, dtype=I32)}, {"tree": Fake(4, 2, dtype=I64)}, {"tree": Fake(10, dtype=I64)},
                 {"positions": Fake(5, dtype=I64)}, {"positions": Fake(5, 1, dtype=I32)}):
        assert run(lambda: tree(**more)) == B.QPG_EINVAL, more


def test_host_tensors_are_refused():
    f = {"k_cache": torch.zeros(10, 2, 16, 64, dtype=F16), "v_cache": torch.zeros(10, 2, 16, 64, dtype=F16),
         "table": torch.zeros(3, 4, dtype=I32), "lens": torch.zeros(3, dtype=I32), "offsets": torch.zeros(4, dtype=I32)}
    for call in (lambda: B.cache_append(torch.zeros(5, 256), torch.zeros(5, 128), torch.zeros(5, 128), **f),
                 lambda: B.cache_attention(torch.zeros(5, 4, 64, dtype=F16), **f)):
        with pytest.raises(B.QPGError) as e:
            call()
        assert e.value.status == B.QPG_EINVAL
