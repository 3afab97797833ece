"""What the binding of the MXFP4 and expert operators refuses by itself, before the library is
called (on the CPU, with stand-ins that have a device tensor's type, shape and place)."""
import os
import subprocess
import sys

import pytest
import torch

from quantized_prefill_gemm_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libqpg.so not built")


class Fake:
    """A contiguous tensor on cuda:0, without memory."""
    is_cuda, device = True, torch.device("cuda:0")

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


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


def u8(n):
    return Fake(n, dtype=torch.uint8)


def i32(*shape):
    return Fake(*shape, dtype=torch.int32)


@pytest.mark.parametrize("N,K", [(8, 64), (2048, 4096), (100, 1056), (33, 32)])
def test_weights_of_another_number_of_rows(run, N, K):
    """A matrix of more rows (or of more experts) is not its first N rows; bytes behind it that
    make up no row are let pass, and so is a workspace for more tokens."""
    x, size = Fake(4, K), lambda rows: B.mxfp4_bytes(rows, K)
    xm = u8(size(4))
    calls = (lambda w: B.mmq_mxfp4(w, x, N), lambda w: B.mmq_mxfp4_mx(w, xm, 4, N, K),
             lambda w: B.mmq_mxfp4_experts(w, xm, 4, i32(2), None, 1, 1, N, K))
    for call in calls:
        assert run(lambda: call(u8(size(N)))) == "called"
        assert run(lambda: call(u8(size(N) + 1))) == "called"
        for rows in (N + 1, 2 * N, 7 * N + 3):
            assert run(lambda: call(u8(size(rows)))) == B.QPG_EINVAL, rows
        assert run(lambda: call(u8(size(N) - 1))) == B.QPG_EINVAL
    assert run(lambda: B.mmq_mxfp4_mx(u8(size(N)), u8(size(64)), 4, N, K)) == "called"
    assert run(lambda: B.mmq_mxfp4(u8(size(N)), x, N, xm_ws=u8(size(64)))) == "called"
    assert run(lambda: B.mmq_mxfp4_experts(u8(size(3 * N)), xm, 4, i32(4), i32(8), 2, 3, N, K)) == "called"
    assert run(lambda: B.mmq_mxfp4_experts(u8(size(4 * N)), xm, 4, i32(4), i32(8), 2, 3, N, K)) == B.QPG_EINVAL


def test_weights_of_an_unsupported_shape(run):
    """An empty buffer has the size (0) that mxfp4_bytes gives for a shape it does not support."""
    x, xm = Fake(4, 64), u8(B.mxfp4_bytes(4, 64))
    for N in (0, -1, 2 ** 31):
        assert run(lambda: B.mmq_mxfp4(u8(0), x, N)) == B.QPG_EINVAL
        assert run(lambda: B.mmq_mxfp4_mx(u8(0), xm, 4, N, 64)) == B.QPG_EINVAL
        assert run(lambda: B.mmq_mxfp4_experts(u8(0), xm, 4, i32(2), None, 1, 1, N, 64)) == B.QPG_EINVAL


def test_order_of_another_number_of_choices(run):
    """order has rows * top_k entries: with another top_k, or xm of another number of tokens, rows
    would be taken from the wrong tokens."""
    E, N, K, T = 3, 16, 64, 6
    w, xm = u8(B.mxfp4_bytes(E * N, K)), u8(B.mxfp4_bytes(T, K))

    def call(order, top_k, rows=T):
        return run(lambda: B.mmq_mxfp4_experts(w, xm, rows, i32(E + 1), order, top_k, E, N, K))
    assert call(i32(12), 2) == "called" and call(None, 1) == "called" and call(i32(6), 1) == "called"
    for order, top_k in ((i32(12), 1), (i32(12), 3), (i32(12), 4), (i32(12), 0), (i32(12), -2), (i32(6, 2), 2), (i32(11), 2)):
        assert call(order, top_k) == B.QPG_EINVAL, (order.shape, top_k)
    assert call(i32(12), 2, rows=5) == B.QPG_EINVAL and call(i32(12), 3, rows=4) == "called"


def test_imports_on_a_torch_without_a_gpu_backend():
    """The module, and with it the host entry points of every operator, loads where torch has no
    _cuda_getCurrentRawStream."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import quantized_prefill_gemm_amd as qpg\n"
            "print(qpg.q8_1_bytes(1, 256), qpg.mxfp4_bytes(1, 64))\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(B.__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == [str(B.q8_1_bytes(1, 256)), "34"]
