"""ctypes binding of libqpg.so: argument marshalling only.

Every step of the path runs in the HIP kernels of libqpg.so. torch provides device
memory and the stream (torch.cuda.current_stream()); nothing here computes. If the
library has not been built, the first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqpg.so")

QPG_OK, QPG_EINVAL, QPG_EALIGN, QPG_EHIP, QPG_EDEVICE, QPG_ESCRATCH = 0, -1, -2, -3, -4, -5
NOALLOC_SCRATCH_BYTES = 32 << 20     # QPG_NOALLOC_SCRATCH_BYTES of qpg.h


class QPGError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqpg.so once. Raises if it is missing (build with __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QPGError(QPG_EINVAL, f"libqpg.so not built at {LIB_PATH}")
        L = ctypes.CDLL(LIB_PATH)
        P, I64 = ctypes.c_void_p, ctypes.c_int64
        L.qpg_strerror.argtypes = [ctypes.c_int]
        L.qpg_strerror.restype = ctypes.c_char_p
        L.qpg_q8_1_bytes.argtypes = [I64, I64]
        L.qpg_q8_1_bytes.restype = ctypes.c_size_t
        L.quantize_q8_1.argtypes = [P, P, I64, I64, P]
        for f in (L.mmq_q4K, L.mmq_q6K):
            f.argtypes = [P, P, P, I64, I64, I64, P, P]
        L.mmq_q4K_noalloc.argtypes = [P, P, P, I64, I64, I64, P]
        L.mmq_q4K_noalloc.restype = ctypes.c_int
        for f in (L.mmq_q4K_q8, L.mmq_q6K_q8, L.mmq_q4K_isums, L.mmq_q6K_isums):
            f.argtypes = [P, P, P, I64, I64, I64, P]
        L.qpg_q6K_prep_bytes.argtypes = [I64, I64]
        L.qpg_q6K_prep_bytes.restype = ctypes.c_size_t
        L.q6K_prepare.argtypes = [P, P, I64, I64, P]
        for f in (L.mmq_q6K_prep_q8, L.mmq_q6K_prep_isums):
            f.argtypes = [P, P, P, I64, I64, I64, P]
        L.qpg_q6K_exp_bytes.argtypes = [I64, I64]
        L.qpg_q6K_exp_bytes.restype = ctypes.c_size_t
        L.q6K_expand.argtypes = [P, P, I64, I64, P]
        for f in (L.mmq_q6K_exp_q8, L.mmq_q6K_exp_csums):
            f.argtypes = [P, P, P, I64, I64, I64, P]
        L.qpg_mmq_sk_bytes.argtypes = [I64, I64, I64, ctypes.c_int]
        L.qpg_mmq_sk_bytes.restype = ctypes.c_size_t
        for f in (L.mmq_q4K_q8_sk, L.mmq_q6K_q8_sk, L.mmq_q6K_prep_q8_sk, L.mmq_q6K_exp_q8_sk):
            f.argtypes = [P, P, P, I64, I64, I64, P, ctypes.c_size_t, P]
            f.restype = ctypes.c_int
        for f in (L.quantize_q8_1, L.mmq_q4K, L.mmq_q6K, L.mmq_q4K_q8, L.mmq_q6K_q8, L.mmq_q4K_isums,
                  L.mmq_q6K_isums, L.q6K_prepare, L.mmq_q6K_prep_q8, L.mmq_q6K_prep_isums, L.q6K_expand,
                  L.mmq_q6K_exp_q8, L.mmq_q6K_exp_csums):
            f.restype = ctypes.c_int
        INT, SIZE = ctypes.c_int, ctypes.c_size_t
        for f, res, args in (
                (L.qpg_mxfp4_bytes, SIZE, [I64, I64]), (L.qpg_experts_sort_bytes, SIZE, [I64, I64]),
                (L.quantize_mxfp4, INT, [P, INT, P, I64, I64, P]), (L.dequantize_mxfp4, INT, [P, P, INT, I64, I64, P]),
                (L.mmq_mxfp4_mx, INT, [P, P, P, INT, I64, I64, I64, P]),
                (L.mmq_mxfp4, INT, [P, P, INT, P, INT, I64, I64, I64, P, P]),
                (L.mmq_mxfp4_experts, INT, [P, P, I64, P, P, I64, P, INT, I64, I64, I64, I64, P]),
                (L.experts_sort, INT, [P, INT, I64, I64, P, P, P, P, P]),
                (L.experts_gather, INT, [P, INT, P, P, I64, I64, I64, P]),
                (L.experts_gather_zero, INT, [P, INT, P, P, I64, I64, I64, P]),
                (L.experts_combine, INT, [P, INT, P, P, P, INT, I64, I64, I64, P]),
                (L.experts_combine_grad, INT, [P, INT, P, INT, P, P, P, P, I64, I64, I64, P]),
                (L.experts_combine_grad_zero, INT, [P, INT, P, INT, P, P, P, P, I64, I64, I64, P])):
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


EXPORTS = ("qpg_strerror", "qpg_q8_1_bytes", "quantize_q8_1", "mmq_q4K", "mmq_q6K", "mmq_q4K_q8",
           "mmq_q6K_q8", "mmq_q4K_isums", "mmq_q6K_isums", "qpg_q6K_prep_bytes", "q6K_prepare",
           "mmq_q6K_prep_q8", "mmq_q6K_prep_isums", "qpg_q6K_exp_bytes", "q6K_expand", "mmq_q6K_exp_q8",
           "mmq_q6K_exp_csums", "qpg_mmq_sk_bytes", "mmq_q4K_q8_sk", "mmq_q6K_q8_sk", "mmq_q6K_prep_q8_sk",
           "mmq_q6K_exp_q8_sk", "mmq_q4K_noalloc", "qpg_mxfp4_bytes", "quantize_mxfp4", "dequantize_mxfp4",
           "mmq_mxfp4_mx", "mmq_mxfp4", "qpg_experts_sort_bytes", "experts_sort", "mmq_mxfp4_experts",
           "experts_gather", "experts_gather_zero", "experts_combine", "experts_combine_grad",
           "experts_combine_grad_zero")


def _check(rc: int, what: str):
    if rc != QPG_OK:
        raise QPGError(rc, f"{what}: {lib().qpg_strerror(rc).decode()}")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise QPGError(QPG_EINVAL, f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise QPGError(QPG_EINVAL, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise QPGError(QPG_EINVAL, f"{name} must be contiguous")


def _same_device(t: torch.Tensor, ref: torch.Tensor, name: str):
    if t.device != ref.device:
        raise QPGError(QPG_EINVAL, f"{name} is on {t.device}, the inputs on {ref.device}")


def _out(t: torch.Tensor, dtype, name: str, need: int, ref: torch.Tensor):
    """A caller-supplied output: device tensor of dtype, contiguous, on ref's device and
    holding at least `need` elements (the C ABI takes no output size, so an undersized
    buffer would be written past its end)."""
    _dev(t, dtype, name)
    _same_device(t, ref, name)
    if t.numel() < need:
        raise QPGError(QPG_EINVAL, f"{name} holds {t.numel()} elements, {need} needed")


def q8_1_bytes(M: int, K: int) -> int:
    return int(lib().qpg_q8_1_bytes(M, K))


def quantize_q8_1(x: torch.Tensor, xq: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x f32 [M, K] (device) -> uint8 q8_1 buffer of q8_1_bytes(M, K) bytes."""
    _dev(x, torch.float32, "x")
    M, K = x.shape
    nbytes = q8_1_bytes(M, K)
    if xq is None:
        xq = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    _out(xq, torch.uint8, "xq", nbytes, x)
    _check(lib().quantize_q8_1(_ptr(x), _ptr(xq), M, K, _stream(stream)), "quantize_q8_1")
    return xq


def _wcheck(w: torch.Tensor, N: int, K: int, bytes_per_block: int):
    _dev(w, torch.uint8, "w")
    if w.numel() != N * (K // 256) * bytes_per_block:
        raise QPGError(QPG_EINVAL, "w size does not match N x K")


def _mmq(which: str, w, x, N, y, xq_ws, stream):
    _dev(x, torch.float32, "x")
    M, K = x.shape
    _wcheck(w, N, K, 144 if which == "q4K" else 210)
    _same_device(w, x, "w")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _out(y, torch.float32, "y", M * N, x)
    if xq_ws is None:
        xq_ws = torch.empty(max(q8_1_bytes(M, K), 1), dtype=torch.uint8, device=x.device)
    _out(xq_ws, torch.uint8, "xq_ws", q8_1_bytes(M, K), x)
    fn = lib().mmq_q4K if which == "q4K" else lib().mmq_q6K
    _check(fn(_ptr(w), _ptr(x), _ptr(y), M, N, K, _ptr(xq_ws), _stream(stream)), "mmq_" + which)
    return y


def mmq_q4K(w: torch.Tensor, x: torch.Tensor, N: int, y=None, xq_ws=None, stream=None) -> torch.Tensor:
    """Y f32 [M, N] = q4_K W [N, K] x q8_1(x)^T; w is the raw uint8 block buffer."""
    return _mmq("q4K", w, x, N, y, xq_ws, stream)


def mmq_q6K(w: torch.Tensor, x: torch.Tensor, N: int, y=None, xq_ws=None, stream=None) -> torch.Tensor:
    return _mmq("q6K", w, x, N, y, xq_ws, stream)


def mmq_q4K_noalloc(w: torch.Tensor, x: torch.Tensor, N: int, y: torch.Tensor, stream=None) -> torch.Tensor:
    """mmq_q4K with the q8_1 activations in the library's fixed per-device scratch: the C call
    allocates nothing (y is the caller's). Calls overlapping on one device race."""
    _dev(x, torch.float32, "x")
    M, K = x.shape
    _wcheck(w, N, K, 144)
    _same_device(w, x, "w")
    _out(y, torch.float32, "y", M * N, x)
    _check(lib().mmq_q4K_noalloc(_ptr(w), _ptr(x), _ptr(y), M, N, K, _stream(stream)), "mmq_q4K_noalloc")
    return y


def _mmq_q8(which: str, w, xq, M, N, K, out, stream, isums: bool):
    _dev(xq, torch.uint8, "xq")
    if xq.numel() < q8_1_bytes(M, K):
        raise QPGError(QPG_EINVAL, "xq too small")
    _wcheck(w, N, K, 144 if which == "q4K" else 210)
    _same_device(w, xq, "w")
    if isums:
        per = 32 if which == "q4K" else 16
        if out is None:
            out = torch.empty((M, N, K // per), dtype=torch.int32, device=xq.device)
        _out(out, torch.int32, "s", M * N * (K // per), xq)
        fn = lib().mmq_q4K_isums if which == "q4K" else lib().mmq_q6K_isums
    else:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=xq.device)
        _out(out, torch.float32, "y", M * N, xq)
        fn = lib().mmq_q4K_q8 if which == "q4K" else lib().mmq_q6K_q8
    _check(fn(_ptr(w), _ptr(xq), _ptr(out), M, N, K, _stream(stream)),
           ("mmq_%s_isums" if isums else "mmq_%s_q8") % which)
    return out


def mmq_q4K_q8(w, xq, M, N, K, y=None, stream=None):
    return _mmq_q8("q4K", w, xq, M, N, K, y, stream, False)


def mmq_q6K_q8(w, xq, M, N, K, y=None, stream=None):
    return _mmq_q8("q6K", w, xq, M, N, K, y, stream, False)


def mmq_q4K_isums(w, xq, M, N, K, s=None, stream=None):
    return _mmq_q8("q4K", w, xq, M, N, K, s, stream, True)


def mmq_q6K_isums(w, xq, M, N, K, s=None, stream=None):
    return _mmq_q8("q6K", w, xq, M, N, K, s, stream, True)


def q6K_prep_bytes(N: int, K: int) -> int:
    return int(lib().qpg_q6K_prep_bytes(N, K))


def q6K_prepare(w: torch.Tensor, N: int, K: int, wp=None, stream=None) -> torch.Tensor:
    """Raw q6_K blocks (uint8, N*(K/256)*210 bytes, device) -> prepared layout (uint8)."""
    _wcheck(w, N, K, 210)
    nbytes = q6K_prep_bytes(N, K)
    if nbytes == 0:
        raise QPGError(QPG_EINVAL, f"unsupported shape N={N} K={K}")
    if wp is None:
        wp = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _out(wp, torch.uint8, "wp", nbytes, w)
    _check(lib().q6K_prepare(_ptr(w), _ptr(wp), N, K, _stream(stream)), "q6K_prepare")
    return wp


def _mmq_prep(wp, xq, M, N, K, out, stream, isums: bool):
    _dev(xq, torch.uint8, "xq")
    if xq.numel() < q8_1_bytes(M, K):
        raise QPGError(QPG_EINVAL, "xq too small")
    _dev(wp, torch.uint8, "wp")
    _same_device(wp, xq, "wp")
    if wp.numel() < q6K_prep_bytes(N, K):
        raise QPGError(QPG_EINVAL, "wp too small")
    if isums:
        if out is None:
            out = torch.empty((M, N, K // 16), dtype=torch.int32, device=xq.device)
        _out(out, torch.int32, "s", M * N * (K // 16), xq)
        fn = lib().mmq_q6K_prep_isums
    else:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=xq.device)
        _out(out, torch.float32, "y", M * N, xq)
        fn = lib().mmq_q6K_prep_q8
    _check(fn(_ptr(wp), _ptr(xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_q6K_prep_isums" if isums else "mmq_q6K_prep_q8")
    return out


def mmq_q6K_prep_q8(wp, xq, M, N, K, y=None, stream=None):
    return _mmq_prep(wp, xq, M, N, K, y, stream, False)


def mmq_q6K_prep_isums(wp, xq, M, N, K, s=None, stream=None):
    return _mmq_prep(wp, xq, M, N, K, s, stream, True)


def q6K_exp_bytes(N: int, K: int) -> int:
    return int(lib().qpg_q6K_exp_bytes(N, K))


def q6K_expand(w: torch.Tensor, N: int, K: int, we=None, stream=None) -> torch.Tensor:
    """Raw q6_K blocks (uint8, N*(K/256)*210 bytes, device) -> expanded layout (uint8)."""
    _wcheck(w, N, K, 210)
    nbytes = q6K_exp_bytes(N, K)
    if nbytes == 0:
        raise QPGError(QPG_EINVAL, f"unsupported shape N={N} K={K}")
    if we is None:
        we = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _out(we, torch.uint8, "we", nbytes, w)
    _check(lib().q6K_expand(_ptr(w), _ptr(we), N, K, _stream(stream)), "q6K_expand")
    return we


def _mmq_exp(we, xq, M, N, K, out, stream, csums: bool):
    _dev(xq, torch.uint8, "xq")
    if xq.numel() < q8_1_bytes(M, K):
        raise QPGError(QPG_EINVAL, "xq too small")
    _dev(we, torch.uint8, "we")
    _same_device(we, xq, "we")
    if we.numel() < q6K_exp_bytes(N, K):
        raise QPGError(QPG_EINVAL, "we too small")
    if csums:
        if out is None:
            out = torch.empty((M, N, K // 32), dtype=torch.int32, device=xq.device)
        _out(out, torch.int32, "s", M * N * (K // 32), xq)
        fn = lib().mmq_q6K_exp_csums
    else:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=xq.device)
        _out(out, torch.float32, "y", M * N, xq)
        fn = lib().mmq_q6K_exp_q8
    _check(fn(_ptr(we), _ptr(xq), _ptr(out), M, N, K, _stream(stream)),
           "mmq_q6K_exp_csums" if csums else "mmq_q6K_exp_q8")
    return out


def mmq_q6K_exp_q8(we, xq, M, N, K, y=None, stream=None):
    return _mmq_exp(we, xq, M, N, K, y, stream, False)


def mmq_q6K_exp_csums(we, xq, M, N, K, s=None, stream=None):
    return _mmq_exp(we, xq, M, N, K, s, stream, True)


# Weight forms of the K-split entry points (the form argument of qpg_mmq_sk_bytes).
SK_FORMS = {"q4K": 0, "q6K": 1, "q6K_prep": 2, "q6K_exp": 3}
_SK_FN = {"q4K": "mmq_q4K_q8_sk", "q6K": "mmq_q6K_q8_sk", "q6K_prep": "mmq_q6K_prep_q8_sk",
          "q6K_exp": "mmq_q6K_exp_q8_sk"}


def mmq_sk_bytes(M: int, N: int, K: int, form: str) -> int:
    """Workspace bytes of the K-split entry point for this shape (0: no split is made)."""
    return int(lib().qpg_mmq_sk_bytes(M, N, K, SK_FORMS[form]))


def _mmq_sk(form: str, w, xq, M, N, K, y, ws, stream):
    _dev(xq, torch.uint8, "xq")
    if xq.numel() < q8_1_bytes(M, K):
        raise QPGError(QPG_EINVAL, "xq too small")
    if form in ("q4K", "q6K"):
        _wcheck(w, N, K, 144 if form == "q4K" else 210)
    else:
        _dev(w, torch.uint8, "w")
        need = q6K_prep_bytes(N, K) if form == "q6K_prep" else q6K_exp_bytes(N, K)
        if w.numel() < need:
            raise QPGError(QPG_EINVAL, "w too small")
    _same_device(w, xq, "w")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=xq.device)
    _out(y, torch.float32, "y", M * N, xq)
    nws = mmq_sk_bytes(M, N, K, form)
    if ws is None and nws:
        ws = torch.empty(nws // 4, dtype=torch.float32, device=xq.device)
    if ws is not None:
        _out(ws, torch.float32, "ws", nws // 4, xq)
    wsb = 0 if ws is None else ws.numel() * 4
    _check(getattr(lib(), _SK_FN[form])(_ptr(w), _ptr(xq), _ptr(y), M, N, K, _ptr(ws), wsb, _stream(stream)),
           _SK_FN[form])
    return y


def mmq_q4K_q8_sk(w, xq, M, N, K, y=None, ws=None, stream=None):
    return _mmq_sk("q4K", w, xq, M, N, K, y, ws, stream)


def mmq_q6K_q8_sk(w, xq, M, N, K, y=None, ws=None, stream=None):
    return _mmq_sk("q6K", w, xq, M, N, K, y, ws, stream)


def mmq_q6K_prep_q8_sk(wp, xq, M, N, K, y=None, ws=None, stream=None):
    return _mmq_sk("q6K_prep", wp, xq, M, N, K, y, ws, stream)


def mmq_q6K_exp_q8_sk(we, xq, M, N, K, y=None, ws=None, stream=None):
    return _mmq_sk("q6K_exp", we, xq, M, N, K, y, ws, stream)


# ---- MXFP4 and experts. The tensors of a call lie on one device, which need not be the current
# one. Outputs and workspaces that are not given are allocated on the stream the call runs on.
# No call records an autograd graph, whatever its operands require: gradients are calls of their own.
# A small call is bound by the host (a launch takes 3.7 us, torch.cuda.current_stream() 2.9, an
# allocation 1.4), so the checks below are one comparison each where nothing is wrong.
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}      # QPG_F32, QPG_F16, QPG_BF16


def _current_raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# 0.1 us where torch has it (a torch built without a GPU backend does not, and still loads this module)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream)


def _run(t: torch.Tensor, stream, call):
    """call(raw stream) with t's device current and `stream` (t's device's current one if None)
    the one that torch allocates on."""
    dev = t.get_device()
    if stream is None and dev == torch.cuda.current_device():
        return call(_raw_stream(dev))
    if stream is not None and stream.device != t.device:
        raise QPGError(QPG_EINVAL, f"the stream is on {stream.device}, the operands on {t.device}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return call(_raw_stream(dev))


def _type(dtype, name: str) -> int:
    code = _TYPES.get(dtype)
    if code is None:
        raise QPGError(QPG_EINVAL, f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return code


def _float(t: torch.Tensor, name: str) -> int:
    """The type code of a float operand, a contiguous matrix on a device."""
    code = _type(t.dtype, name)
    if t.get_device() < 0 or not t.is_contiguous():
        _dev(t, t.dtype, name)
    if t.dim() != 2:
        raise QPGError(QPG_EINVAL, f"{name} must have 2 dimensions, got {tuple(t.shape)}")
    return code


def _is(t: torch.Tensor, dtype, shape, name: str, ref: torch.Tensor):
    """An operand of a known type and shape, on ref's device."""
    if t.dtype is not dtype or t.get_device() != ref.get_device() or not t.is_contiguous():
        _dev(t, dtype, name)
        _same_device(t, ref, name)
    if t.shape != shape:
        raise QPGError(QPG_EINVAL, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _mx(t: torch.Tensor, rows: int, K: int, name: str, ref: torch.Tensor):
    """An MXFP4 operand of rows x K values: uint8, at least its size. Activations may lie in a
    workspace for more tokens; the scales follow the codes of `rows` rows there too."""
    need = _mx_bytes(rows, K, name)
    if t.dtype is not torch.uint8 or t.get_device() != ref.get_device() or t.get_device() < 0 \
            or not t.is_contiguous() or t.numel() < need:
        _out(t, torch.uint8, name, need, ref)


def _mx_weights(w: torch.Tensor, rows: int, K: int, ref: torch.Tensor):
    """MXFP4 weights of rows x K values. The scales start where the codes of all rows end, so the
    buffer of a matrix of more rows is no buffer of its first ones: a size of a whole number of
    other rows is refused. (Bytes behind the matrix that make up no rows are let pass.)"""
    need = _mx_bytes(rows, K, "w")
    if w.numel() == need and w.dtype is torch.uint8 and w.get_device() == ref.get_device() >= 0 and w.is_contiguous():
        return
    _mx(w, rows, K, "w", ref)
    if w.numel() != need and w.numel() * 32 % (17 * K) == 0:
        raise QPGError(QPG_EINVAL, f"w is the size of {w.numel() * 32 // (17 * K)} x {K} MXFP4 values, not of {rows} x {K}")


@functools.lru_cache(maxsize=4096)
def mxfp4_bytes(rows: int, K: int) -> int:
    """Size of an MXFP4 buffer of rows x K values (0: unsupported shape)."""
    return int(lib().qpg_mxfp4_bytes(rows, K))


def _mx_bytes(rows: int, K: int, name: str) -> int:
    n = mxfp4_bytes(rows, K)
    if n == 0:
        raise QPGError(QPG_EINVAL, f"unsupported MXFP4 shape of {name}: {rows} x {K}")
    return n


def _given(y, dtype, shape, name: str, ref: torch.Tensor):
    """(dtype, type code) of an output: y's own where y is given, which then has that shape."""
    if y is None:
        return dtype, _type(dtype, name)
    code = _type(y.dtype, name)
    _is(y, y.dtype, shape, name, ref)
    return y.dtype, code


def quantize_mxfp4(x: torch.Tensor, xm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [M, K] (float32, float16 or bfloat16) -> uint8 MXFP4 buffer of mxfp4_bytes(M, K) bytes."""
    code = _float(x, "x")
    M, K = x.shape
    nbytes = _mx_bytes(M, K, "x")
    if xm is not None:
        _mx(xm, M, K, "xm", x)

    def call(s):
        out = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if xm is None else xm
        _check(lib().quantize_mxfp4(x.data_ptr(), code, out.data_ptr(), M, K, s), "quantize_mxfp4")
        return out
    return _run(x, stream, call)


def dequantize_mxfp4(xm: torch.Tensor, M: int, K: int, y: torch.Tensor | None = None, dtype=torch.float32,
                     stream=None) -> torch.Tensor:
    """MXFP4 buffer -> y [M, K], the values its codes stand for (dtype: y's where y is given)."""
    _mx(xm, M, K, "xm", xm)
    dtype, code = _given(y, dtype, (M, K), "y", xm)

    def call(s):
        out = torch.empty((M, K), dtype=dtype, device=xm.device) if y is None else y
        _check(lib().dequantize_mxfp4(xm.data_ptr(), out.data_ptr(), code, M, K, s), "dequantize_mxfp4")
        return out
    return _run(xm, stream, call)


def mmq_mxfp4(w: torch.Tensor, x: torch.Tensor, N: int, y=None, xm_ws=None, dtype=torch.float32,
              stream=None) -> torch.Tensor:
    """y [M, N] = MXFP4(x [M, K]) x w [N, K]^T from float activations; w is an MXFP4 buffer. xm_ws:
    mxfp4_bytes(M, K) bytes of workspace that holds MXFP4(x) afterwards."""
    x_code = _float(x, "x")
    M, K = x.shape
    nbytes = _mx_bytes(M, K, "x")
    _mx_weights(w, N, K, x)
    dtype, y_code = _given(y, dtype, (M, N), "y", x)
    if xm_ws is not None:
        _mx(xm_ws, M, K, "xm_ws", x)

    def call(s):
        out = torch.empty((M, N), dtype=dtype, device=x.device) if y is None else y
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if xm_ws is None else xm_ws
        _check(lib().mmq_mxfp4(w.data_ptr(), x.data_ptr(), x_code, out.data_ptr(), y_code, M, N, K, ws.data_ptr(), s),
               "mmq_mxfp4")
        return out
    return _run(x, stream, call)


def mmq_mxfp4_mx(w: torch.Tensor, xm: torch.Tensor, M: int, N: int, K: int, y=None, dtype=torch.float32,
                 stream=None) -> torch.Tensor:
    """y [M, N] = xm [M, K] x w [N, K]^T, both MXFP4 buffers."""
    _mx(xm, M, K, "xm", xm)
    _mx_weights(w, N, K, xm)
    dtype, code = _given(y, dtype, (M, N), "y", xm)

    def call(s):
        out = torch.empty((M, N), dtype=dtype, device=xm.device) if y is None else y
        _check(lib().mmq_mxfp4_mx(w.data_ptr(), xm.data_ptr(), out.data_ptr(), code, M, N, K, s), "mmq_mxfp4_mx")
        return out
    return _run(xm, stream, call)


@functools.lru_cache(maxsize=4096)
def experts_sort_bytes(S: int, E: int) -> int:
    """Bytes of experts_sort's workspace (0: it needs none, or the shape is not supported)."""
    return int(lib().qpg_experts_sort_bytes(S, E))


def experts_sort(ids: torch.Tensor, E: int, offsets=None, order=None, slots=None, ws=None, stream=None):
    """ids [T, top_k] (int32 or int64) -> (offsets [E + 1], order [T * top_k], slots [T, top_k]), int32:
    the choices sorted by expert, stably. A choice outside [0, E) gets no row (slots -1); order
    is -1 behind the last row."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise QPGError(QPG_EINVAL, f"ids must be int32 or int64, got {ids.dtype}")
    _dev(ids, ids.dtype, "ids")
    if ids.dim() != 2:
        raise QPGError(QPG_EINVAL, f"ids must have 2 dimensions, got {tuple(ids.shape)}")
    S = ids.numel()
    if S < 1 or not 1 <= E <= 1024:
        raise QPGError(QPG_EINVAL, f"unsupported sort of {S} choices over {E} experts")
    for t, shape, name in ((offsets, (E + 1,), "offsets"), (order, (S,), "order"), (slots, ids.shape, "slots")):
        if t is not None:
            _is(t, torch.int32, shape, name, ids)
    nws = experts_sort_bytes(S, E)
    if ws is not None:
        _out(ws, torch.uint8, "ws", nws, ids)

    def call(s):
        o, r, p, w = offsets, order, slots, ws
        if o is None:
            o = torch.empty(E + 1, dtype=torch.int32, device=ids.device)
        if r is None:
            r = torch.empty(S, dtype=torch.int32, device=ids.device)
        if p is None:
            p = torch.empty(ids.shape, dtype=torch.int32, device=ids.device)
        if w is None and nws:
            w = torch.empty(nws, dtype=torch.uint8, device=ids.device)
        _check(lib().experts_sort(ids.data_ptr(), ids.element_size(), S, E, o.data_ptr(), r.data_ptr(), p.data_ptr(),
                                  None if w is None else w.data_ptr(), s), "experts_sort")
        return o, r, p
    return _run(ids, stream, call)


def mmq_mxfp4_experts(w: torch.Tensor, xm: torch.Tensor, rows: int, offsets: torch.Tensor, order, top_k: int, E: int,
                      N: int, K: int, y=None, dtype=torch.float32, stream=None) -> torch.Tensor:
    """y[p] = activation row x w[expert of p]^T for every sorted row p. w: MXFP4 of E * N rows, xm:
    MXFP4 of `rows` rows -- the tokens, read through order [S], S = rows * top_k (row order[p] //
    top_k; tokens that only pad a batch have choices outside [0, E)), or with order None the rows
    in sorted order themselves (S = rows). Rows of y behind the last (offsets[E]) are not written."""
    _mx(xm, rows, K, "xm", xm)
    _mx_weights(w, E * N, K, xm)
    _is(offsets, torch.int32, (E + 1,), "offsets", xm)
    S = rows
    if order is not None:
        S *= top_k
        _is(order, torch.int32, (S,), "order", xm)
    dtype, code = _given(y, dtype, (S, N), "y", xm)

    def call(s):
        out = torch.empty((S, N), dtype=dtype, device=xm.device) if y is None else y
        _check(lib().mmq_mxfp4_experts(w.data_ptr(), xm.data_ptr(), rows, offsets.data_ptr(),
                                       None if order is None else order.data_ptr(), top_k, out.data_ptr(), code, S, E, N,
                                       K, s), "mmq_mxfp4_experts")
        return out
    return _run(xm, stream, call)


def _slots(slots: torch.Tensor, ref: torch.Tensor):
    if slots.dtype is not torch.int32 or slots.get_device() != ref.get_device() or not slots.is_contiguous():
        _dev(slots, torch.int32, "slots")
        _same_device(slots, ref, "slots")
    if slots.dim() != 2:
        raise QPGError(QPG_EINVAL, f"slots must have 2 dimensions, got {tuple(slots.shape)}")
    return slots.shape


def experts_gather(x: torch.Tensor, slots: torch.Tensor, xs=None, stream=None) -> torch.Tensor:
    """xs [T * top_k, H]: row slots[t, j] is x[t]. Rows that no choice has are not written in an xs
    that is given, zeros in one allocated here."""
    code = _float(x, "x")
    T, top_k = _slots(slots, x)
    H = x.shape[1]
    if x.shape[0] != T:
        raise QPGError(QPG_EINVAL, f"x has {x.shape[0]} tokens, slots {T}")
    if xs is not None:
        _is(xs, x.dtype, (T * top_k, H), "xs", x)

    def call(s):
        out, f = xs, lib().experts_gather
        if xs is None:
            out, f = torch.empty((T * top_k, H), dtype=x.dtype, device=x.device), lib().experts_gather_zero
        _check(f(x.data_ptr(), code, slots.data_ptr(), out.data_ptr(), T, top_k, H, s), "experts_gather")
        return out
    return _run(x, stream, call)


def _combine(ys, slots, weights, y, dtype, stream, what):
    ys_code = _float(ys, "ys")
    T, top_k = _slots(slots, ys)
    H = ys.shape[1]
    if ys.shape[0] != T * top_k:
        raise QPGError(QPG_EINVAL, f"{ys.shape[0]} sorted rows, slots for {T * top_k}")
    if weights is not None:
        _is(weights, torch.float32, (T, top_k), "weights", ys)
    dtype, y_code = _given(y, ys.dtype if dtype is None else dtype, (T, H), "y", ys)

    def call(s):
        out = torch.empty((T, H), dtype=dtype, device=ys.device) if y is None else y
        _check(lib().experts_combine(ys.data_ptr(), ys_code, slots.data_ptr(),
                                     None if weights is None else weights.data_ptr(), out.data_ptr(), y_code, T, top_k, H,
                                     s), what)
        return out
    return _run(ys, stream, call)


def experts_gather_grad(dxs: torch.Tensor, slots: torch.Tensor, dx=None, stream=None) -> torch.Tensor:
    """Gradient of experts_gather: dx [T, H], dx[t] = sum over j of dxs[slots[t, j]] (of dxs's type)."""
    return _combine(dxs, slots, None, dx, None, stream, "experts_gather_grad")


def experts_combine(ys: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, y=None, dtype=None,
                    stream=None) -> torch.Tensor:
    """y [T, H]: y[t] = sum over j of weights[t, j] * ys[slots[t, j]]; choices without a row add nothing.
    dtype: y's type (ys's if neither is given)."""
    if weights is None:
        raise QPGError(QPG_EINVAL, "weights must be a float32 tensor")
    return _combine(ys, slots, weights, y, dtype, stream, "experts_combine")


def experts_combine_grad(dy: torch.Tensor, ys: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, dys=None,
                         dweights=None, stream=None):
    """Gradients of experts_combine: (dys [T * top_k, H] of ys's type, dweights [T, top_k] float32).
    Rows of dys that no choice has are not written in a dys that is given, zeros -- their gradient --
    in one allocated here."""
    dy_code, ys_code = _float(dy, "dy"), _float(ys, "ys")
    T, top_k = _slots(slots, ys)
    H = ys.shape[1]
    _is(dy, dy.dtype, (T, H), "dy", ys)
    _is(ys, ys.dtype, (T * top_k, H), "ys", ys)
    _is(weights, torch.float32, (T, top_k), "weights", ys)
    if dys is not None:
        _is(dys, ys.dtype, (T * top_k, H), "dys", ys)
    if dweights is not None:
        _is(dweights, torch.float32, (T, top_k), "dweights", ys)

    def call(s):
        d, f = dys, lib().experts_combine_grad
        if dys is None:
            d, f = torch.empty((T * top_k, H), dtype=ys.dtype, device=ys.device), lib().experts_combine_grad_zero
        dw = torch.empty((T, top_k), dtype=torch.float32, device=ys.device) if dweights is None else dweights
        _check(f(dy.data_ptr(), dy_code, ys.data_ptr(), ys_code, slots.data_ptr(), weights.data_ptr(), d.data_ptr(),
                 dw.data_ptr(), T, top_k, H, s), "experts_combine_grad")
        return d, dw
    return _run(ys, stream, call)
