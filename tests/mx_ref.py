"""MXFP4 and the expert operators in 64 bits on the CPU, written from their definitions: what the
GPU tests compare with. Nothing here is used by the library."""
import math

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def encode(x):
    """Values [rows][K] -> (codes uint8 [rows][K], scale bytes uint8 [rows][K/32]). The nearest
    code by its distance, the even one of two that are equally near."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, 32)
    finite = np.isfinite(b).all(axis=2)
    b = np.where(finite[:, :, None], b, 0.0)
    amax = np.abs(b).max(axis=2)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1, -10000) - 2 + 127
    e = np.maximum(e, 0)
    v = b / np.ldexp(1.0, e - 127)[:, :, None]
    dist = np.abs(np.abs(v)[..., None] - GRID)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    code = np.where(finite[:, :, None], code + 8 * np.signbit(np.where(finite[:, :, None], v, 0.0)), 0)
    return code.astype(np.uint8).reshape(x.shape), np.where(finite, e, 255).astype(np.uint8)


def pack(codes, scales):
    """The MXFP4 buffer of codes and scale bytes."""
    return np.concatenate([(codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(-1), scales.reshape(-1)])


def unpack(buf, rows, K):
    p = buf[: rows * K // 2].reshape(rows, K // 2)
    codes = np.stack([p & 15, p >> 4], axis=2).reshape(rows, K)
    return codes, buf[rows * K // 2: rows * K // 2 + rows * K // 32].reshape(rows, K // 32)


def decode(codes, scales):
    power = np.array([math.ldexp(1.0, i - 127) for i in range(255)] + [math.nan])
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        return v * np.repeat(power[scales], 32, axis=1)


def values(buf, rows, K):
    return decode(*unpack(buf, rows, K))


def weights(rows, K, rng, scale=0.02):
    """An MXFP4 buffer of normal weights."""
    return pack(*encode((rng.standard_normal((rows, K)) * scale).astype(np.float32)))


# Half a step of a stored type, relative, and the distance below which its values are even
# (half the smallest subnormal).
HALF = {"float32": (2.0 ** -24, 2.0 ** -150), "float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}


def rounding(y, kind):
    rel, least = HALF[kind]
    return np.abs(y) * rel + least


def product_bound(x, w, y, kind):
    """How far a product may be from its exact value y = x w^T. A matrix step adds 64 or 128
    exact products and the running f32 sum; its result is within one f32 step (2^-23) of the sum
    of the magnitudes, and at most K/64 steps and 8 partial sums follow each other:
    (K/64 + 9) * 2^-23 * (|x| |w|^T), then the rounding to the stored type."""
    K = x.shape[1]
    with np.errstate(invalid="ignore"):
        return (K / 64 + 9) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 1.0001 * rounding(y, kind)


def sort(ids, E):
    """offsets, order, slots of ids [T][top_k]."""
    flat = [int(v) for v in ids.reshape(-1)]
    by = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    order = np.full(len(flat), -1, dtype=np.int32)
    order[: len(by)] = [i for _, i in by]
    slots = np.full(len(flat), -1, dtype=np.int32)
    slots[order[: len(by)]] = np.arange(len(by))
    counts = np.bincount([e for e, _ in by], minlength=E) if by else np.zeros(E, dtype=np.int64)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order, slots.reshape(ids.shape)
