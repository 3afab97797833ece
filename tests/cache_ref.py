"""The operators over a paged cache in 64 bits on the CPU, and how far from it a kernel may be.

Bounds: an f32 operation is off by half a step (2^-24 relative), a value rounded to a type by eps / 2. A
score is a sum of `dim` products (exact in f32) in f32: within dim * 2^-24 of the sum of their magnitudes; scaling,
bias, cap and the power's argument add a few steps of the values they have. A share is off by its score's error, twice
(once through the maximum), the power's and the rounding to the cache's type (unless the output has more bits). The
sums of n shares, and of n products, are each within n * 2^-24 of the sum of magnitudes.
"""
import math

import torch

F64 = torch.float64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STEP = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


class Batch:
    """new[b] tokens at the end of each sequence of lens[b], rows in no sequence before and behind, pages in
    no order; everything in the pool that is no token is NaN."""

    def __init__(self, new, lens, kv, dim, page, kind, seed=0, lead=0, pad=0, spare=2, extra_width=0):
        g = self.gen = torch.Generator().manual_seed(seed)
        self.new, self.lens_list, self.kv, self.dim, self.page, self.kind = new, lens, kv, dim, page, kind
        self.dtype = TYPES[kind]
        offsets = [lead]
        for n in new:
            offsets.append(offsets[-1] + n)
        self.rows = offsets[-1] + pad
        need = [-(-n // page) for n in lens]
        self.width = max(max(need), 1) + extra_width
        self.pool = sum(need) + spare
        mixed = torch.randperm(self.pool, generator=g)
        self.table = torch.full((len(new), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = mixed[at:at + n].to(torch.int32)
            at += n
        self.lens, self.offsets = (torch.tensor(x, dtype=torch.int32) for x in (lens, offsets))
        self.k, self.v = (torch.full((self.pool, kv, page, dim), math.nan, dtype=self.dtype) for _ in range(2))
        for b, n in enumerate(lens):
            for c in (self.k, self.v):
                rows = torch.randn((n, kv, dim), generator=g).to(self.dtype)
                for p in range(need[b]):
                    part = rows[p * page:(p + 1) * page]
                    c[self.table[b, p], :, :len(part)] = part.permute(1, 0, 2)

    def normal(self, *shape, scale=1.0, kind=None):
        return (torch.randn(shape, generator=self.gen) * scale).to(TYPES[kind or self.kind])

    def keys(self, b, cache):
        """[len][kv][dim] of sequence b, as stored."""
        spot = torch.arange(self.lens_list[b])
        return cache[self.table[b].long()[spot // self.page], :, spot % self.page]

    def index(self, device):
        return [t.to(device) for t in (self.table, self.lens, self.offsets)]


def tree_of(gen, new, branch):
    """Parents at most `branch` nodes back -> rows of bits (as Python ints) and depths, sequence by sequence."""
    bits, depths = [], []
    for n in new:
        mine, deep = [], []
        for i in range(n):
            up = max(0, i - int(torch.randint(1, branch + 1, (1,), generator=gen)))
            mine.append((1 << i) | (mine[up] if i else 0))
            deep.append(deep[up] + 1 if i else 0)
        bits += mine
        depths += deep
    return bits, depths


def words_of(bits, rows, lead, words):
    t = torch.zeros((rows, words), dtype=torch.int64)
    for i, x in enumerate(bits):
        for w in range(words):
            v = (x >> (64 * w)) & (2 ** 64 - 1)
            t[lead + i, w] = v - 2 ** 64 if v >= 2 ** 63 else v
    return t


def attention(batch, q, y_type, scale=None, cap=0.0, slopes=None, window=0, prefix=None, tree=None, positions=None):
    """(y [rows][heads][dim] in 64 bits, bound of the same shape, which rows are in a sequence)."""
    heads, dim = q.shape[1], q.shape[2]
    group = heads // batch.kv
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    y = torch.zeros(q.shape, dtype=F64)
    bound = torch.zeros(q.shape, dtype=F64)
    mine = torch.zeros(batch.rows, dtype=torch.bool)
    y_type = TYPES[y_type]
    # shares of more bits than the cache's type where the output has more
    u = half(batch.dtype) if half(y_type) >= half(batch.dtype) else 4 * STEP
    for b, (n, length) in enumerate(zip(batch.new, batch.lens_list)):
        r0 = int(batch.offsets[b])
        if n == 0:
            continue
        mine[r0:r0 + n] = True
        if length == 0:
            continue
        k, v = (batch.keys(b, c).to(F64) for c in (batch.k, batch.v))
        ctx = length - n
        here = torch.arange(ctx, length)
        there = torch.arange(length)
        j = torch.arange(length)
        if tree is not None:
            here = positions[r0:r0 + n].long()
            there = torch.cat([there[:max(ctx, 0)], here])
            see = torch.ones((n, length), dtype=torch.bool)
            for i in range(n):
                for m in range(n):
                    word = int(tree[r0 + i, m // 64]) if m < 64 * tree.shape[1] else 0
                    see[i, ctx + m] = bool((word >> (m % 64)) & 1)
        else:
            see = there[None, :] <= here[:, None]
        far = here[:, None] - there[None, :]
        if window:
            see &= far < window
        if prefix is not None:
            see |= j[None, :] < int(prefix[b])
        for h in range(heads):
            qh, kh, vh = q[r0:r0 + n, h].to(F64), k[:, h // group], v[:, h // group]
            s = scale * (qh @ kh.T)
            size = scale * (qh.abs() @ kh.abs().T)
            off = (dim + 8) * STEP * size
            if cap:
                s = cap * torch.tanh(s / cap)
                # 1 - 2 / (e + 1): a few steps of 1, times the cap; with a finer output or a large cap of the value itself
                off = off + (16 * STEP * cap if u == half(batch.dtype) and cap <= 128 else 16 * STEP * s.abs())
            if slopes is not None:
                bias = float(slopes[h]) * far.abs().to(F64)
                s = s - bias
                off = off + 8 * STEP * (bias + s.abs())
            off = off + 8 * STEP * s.abs()
            s = torch.where(see, s, torch.full((), -math.inf, dtype=F64))
            top = s.amax(dim=1, keepdim=True)
            w = torch.where(see, torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top)), torch.zeros((), dtype=F64))
            total = w.sum(dim=1, keepdim=True)
            w = w / torch.where(total > 0, total, torch.ones_like(total))
            # a sum over what a row sees alone: values that are no numbers count by where they are seen
            vs = torch.where(torch.isfinite(vh), vh, torch.zeros((), dtype=F64))
            up, down = (see.to(F64) @ (torch.isnan(vh) | (vh == x)).to(F64) > 0 for x in (math.inf, -math.inf))
            y[r0:r0 + n, h] = w @ vs + torch.where(up, math.inf, 0.0) - torch.where(down, math.inf, 0.0)
            size = w @ vs.abs()
            worst = torch.where(see, off, torch.zeros((), dtype=F64)).amax(dim=1, keepdim=True)
            rel = 2 * torch.expm1(worst) + u + (2 * length + 64) * STEP
            least = length * 2.0 ** -31 * vs.abs().max() if batch.kind == "f16" else 0.0       # shares below f16's normal numbers
            bound[r0:r0 + n, h] = rel * size + least
    tiny = 2.0 ** -25 if y_type == torch.float16 else 0.0
    return y, bound * (1 + half(y_type)) + half(y_type) * y.abs() + tiny, mine


def append(batch, q, k, v, freqs=None, positions=None, adjacent=False, q_norm=None, k_norm=None, eps=1e-6):
    """(values, bounds) of q's rows [rows][heads][dim], k's and v's [rows][kv][dim], and (row, page, place) of the
    rows that have a place."""
    dim, places, where = batch.dim, {}, []
    for b, (n, length) in enumerate(zip(batch.new, batch.lens_list)):
        r0 = int(batch.offsets[b])
        for i in range(n):
            p = length - n + i
            places[r0 + i] = p
            if p >= 0 and 0 <= int(batch.table[b, p // batch.page]) < batch.pool:
                where.append((r0 + i, int(batch.table[b, p // batch.page]), p % batch.page))
    at = torch.tensor([places.get(r, 0) for r in range(batch.rows)], dtype=F64) if positions is None else positions.to(F64)
    out = []
    for x, norm, turn in ((q, q_norm, True), (k, k_norm, True), (v, None, False)):
        if x is None:
            out.append((None, None))
            continue
        y = x.to(F64).reshape(batch.rows, -1, dim)
        off = torch.zeros_like(y)
        if norm is not None:
            y = y / torch.sqrt((y * y).mean(dim=2, keepdim=True) + eps) * norm.to(F64)
            off = (dim / 2 + 8) * STEP * y.abs()           # the square root halves the sum's error
        if turn and freqs is not None:
            rot = 2 * freqs.numel()
            a, b = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if adjacent else \
                (torch.arange(rot // 2), torch.arange(rot // 2, rot))
            angle = at[:, None, None] * freqs.to(F64)[None, None, :]
            cos, sin = torch.cos(angle), torch.sin(angle)
            # the angle in f32 turns once its fraction is taken, f32's sine and cosine, and 64 bits of the product
            e = 16 * STEP + 2.0 ** -50 * angle.abs()
            p, r, op, orr = y[..., a], y[..., b], off[..., a], off[..., b]
            size = p.abs() + r.abs()
            y, off = y.clone(), off.clone()
            y[..., a], y[..., b] = p * cos - r * sin, p * sin + r * cos
            off[..., a] = off[..., b] = op + orr + size * e
        tiny = 2.0 ** -25 if batch.dtype == torch.float16 else 0.0
        out.append((y, off * (1 + half(batch.dtype)) + half(batch.dtype) * y.abs() + tiny))
    return out, where
