"""The operators between a layer's projections, over a paged cache of keys and values, as cases to be timed and compared.

Three operators: appending new keys and values to the cache with the norm of each head and the rotation by position on
the way (which also gives the rotated queries), attention of new tokens over the cache, and attention of a tree of
drafted tokens over it. With `own` false `run` computes them in plain torch operations in 32 bits (angles in 64), with
`own` true through quantized_prefill_gemm_amd.

Cache: keys and values, each [pages][kv heads][page][dim]; table [B][width] names the pages of a sequence, lens [B] its
length with the new tokens, offsets [B + 1] the rows of the new tokens, which are the sequence's last.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _case(op, name=None, **more):
    base = {"op": op, "b": 1, "new": 1, "new_most": 0, "ctx": 0, "ctx_most": 0, "pad": 0, "heads": 32, "kv": 32, "dim": 128,
            "page": 64, "type": "bf16"}
    if op == "append":
        base.update(x="f32", fused=False, rot=128, adjacent=True, norm=False)
    else:
        base.update(y="bf16", cap=0.0, bias=False, window=0)
        base.update({"tree": 2} if op == "tree" else {"prefix": 0})
    return {**({"name": name} if name else {}), **base, **more}


def listed():
    return [
        # one decoded token of the 7B-shaped stack: products in 32 bits, half-precision cache
        _case("append", "append token", ctx=1023, type="f16"),
        # a decode batch padded to a graph's size, from one fused projection, heads of an odd size rotated in part
        _case("append", "append batch", b=57, ctx=3, ctx_most=2100, pad=7, heads=9, kv=3, dim=80, page=16, x="bf16",
              fused=True, rot=32, adjacent=False, norm=True),
        # prompts as they arrive, with norms of queries and keys
        _case("append", "append prompts", b=5, new=700, new_most=3300, heads=32, kv=8, x="bf16", adjacent=False, norm=True),
        # the same stack's token: its heads over a thousand cached tokens
        _case("attention", "attention token", ctx=1023, type="f16", y="f32"),
        # a decode batch with shared key heads over long and short caches
        _case("attention", "attention batch", b=64, ctx=130, ctx_most=8100, kv=8),
        # the stack's prompt, into the output projection's 32 bits
        _case("attention", "attention prompt", new=1024, type="f16", y="f32"),
        # a long prompt, the largest case
        _case("attention", "attention long prompt", new=8192, kv=8),
        # pieces of prompts over earlier pieces: capped scores, a sliding window, wide heads
        _case("attention", "attention capped window", b=3, new=600, new_most=1900, ctx=100, ctx_most=5000, heads=16, kv=8,
              dim=256, page=16, cap=50.0, window=1024),
        # prompts whose first part sees itself whole, beside others that are being decoded: scores fall with the distance
        _case("attention", "attention biased prefix", b=6, new=1, new_most=777, ctx=1, ctx_most=1500, heads=12, kv=12, dim=80,
              page=32, type="f16", y="f16", bias=True, prefix=129),
        # one user's drafted tokens
        _case("tree", "tree of one", new=26, ctx=2047, kv=8),
        # a batch of users' drafts
        _case("tree", "tree batch", b=16, new=33, new_most=64, ctx=500, ctx_most=4100, kv=8),
        # drafts of odd sizes and small heads over windows, capped
        _case("tree", "tree window", b=23, new=5, new_most=100, ctx=1, ctx_most=3000, heads=14, kv=2, dim=64, page=32, type="f16",
              y="f32", cap=30.0, window=777, tree=4),
    ]


MOST_PAIRS = 8192 * 8192 * 32                  # scores of the largest listed case, as the plain form lays them out
MOST_VALUES = 64 * 8101 * 8 * 128              # key values of the largest cache


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "tree"])
    while True:
        kv = _log(rng, 1, 32)
        heads = kv * _log(rng, 1, max(1, min(16, 64 // kv)))
        dim = rng.choice([64, 128, 128, 256, 8 * _log(rng, 2, 32)])
        few = rng.random() < 0.5                   # decoding, or prompts
        b = _log(rng, 1, 96 if few else 8)
        c = _case(op, b=b, heads=heads, kv=kv, dim=dim, page=rng.choice([16, 32, 64, 128, 256]),
                  type=rng.choice(["f16", "bf16"]), ctx=_log(rng, 1, 4000) - 1)
        c["ctx_most"] = rng.choice([0, c["ctx"] + _log(rng, 1, 8000)])
        if op == "append":
            c.update(x=rng.choice(["f32", "f16", "bf16"]), rot=rng.choice([dim, dim, 8 * rng.randint(0, dim // 8)]),
                     adjacent=rng.random() < 0.5, norm=rng.random() < 0.5, fused=rng.random() < 0.5,
                     pad=rng.choice([0, 0, rng.randint(1, 9)]))
        else:
            c.update(y=rng.choice([c["type"], c["type"], "f32"]), cap=rng.choice([0.0, 0.0, 30.0]),
                     bias=rng.random() < 0.25, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
        if op == "tree":
            c.update(new=_log(rng, 1, 64), tree=rng.randint(1, 5))
            c["new_most"] = rng.choice([0, c["new"] + rng.randint(1, 64)])
        elif not few:
            c["new"] = _log(rng, 2, 4096)
            c["new_most"] = rng.choice([0, c["new"] + _log(rng, 1, 4096)])
        if op == "attention":
            c["prefix"] = rng.choice([0, 0, 0, _log(rng, 1, 3000)])
        new, ctx = _sizes(c)
        length = max(n + k for n, k in zip(new, ctx))
        pairs = b * max(new) * length * heads
        if op == "append":
            pairs = 0
            if sum(new) * (heads + 2 * kv) * dim > 40_000_000:
                continue
        if pairs <= MOST_PAIRS // 2 and b * length * kv * dim <= MOST_VALUES // 2:
            return c


def _sizes(c):
    """New tokens and earlier ones of each sequence: spread between the case's least and most, the same for every seed."""
    new = [c["new"]] * c["b"]
    if c["new_most"]:
        new = [round(c["new"] * (c["new_most"] / c["new"]) ** ((i * 0.6180339887) % 1.0)) for i in range(c["b"])]
    ctx = [c["ctx"]] * c["b"]
    if c["ctx_most"]:
        ctx = [round(c["ctx"] + (c["ctx_most"] - c["ctx"]) * ((0.5 + i * 0.7548776662) % 1.0)) for i in range(c["b"])]
    return new, ctx


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(2_000_003 + int(seed))


def _normal(shape, gen, kind="f32", scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(TYPES[kind])


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _batch(c, gen):
    """The batch's index arrays: a pool with a few pages to spare, pages in no order."""
    new, ctx = _sizes(c)
    lens = [n + k for n, k in zip(new, ctx)]
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    need = [-(-n // c["page"]) for n in lens]
    width, pool = max(need), sum(need) + 3
    mixed = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((c["b"], width), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = mixed[at:at + n]
        at += n
    return {"new": new, "ctx": ctx, "table": table, "lens": _ints(lens), "offsets": _ints(offsets), "pool": pool,
            "rows": offsets[-1] + c["pad"], "most_new": max(new), "most_len": max(lens)}


def _tree(c, new, ctx, gen):
    """A random tree of each sequence's drafts: node 0 the root, each other one below one of the `tree` nodes before it.
    Rows of bits (a node's ancestors and itself) and positions."""
    words = -(-max(new) // 64)
    picks = torch.randint(1, c["tree"] + 1, (sum(new),), generator=gen, device=DEV).cpu().tolist()
    bits, positions, at = [], [], 0
    for n, k in zip(new, ctx):
        rows, depth = [], []
        for i in range(n):
            up = max(0, i - picks[at + i])
            rows.append((1 << i) | (rows[up] if i else 0))
            depth.append(depth[up] + 1 if i else 0)
        bits += rows
        positions += [k + d for d in depth]
        at += n
    whole = [[(r >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for r in bits]
    signed = [[v - 2 ** 64 if v >= 2 ** 63 else v for v in row] for row in whole]
    return torch.tensor(signed, dtype=torch.int64, device=DEV), _ints(positions)


def prepare(case, seed):
    gen, c = _gen(seed), case
    s = {"case": c, **_batch(c, gen)}
    rows, heads, kv, dim = s["rows"], c["heads"], c["kv"], c["dim"]
    pool = (s["pool"], kv, c["page"], dim)
    if c["op"] == "append":
        wide = [heads * dim, kv * dim, kv * dim]
        # a few channels of queries and keys are far larger than the rest
        gain = 1.0 + 10.0 * (torch.rand(heads * dim + kv * dim, generator=gen, device=DEV) < 0.02)
        x = torch.randn((rows, sum(wide)), generator=gen, device=DEV)
        x[:, : gain.numel()] *= gain
        x = x.to(TYPES[c["x"]])
        parts = x.split(wide, dim=1)
        s["q"], s["k"], s["v"] = parts if c["fused"] else [p.contiguous() for p in parts]
        s["kc"], s["vc"] = _normal(pool, gen, c["type"]), _normal(pool, gen, c["type"])
        s["freqs"] = None
        if c["rot"]:
            at = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV)
            s["freqs"] = torch.pow(torch.full_like(at, 10000.0), -at / c["rot"]).to(torch.float32)
        s["q_norm"] = 1.0 + _normal((dim,), gen, "f32", 0.2) if c["norm"] else None
        s["k_norm"] = 1.0 + _normal((dim,), gen, "f32", 0.2) if c["norm"] else None
        s["out"] = torch.zeros((rows, heads, dim), dtype=TYPES[c["type"]], device=DEV) if c["pad"] else None
        return s
    # keys share a direction that queries like more or less: rows between flat and peaked
    s["q"] = _normal((rows, heads, dim), gen, c["type"], 1.5)
    lean = torch.randn((1, kv, 1, dim), generator=gen, device=DEV)
    s["kc"] = torch.randn(pool, generator=gen, device=DEV).add_(0.5 * lean).to(TYPES[c["type"]])
    s["vc"] = _normal(pool, gen, c["type"])
    s["slopes"] = None
    if c["bias"]:
        s["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, heads + 1, dtype=torch.float32, device=DEV) / heads)
    if c["op"] == "tree":
        s["tree"], s["positions"] = _tree(c, s["new"], s["ctx"], gen)
    else:
        s["prefix"] = _ints([(c["prefix"] * (i + 1)) // c["b"] for i in range(c["b"])]) if c["prefix"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _rows(s):
    """Of each row: its sequence, its place among the new tokens, its place in the sequence. Rows behind the last
    sequence count as the last row that is in one."""
    offsets = s["offsets"].to(torch.int64)
    row = torch.minimum(torch.arange(s["rows"], device=DEV), offsets[-1] - 1)
    seq = (row.unsqueeze(1) >= offsets[1:].unsqueeze(0)).sum(dim=1)
    at = row - offsets[seq]
    return row, seq, at, s["lens"].to(torch.int64)[seq] - (offsets[seq + 1] - offsets[seq]) + at


def _normed(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight


def _rotated(x, c, cos, sin):
    """x [rows][heads][dim]; cos, sin [rows][1][rot / 2]."""
    rot = c["rot"]
    if not rot:
        return x
    part, rest = x[..., :rot], x[..., rot:]
    if c["adjacent"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_append(s, c):
    row, seq, _, place = _rows(s)
    cos = sin = None
    if c["rot"]:
        angle = place.double().unsqueeze(1) * s["freqs"].double().unsqueeze(0)
        cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    kind = TYPES[c["type"]]
    q, k, v = (s[n].float().reshape(s["rows"], -1, c["dim"])[row] for n in "qkv")
    q = _rotated(_normed(q, s["q_norm"]), c, cos, sin).to(kind)
    k = _rotated(_normed(k, s["k_norm"]), c, cos, sin).to(kind)
    page = s["table"].to(torch.int64)[seq, place // c["page"]]
    s["kc"][page, :, place % c["page"]] = k
    s["vc"][page, :, place % c["page"]] = v.to(kind)
    if s["out"] is not None:
        real = torch.arange(s["rows"], device=DEV) < s["offsets"][-1]
        q = torch.where(real.reshape(-1, 1, 1), q, s["out"])
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def _keys(cache, s, c):
    """[B][kv][length][dim] in 32 bits, zeros behind a sequence's end."""
    x = cache[s["table"].to(torch.int64)]                                    # [B][width][kv][page][dim]
    x = x.permute(0, 2, 1, 3, 4).reshape(c["b"], c["kv"], -1, c["dim"])[:, :, : s["most_len"]].float()
    real = torch.arange(s["most_len"], device=DEV) < s["lens"].unsqueeze(1)
    return torch.where(real[:, None, :, None], x, torch.zeros((), device=DEV))


def _plain_attention(s, c):
    b, kv, dim, group, most, length = c["b"], c["kv"], c["dim"], c["heads"] // c["kv"], s["most_new"], s["most_len"]
    offsets, lens = s["offsets"].to(torch.int64), s["lens"].to(torch.int64)
    new = offsets[1:] - offsets[:-1]
    begin = (lens - new).unsqueeze(1)
    i = torch.arange(most, device=DEV).unsqueeze(0)
    j = torch.arange(length, device=DEV).unsqueeze(0)
    at = torch.minimum(offsets[:-1].unsqueeze(1) + i, offsets[-1] - 1)       # [B][most]: rows of q
    here, there = begin + i, j.expand(b, length)                             # positions of queries and keys
    if c["op"] == "tree":
        node = (j - begin).clamp(min=0)                                      # [B][length]
        bits = torch.gather(s["tree"][at], 2, (node // 64).clamp(max=s["tree"].shape[1] - 1).unsqueeze(1).expand(b, most, length))
        kin = ((bits >> (node % 64).unsqueeze(1)) & 1).bool()
        key_row = torch.minimum(offsets[:-1].unsqueeze(1) + node, offsets[-1] - 1)
        here = s["positions"].to(torch.int64)[at]
        there = torch.where(j < begin, there, s["positions"].to(torch.int64)[key_row])
        seen = (j < begin).unsqueeze(1) | kin
    else:
        seen = there.unsqueeze(1) <= here.unsqueeze(2)
    gap = here.unsqueeze(2) - there.unsqueeze(1)                             # [B][most][length]
    if c["window"]:
        seen = seen & (gap < c["window"])
    if c["op"] == "attention" and s["prefix"] is not None:
        seen = seen | (j < s["prefix"].unsqueeze(1)).unsqueeze(1)
    seen = (seen & (j < lens.unsqueeze(1)).unsqueeze(1)).reshape(b, 1, 1, most, length)
    q = s["q"][at].float().reshape(b, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(b * kv, group * most, dim)
    k, v = (_keys(s[n], s, c).reshape(b * kv, length, dim) for n in ("kc", "vc"))
    x = torch.bmm(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(dim))
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x = x.reshape(b, kv, group, most, length)
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(1, kv, group, 1, 1) * gap.abs().float().reshape(b, 1, 1, most, length)
    x = torch.where(seen, x, torch.full((), -math.inf, device=DEV))
    top = x.amax(dim=-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.bmm(x.reshape(b * kv, group * most, length), v).reshape(b, kv, group, most, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    _, seq, inside, _ = _rows(s)
    return o.permute(0, 3, 1, 2, 4).reshape(b, most, c["heads"], dim)[seq, inside].to(TYPES[c["y"]])


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import quantized_prefill_gemm_amd as qpg
    c = s["case"]
    if c["op"] == "append":
        q = qpg.cache_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], s["offsets"], freqs=s["freqs"],
                             adjacent=c["adjacent"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, y=s["out"])
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if c["op"] == "attention":
        return qpg.cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["offsets"], cap=c["cap"],
                                   slopes=s["slopes"], window=c["window"], prefix=s["prefix"], dtype=TYPES[c["y"]])
    return qpg.cache_attention_tree(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["offsets"], s["tree"], s["positions"],
                                    cap=c["cap"], slopes=s["slopes"], window=c["window"], dtype=TYPES[c["y"]])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    return _plain_append(state, c) if c["op"] == "append" else _plain_attention(state, c)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, new, ctx = case, *_sizes(case)
    size = lambda kind: 4 if kind == "f32" else 2  # noqa: E731
    index = 4 * sum(-(-(n + k) // c["page"]) for n, k in zip(new, ctx)) + 8 * c["b"]
    if c["op"] == "append":
        values = sum(new) * (c["heads"] + 2 * c["kv"]) * c["dim"]
        return {"bytes": values * (size(c["x"]) + size(c["type"])) + index, "flops": (3 * bool(c["rot"]) + 4 * c["norm"]) * values}
    seen = keys = 0
    for i, (n, k) in enumerate(zip(new, ctx)):
        if c["op"] == "tree":
            near = k if not c["window"] else min(k, c["window"])
            seen += n * near + n * min(n, 2 + n // (c["tree"] + 1))       # a node has about so many ancestors
            keys += near + n
            continue
        first = (c["prefix"] * (i + 1)) // c["b"]
        length = n + k
        if c["window"]:
            seen += sum(min(k + t + 1, c["window"]) + max(0, min(first, length) - 0 if k + t + 1 < first else
                                                         min(first, k + t + 1 - c["window"])) for t in range(n))
            keys += min(length, max(0, min(first, length)) + n + c["window"])
        else:
            seen += sum(max(k + t + 1, min(first, length)) for t in range(n))
            keys += length
    rows = sum(new) * c["heads"] * c["dim"]
    return {"bytes": rows * (size(c["type"]) + size(c["y"])) + 2 * 2 * keys * c["kv"] * c["dim"] + index,
            "flops": 4 * seen * c["heads"] * c["dim"]}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_append(s, c):
    turned = {}
    place = torch.cat([torch.arange(k, k + n, device=DEV) for n, k in zip(s["new"], s["ctx"])])
    total, half = place.numel(), c["rot"] // 2
    for name, weight in (("q", s["q_norm"]), ("k", s["k_norm"]), ("v", None)):
        x = s[name][:total].double().reshape(total, -1, c["dim"])
        if weight is not None:
            x = weight.double() * x / torch.sqrt(x.pow(2).sum(dim=2, keepdim=True) / c["dim"] + EPS)
        if name != "v" and half:
            # a pair as one complex number, turned by the angle
            pair = [2 * torch.arange(half, device=DEV), 2 * torch.arange(half, device=DEV) + 1] if c["adjacent"] else \
                [torch.arange(half, device=DEV), torch.arange(half, device=DEV) + half]
            z = torch.complex(x[..., pair[0]], x[..., pair[1]])
            z = z * torch.exp(1j * (place.double()[:, None] * s["freqs"].double()[None, :]))[:, None, :]
            x = x.clone()
            x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
        turned[name] = x
    out = torch.zeros((s["rows"], c["heads"], c["dim"]), dtype=torch.float64, device=DEV)
    out[:total] = turned["q"]
    caches, at = [s["kc"].double(), s["vc"].double()], 0
    for i, (n, k) in enumerate(zip(s["new"], s["ctx"])):
        spot = torch.arange(k, k + n, device=DEV)
        page = s["table"][i].long()[spot // c["page"]]
        for cache, name in zip(caches, "kv"):
            cache[page, :, spot % c["page"]] = turned[name][at:at + n]
        at += n
    return {"q": out, "k": caches[0], "v": caches[1]}


def _exact_attention(s, c):
    out, at, group = [], 0, c["heads"] // c["kv"]
    for i, (n, k) in enumerate(zip(s["new"], s["ctx"])):
        length = n + k
        spot = torch.arange(length, device=DEV)
        page = s["table"][i].long()[spot // c["page"]]
        where_q = torch.arange(k, length, device=DEV)
        where_k = spot.clone()
        if c["op"] == "tree":
            where_q = s["positions"][at:at + n].long()
            where_k[k:] = where_q
            node = torch.arange(n, device=DEV)
            see = torch.ones((n, length), dtype=torch.bool, device=DEV)
            see[:, k:] = (torch.bitwise_right_shift(s["tree"][at:at + n][:, node // 64], node % 64) % 2) != 0
        else:
            see = where_k[None, :] <= where_q[:, None]
        far = where_q[:, None] - where_k[None, :]
        if c["window"]:
            see = torch.logical_and(see, far < c["window"])
        if c["op"] == "attention" and s["prefix"] is not None:
            see = torch.logical_or(see, spot[None, :] < int(s["prefix"][i]))
        heads = []
        for h in range(c["heads"]):
            keys = s["kc"][page, h // group, spot % c["page"]].double()
            values = s["vc"][page, h // group, spot % c["page"]].double()
            score = (s["q"][at:at + n, h].double() @ keys.t()) / math.sqrt(c["dim"])
            if c["cap"]:
                score = c["cap"] * torch.tanh(score / c["cap"])
            if s["slopes"] is not None:
                score = score - float(s["slopes"][h]) * far.abs().double()
            score = score.masked_fill(~see, -math.inf)
            share = torch.softmax(score, dim=1).masked_fill(~see, 0.0)      # a row that sees nothing: zeros
            heads.append(share @ values)
        out.append(torch.stack(heads, dim=1))
        at += n
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s, case) if case["op"] == "append" else _exact_attention(s, case)
