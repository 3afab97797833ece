"""The 7B-shaped prefill GEMM stack on one GPU: per layer the seven projections (q, k, v, o:
4096 x 4096; gate, up: 11008 x 4096; down: 4096 x 11008; q4_K except v and down, which are
q6_K), each fed by the q8_1 quantisation of its input. Orchestration only: every step is a
call into libqpg (quantize_q8_1, then the MMQ entry of the weight's form), in stream order,
so a pass can be launched eagerly or captured into one HIP graph (torch's graph API over the
library's own launches).

q, k and v read the same hidden state, gate and up the same normed state, so with quantize
sharing one quantize_q8_1 serves each group: 4 per layer instead of 7
(the prepass the pages run once per distinct activation, "31 - r28 - Direction-A raw-nibble
NB kernel", sec. 3.2).
"""
from __future__ import annotations

import torch

from . import binding as B
from .inputs import STACK_LAYER

# matrix position -> position whose input (and, with sharing, whose q8_1 buffer) it reads
SOURCE = {0: 0, 1: 0, 2: 0, 3: 3, 4: 4, 5: 4, 6: 6}
SOURCES = (0, 3, 4, 6)
MODES = ("all", "shared", "gemm")


class Stack:
    """Weights resident on the device, inputs / q8_1 buffers / outputs allocated once.

    weights[layer][idx]: raw q4_K / q6_K block buffers (uint8 device tensors) in the order of
    STACK_LAYER. q6: weight form of the q6_K matrices -- "raw" blocks, "prepared" or
    "expanded" (made here once, outside any pass). per_layer: every layer gets its own inputs
    and outputs (what a test compares); otherwise one input and one output per matrix
    position, reused by every layer (the layers then differ only in their weights, which is
    all the GEMM cost depends on).
    """

    def __init__(self, weights, M: int, q6: str = "expanded", per_layer: bool = False):
        if q6 not in ("raw", "prepared", "expanded"):
            raise ValueError(f"q6 form {q6!r}")
        self.M, self.q6, self.per_layer = M, q6, per_layer
        self.L = len(weights)
        dev = weights[0][0].device
        self.mats = []
        for layer in range(self.L):
            row = []
            for idx, (name, wtype, N, K) in enumerate(STACK_LAYER):
                w = weights[layer][idx]
                if wtype == "q6_K" and q6 == "prepared":
                    w = B.q6K_prepare(w, N, K)
                elif wtype == "q6_K" and q6 == "expanded":
                    w = B.q6K_expand(w, N, K)
                row.append(w)
            self.mats.append(row)
        nio = self.L if per_layer else 1
        self.x = [{src: torch.zeros((M, STACK_LAYER[src][3]), dtype=torch.float32, device=dev) for src in SOURCES}
                  for _ in range(nio)]
        self.xq = [[torch.empty(B.q8_1_bytes(M, K), dtype=torch.uint8, device=dev) for (_, _, _, K) in STACK_LAYER]
                   for _ in range(nio)]
        self.y = [[torch.empty((M, N), dtype=torch.float32, device=dev) for (_, _, N, _) in STACK_LAYER]
                  for _ in range(nio)]

    def io(self, layer: int) -> int:
        return layer if self.per_layer else 0

    def set_input(self, layer: int, src: int, x: torch.Tensor):
        """Input of the matrices reading position src (0: q/k/v, 3: o, 4: gate/up, 6: down)."""
        self.x[self.io(layer)][src].copy_(x)

    def output(self, layer: int, idx: int) -> torch.Tensor:
        return self.y[self.io(layer)][idx]

    def _gemm(self, layer: int, idx: int, xq: torch.Tensor, stream):
        _, wtype, N, K = STACK_LAYER[idx]
        w, y, M = self.mats[layer][idx], self.output(layer, idx), self.M
        if wtype == "q4_K":
            B.mmq_q4K_q8(w, xq, M, N, K, y, stream=stream)
        elif self.q6 == "prepared":
            B.mmq_q6K_prep_q8(w, xq, M, N, K, y, stream=stream)
        elif self.q6 == "expanded":
            B.mmq_q6K_exp_q8(w, xq, M, N, K, y, stream=stream)
        else:
            B.mmq_q6K_q8(w, xq, M, N, K, y, stream=stream)

    def run(self, mode: str = "shared", stream=None):
        """Enqueue one pass over all layers on `stream` (torch's current stream if None).
        all: a quantize_q8_1 before each of the 7 GEMMs of a layer; shared: one per distinct
        input (4 per layer); gemm: the shared pass without its quantizes (the GEMMs alone, on
        the q8_1 buffers a previous pass left)."""
        if mode not in MODES:
            raise ValueError(f"mode {mode!r}")
        for layer in range(self.L):
            io = self.io(layer)
            for idx in range(len(STACK_LAYER)):
                src = SOURCE[idx]
                if mode == "all":
                    B.quantize_q8_1(self.x[io][src], self.xq[io][idx], stream=stream)
                    self._gemm(layer, idx, self.xq[io][idx], stream)
                elif mode == "shared":
                    if src == idx:
                        B.quantize_q8_1(self.x[io][src], self.xq[io][src], stream=stream)
                    self._gemm(layer, idx, self.xq[io][src], stream)
                else:
                    self._gemm(layer, idx, self.xq[io][src], stream)

    def capture(self, mode: str = "shared") -> torch.cuda.CUDAGraph:
        """One pass captured as a graph: an eager pass on a side stream first (the library's
        first calls query the device), then the capture."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.run(mode)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run(mode)
        return g

    def macs(self) -> int:
        return self.M * self.L * sum(N * K for _, _, N, K in STACK_LAYER)


class ExpertStack(Stack):
    """The stack with experts in place of gate, up and down: per layer the four attention
    projections as in Stack, then each token's top_k experts of E, their matrices MXFP4.

    weights[layer]: q, k, v, o block buffers. experts[layer]: the (gate, up, down) MXFP4 buffers,
    each of E * N rows in expert order. set_routing gives a layer's choices and their weights.
    Position 4 reads the token states [M, 4096], which gate and up take through the sort's order;
    position 6 reads rows already in sorted order [M * top_k, 11008]; outputs 4 and 5 are in
    sorted order, output 6 is the weighted sum over a token's choices [M, 4096]. As in Stack
    the products' inputs are given, none is made from another's output.
    """

    ATTENTION = 4                     # positions 0 .. 3; 4, 5, 6: gate, up, down

    def __init__(self, weights, experts, M: int, E: int, top_k: int, q6: str = "expanded", per_layer: bool = False):
        if len(weights) != len(experts):
            raise ValueError(f"{len(weights)} layers of projections, {len(experts)} of experts")
        if not 1 <= top_k <= E:
            raise ValueError(f"{top_k} choices of {E} experts")
        if q6 not in ("raw", "prepared", "expanded"):
            raise ValueError(f"q6 form {q6!r}")
        self.M, self.E, self.top_k, self.S = M, E, top_k, M * top_k
        self.q6, self.per_layer, self.L = q6, per_layer, len(weights)
        dev = weights[0][0].device
        self.mats = [[self._form(w, *STACK_LAYER[idx][1:]) for idx, w in enumerate(row)] for row in weights]
        self.experts = experts
        nio, S = (self.L if per_layer else 1), self.S
        rows = (M, M, M, M, S, S, M)

        def new(shape, dtype=torch.float32):
            return [torch.empty(shape, dtype=dtype, device=dev) for _ in range(nio)]
        self.x = [{src: torch.zeros((S if src == 6 else M, STACK_LAYER[src][3]), dtype=torch.float32, device=dev)
                   for src in SOURCES} for _ in range(nio)]
        self.xq = [[torch.empty(B.q8_1_bytes(M, K), dtype=torch.uint8, device=dev) for _, _, _, K in STACK_LAYER[:4]]
                   for _ in range(nio)]
        self.xm = [{src: torch.empty(B.mxfp4_bytes(S if src == 6 else M, STACK_LAYER[src][3]), dtype=torch.uint8,
                                     device=dev) for src in (4, 6)} for _ in range(nio)]
        self.y = [[torch.empty((rows[i], N), dtype=torch.float32, device=dev) for i, (_, _, N, _) in enumerate(STACK_LAYER)]
                  for _ in range(nio)]
        self.down = new((S, STACK_LAYER[6][2]))
        self.ids = [torch.zeros((M, top_k), dtype=torch.int64, device=dev) for _ in range(nio)]
        self.gains = [torch.zeros((M, top_k), dtype=torch.float32, device=dev) for _ in range(nio)]
        self.offsets, self.order, self.slots = new(E + 1, torch.int32), new(S, torch.int32), new((M, top_k), torch.int32)
        self.sort_ws = new(max(B.experts_sort_bytes(S, E), 1), torch.uint8)

    def _form(self, w, wtype, N, K):
        if wtype != "q6_K" or self.q6 == "raw":
            return w
        return B.q6K_prepare(w, N, K) if self.q6 == "prepared" else B.q6K_expand(w, N, K)

    def set_routing(self, layer: int, ids: torch.Tensor, gains: torch.Tensor):
        """The experts [M, top_k] that each token of the layer goes to, and their weights."""
        self.ids[self.io(layer)].copy_(ids)
        self.gains[self.io(layer)].copy_(gains)

    def _experts(self, layer: int, idx: int, stream):
        io, (_, _, N, K) = self.io(layer), STACK_LAYER[idx]
        w = self.experts[layer][idx - self.ATTENTION]
        if idx < 6:
            B.mmq_mxfp4_experts(w, self.xm[io][4], self.M, self.offsets[io], self.order[io], self.top_k, self.E, N, K,
                                self.y[io][idx], stream=stream)
        else:
            B.mmq_mxfp4_experts(w, self.xm[io][6], self.S, self.offsets[io], None, 1, self.E, N, K, self.down[io],
                                stream=stream)
            B.experts_combine(self.down[io], self.slots[io], self.gains[io], self.y[io][6], stream=stream)

    def run(self, mode: str = "shared", stream=None):
        """As Stack.run. The sort runs once per layer in `all` and `shared`; `gemm` works on the
        buffers and the order that a previous pass left."""
        if mode not in MODES:
            raise ValueError(f"mode {mode!r}")
        for layer in range(self.L):
            io = self.io(layer)
            for idx in range(self.ATTENTION):
                src = SOURCE[idx]
                at = idx if mode == "all" else src
                if mode == "all" or (mode == "shared" and src == idx):
                    B.quantize_q8_1(self.x[io][src], self.xq[io][at], stream=stream)
                self._gemm(layer, idx, self.xq[io][at], stream)
            if mode != "gemm":
                B.experts_sort(self.ids[io], self.E, self.offsets[io], self.order[io], self.slots[io], self.sort_ws[io],
                               stream=stream)
            for idx in (4, 5, 6):
                src = SOURCE[idx]
                if mode == "all" or (mode == "shared" and src == idx):
                    B.quantize_mxfp4(self.x[io][src], self.xm[io][src], stream=stream)
                self._experts(layer, idx, stream)

    def macs(self) -> int:
        """Of a pass whose choices all have an expert."""
        attention = self.M * sum(N * K for _, _, N, K in STACK_LAYER[:4])
        return self.L * (attention + self.S * sum(N * K for _, _, N, K in STACK_LAYER[4:]))
