"""Cases of the MXFP4 product named by the form they take: in WALKS of a tiled form the workgroups
have more tiles than one, so what is carried from a tile to the next (stage and scale buffers,
waits that count the stores in between, the next tile's early loads) is run with odd and even
numbers of K steps (256 values each), rows of scale bytes that are no whole dwords, odd widths.
test_forms_mx.py holds the cases to that on the CPU, test_gpu_mxfp4_walks.py runs them."""

FORMS = ("S16x16", "S16x32", "S32x16", "S32x32", "T64", "T64x128", "T128", "T256")

# form, tokens, N, K
DENSE = [
    ("T64x128", 40, 70_000, 544), ("T64x128", 33, 70_001, 800), ("T64x128", 40, 65_666, 1024), ("T64x128", 37, 70_000, 32),
    ("T128", 300, 40_000, 544), ("T128", 257, 40_001, 800), ("T128", 300, 40_000, 1056),
    ("T256", 4360, 4352, 544), ("T256", 4230, 4353, 800), ("T256", 4360, 4352, 1056),
]

# form, rows of each expert, choices without an expert, top_k, N, K
_T64 = [65] * 7 + [57]
EXPERTS = [
    ("T64", _T64, 0, 2, 4096, 32), ("T64", _T64, 0, 2, 4095, 544), ("T64", _T64, 0, 2, 4096, 1024), ("T64", _T64, 0, 2, 4094, 800),
    ("T64", [66, 65, 64, 65, 65, 65, 65, 50], 7, 4, 4096, 1056), ("T64", [65, 65, 0, 129, 65, 65, 65, 58], 0, 1, 4096, 1312),
    ("T64x128", [32] * 8, 0, 2, 11_008, 288), ("T64x128", [64, 65, 1, 0, 30, 32, 40, 24], 0, 2, 11_007, 544),
    ("T64x128", [30, 31, 33, 20, 37, 40, 25, 33], 7, 4, 11_008, 800),
    ("T128", [64] * 8, 0, 2, 11_008, 544), ("T128", [129, 1, 0, 128, 100, 50, 4, 90], 10, 1, 11_007, 800),
    ("T128", [129, 1, 0, 128, 100, 50, 4, 100], 0, 4, 11_008, 1056),
    ("T256", [513, 512, 511, 500, 600, 257, 1000, 203], 0, 2, 4100, 544),
    ("T256", [513, 512, 511, 500, 600, 257, 1000, 193], 10, 1, 4099, 800),
]
WALKS = [(f, [m], 0, None, n, k) for f, m, n, k in DENSE] + EXPERTS

# One of every form, for scale bytes of NaN (no walk asked for).
EVERY = [
    ("S16x16", [3, 0, 5, 8], 0, 2, 100, 1056), ("S16x32", [1, 2, 3, 4, 5, 6, 7, 4], 0, 2, 4100, 1056),
    ("S32x16", [20, 31], 1, 1, 1500, 544), ("S32x32", [20, 31], 1, 2, 3000, 544),
    ("T64", [65, 65, 0, 129, 65, 65, 65, 58], 0, 2, 4096, 1056), ("T64x128", [64, 65, 1, 0, 30, 32, 40, 24], 0, 2, 11_007, 544),
    ("T128", [129, 1, 0, 128, 100, 50, 4, 90], 10, 2, 11_008, 544),
    ("T256", [513, 512, 511, 500, 600, 257, 1000, 193], 10, 2, 4100, 544),
]
