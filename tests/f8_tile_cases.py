"""Products of the 8-bit floating-point calls that reach each kind of tile: the shapes
that tests/test_gpu_f8_tiles.py runs and tests/test_f8_kinds.py follows to their
launchers, so that a change of the planner's costs cannot leave a kernel without a test.

A case: (name, outputs, products), a product (m, n, k, fp32 scales, squares of B, kind).
m, n and k are ragged: rows and columns that end inside a tile, k of every kind that the
tiles' rings and tails know (a multiple of 128, of 16, of neither; even and odd counts of
blocks)."""

# large tiles: four columns of outputs at a time, one-byte scales
LARGE = [(4084, 4036, k, False, True, "big") for k in (1500, 2049, 2176, 4001)]
# mid ones, bf16: columns that do not go four at a time
MID_BF16 = [(2029, 4094, k, False, True, "mid") for k in (2700, 2817, 3000, 4001)]
# mid ones, fp32 outputs of fp32 scales, for squares of B and for each row
MID_FP32 = [(2029, 4036, k, True, square, "mid") for k in (700, 1025, 1264) for square in (True, False)]
# small ones: fp32 scales and bf16 outputs, one-byte scales and fp32 outputs, cut sums
SMALL_ANY = [(1029, 1030, k, True, square, "small") for k in (640, 1025) for square in (True, False)]
SMALL_WIDE = [(2029, 4095, 1500, False, True, "small")]
CUT = [(300, 260, 5000, False, True, "cut")]
# a list of experts in one launch of mid tiles, one of them of few tokens
EXPERTS = [(m, 2046, 6100, False, True, "few" if m <= 32 else "mid")
           for m in (200, 130, 31, 190, 129, 250, 170, 225, 140, 160, 230, 135, 199)]

# kinds side by side: no product takes a kind for another's sake
MIXED = [(2029, 4094, 3000, False, True, "mid"), (300, 520, 3000, True, True, "cut"), (20, 260, 3000, False, True, "few")]
MIXED_FP32 = [(2029, 4036, 1025, True, True, "mid"), (300, 519, 1025, False, True, "small")]
# large tiles of an aligned output whose small tiles would be cut in two: (m, n, k, dtype)
PLACED = [(2456, 3240, 15540, "bf16"), (1707, 4668, 15774, "bf16"), (2438, 4904, 13875, "fp32")]

CASES = [("large", dtype, [p]) for dtype in ("bf16", "fp32") for p in LARGE] + \
        [("mid", "bf16", [p]) for p in MID_BF16] + [("mid", "fp32", [p]) for p in MID_FP32] + \
        [("small", "bf16", [p]) for p in SMALL_ANY] + [("small", "fp32", [p]) for p in SMALL_WIDE] + \
        [("cut", dtype, [p]) for dtype in ("bf16", "fp32") for p in CUT] + \
        [("experts", "bf16", EXPERTS), ("mixed", "bf16", MIXED), ("mixed", "fp32", MIXED_FP32)]


def name_of(case):
    name, dtype, products = case
    m, n, k, any_, square, _ = products[0]
    return f"{name}-{dtype}-{len(products)}x{m}x{n}x{k}{'-fp32scales' if any_ else ''}{'-squares' if square else ''}"
