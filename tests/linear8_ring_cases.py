"""Shapes whose products in 8-bit floating point run through their stages' and scales' rings
more than once: more steps than the eight whose scales are held, by tiles of one set of
wavefronts, with the scales of four steps loaded at once and one by one, contractions that
end inside a block and inside 16 bytes.

name: m, n, k, activation, gated, scales, tile, split, steps of a split, whole groups of
four, alone"""
CASES = {
    "256, 12 steps": (4090, 4088, 1500, "none", False, "pow2", "256", False, 12, True, True),
    "256, 16 steps, others late": (4090, 4088, 2041, "relu", False, "late", "256", False, 16, True, True),
    "256, 14 steps one by one": (4090, 4088, 1700, "none", False, "late", "256", False, 14, False, True),
    "256, 12 steps, others": (4090, 4088, 1500, "none", False, "any", "256", False, 12, True, True),
    "256 gated, 12 steps": (4090, 2044, 1500, "silu", True, "pow2", "256", False, 12, True, True),
    "256 gated, 16 steps, others late": (4090, 2044, 2041, "silu", True, "late", "256", False, 16, True, True),
    "256 gated, 14 steps one by one": (4090, 2044, 1700, "gelu", True, "one", "256", False, 14, False, True),
    "256 gated, 12 steps, others": (4090, 2044, 1500, "silu", True, "any", "256", False, 12, True, True),
    "128, 12 steps": (2040, 4080, 1500, "none", False, "one", "128", False, 12, True, False),
    "128, 16 steps, others late": (2040, 4080, 2041, "none", False, "late", "128", False, 16, True, False),
    "128 gated, 16 steps": (2040, 2040, 2041, "silu", True, "pow2", "128", False, 16, True, False),
    "128 gated, 12 steps, others": (2040, 2040, 1500, "silu", True, "any", "128", False, 12, True, False),
    "128 alone, 14 steps": (1530, 1530, 1700, "none", False, "late", "128", False, 14, False, True),
    "128 split, 20 steps": (700, 900, 12200, "none", False, "late", "128", True, 20, True, True),
    "128 split, 43 steps one by one": (1530, 1530, 16300, "none", False, "one", "128", True, 43, False, False),
    "64, 12 steps": (1270, 1270, 1500, "none", False, "one", "64", False, 12, True, False),
    "64, 16 steps, others late": (1270, 1270, 2041, "relu", False, "late", "64", False, 16, True, False),
    "64, 16 steps": (1270, 1270, 2041, "none", False, "pow2", "64", False, 16, True, False),
    "64 gated, 16 steps, others late": (1270, 635, 2041, "silu", True, "late", "64", False, 16, True, False),
    "64 alone, 12 steps": (600, 1000, 1500, "none", False, "late", "64", False, 12, True, True),
}
