"""Shapes whose products in 8-bit floating point take each tile, alone on a compute unit
or not and with the contraction split, with edges cut in both directions and
contractions that end inside a block.

name: m, n, k, activation, gated, scales, tile, split, alone"""
TILES = {"256": 0, "128": 2, "64": 3}
CASES = {
    "256": (4090, 4088, 200, "none", False, "pow2", "256", False, True),
    "256 gated": (4090, 2044, 330, "silu", True, "pow2", "256", False, True),
    "256 other scales": (4090, 4088, 330, "relu", False, "mixed", "256", False, True),
    "256 gated other scales": (4090, 2044, 200, "silu", True, "any", "256", False, True),
    "128 alone": (1530, 1530, 1100, "gelu", False, "pow2", "128", False, True),
    "128 alone gated other scales": (1530, 765, 1100, "silu", True, "mixed", "128", False, True),
    "128": (2040, 4080, 300, "none", False, "any", "128", False, False),
    "128 whole groups of scales": (2040, 4080, 1000, "none", False, "mixed", "128", False, False),
    "128 gated": (2040, 2040, 1000, "gelu_tanh", True, "pow2", "128", False, False),
    "128 split": (700, 900, 9000, "silu", False, "pow2", "128", True, True),
    "128 split gated": (700, 450, 9000, "silu", True, "mixed", "128", True, True),
    "64 alone": (600, 1000, 600, "gelu", False, "mixed", "64", False, True),
    "64 alone gated": (600, 500, 600, "silu", True, "pow2", "64", False, True),
    "64": (1270, 1270, 600, "relu", False, "any", "64", False, False),
    "64 gated": (1270, 635, 200, "gelu", True, "mixed", "64", False, False),
    "64 split": (200, 300, 9000, "none", False, "mixed", "64", True, True),
}


def product_of(case):
    """rows, rows of w and contraction"""
    m, n, k, _, gated = case[:5]
    return m, (2 * n if gated else n), k
