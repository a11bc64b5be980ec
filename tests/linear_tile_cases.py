"""Shapes whose products take the large tiles, with edges cut in both directions and
contractions that end inside a step.

name: m, n, k, activation, gated, the product meant, its tile, and whether its
contraction is split."""
TILES = {"256": 0, "256x128": 1, "128": 2, "64": 3}
CASES = {
    "out 256": (4090, 4088, 200, "none", False, "out", "256", False),
    "out 256 gated": (4090, 2044, 200, "silu", True, "out", "256", False),
    "out 256 copied rows": (4090, 4087, 203, "gelu", False, "out", "256", False),
    "out 256 split": (1530, 3064, 8200, "gelu_tanh", False, "out", "256", True),
    "out 256 split gated": (1530, 1532, 8200, "silu", True, "out", "256", True),
    "out 256x128": (1530, 3064, 4104, "relu", False, "out", "256x128", False),
    "out 256x128 gated": (1530, 1532, 4104, "gelu", True, "out", "256x128", False),
    "out 256x128 split": (2550, 1528, 8200, "none", False, "out", "256x128", True),
    "dx 256": (4090, 200, 4088, "none", False, "dx", "256", False),
    "dx 256 filled rows": (4090, 203, 4088, "gelu", False, "dx", "256", False),
    "dx 256 gated": (4090, 100, 4088, "silu", True, "dx", "256", False),
    "dx 256 split": (1530, 8200, 3064, "none", False, "dx", "256", True),
    "dx 256x128": (1530, 4104, 3064, "silu", False, "dx", "256x128", False),
    "dx 256x128 split gated": (2550, 4100, 1528, "gelu_tanh", True, "dx", "256x128", True),
    "dw 256": (203, 4088, 4088, "none", False, "dw", "256", False),
    "dw 256 cut": (203, 4090, 4086, "gelu", False, "dw", "256", False),
    "dw 256 gated": (203, 2044, 4088, "silu", True, "dw", "256", False),
    "dw 256 split": (8203, 1530, 3064, "relu", False, "dw", "256", True),
    "dw 256x128": (4101, 1530, 3064, "silu", False, "dw", "256x128", False),
    "dw 256x128 split": (8203, 2550, 1528, "gelu", False, "dw", "256x128", True),
}


def product_of(case):
    """rows, columns and contraction of the product meant"""
    m, n, k, _, gated, product, _, _ = case
    rows = 2 * n if gated else n
    return {"out": (m, rows, k), "dx": (m, k, rows), "dw": (rows, k, m)}[product]
