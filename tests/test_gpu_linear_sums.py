"""Long sums of the products on the GPU by the norm of every row and column
(layer_sums): the bounds of every element grow with a sum's length, and at these
lengths let whole rows go missing."""
import pytest

import layer_reference as R
from test_gpu_linear_tiles import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1025, 2056, 136), (2050, 1032, 72), (4100, 520, 80), (6000, 136, 4104),
                                   (513, 100, 9000), (2600, 1003, 40), (1300, 50, 41), (900, 90, 1001),
                                   (20000, 24, 40), (33000, 17, 19)])
def test_long_sums_lose_no_row(m, n, k, dt):
    """sums over many rows in the smaller tiles, their splits and the bias's runs"""
    for act, gated in (("none", False), ("gelu_tanh", False), ("silu", True)):
        print(f"sums m={m} n={n} k={k} {dt} {act} gated={gated}", flush=True)
        run(m, n, k, R.TYPES[dt], act, gated, True, True, seed=1)
