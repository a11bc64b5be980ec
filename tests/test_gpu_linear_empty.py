"""Gated products without rows: the gradient of the sums, twice as wide as dout, has no
bytes, dout has no address, and the weights' gradients are zeros."""
import pytest
import torch

from error_compensated_bit_echo_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,k", [(8, 8), (64, 128), (33, 40), (256, 72)])
def test_gated_backward_without_rows(n, k):
    e = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dx, dw, db = e(0, k), e(2 * n, k), e(2 * n)
    print(f"echo_linear_backward m=0 n={n} k={k} gated", flush=True)
    ws = torch.empty(B.echo_linear_backward_workspace(0, n, k, act="silu", gated=True), dtype=torch.uint8, device=DEV)
    B.echo_linear_backward(e(0, n), e(0, k), e(2 * n, k), e(0, 2 * n), dx, dw, dbias=db, act="silu", gated=True, workspace=ws)
    torch.cuda.synchronize()
    assert float(dw.float().abs().sum()) == 0 and float(db.float().abs().sum()) == 0
