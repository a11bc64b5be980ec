"""Products of more tiles than one dimension of a grid holds.

Rows repeat with a period, so every output row is held to the binary64 result of its
place in the period; the first rows by the bounds of test_gpu_linear, the others by
equality with them (a row's sum has one order, whatever its tile)."""
import pytest
import torch

import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from test_gpu_linear import case, on, space
from test_gpu_norm import DEV

pytestmark = pytest.mark.gpu
PERIOD = 1 << 16


def periodic(t, m):
    """t's rows over and over, m of them"""
    out = torch.empty(m, t.shape[1], dtype=t.dtype, device=DEV)
    whole = m // PERIOD * PERIOD
    out[:whole].view(-1, PERIOD, t.shape[1]).copy_(on(t)[None])
    out[whole:].copy_(on(t)[:m - whole])
    return out


def same_everywhere(got, what):
    first = got[:PERIOD].clone()
    for at in range(0, got.shape[0], PERIOD * 512):
        part = got[at:at + PERIOD * 512]
        whole = part.shape[0] // PERIOD * PERIOD
        assert bool((part[:whole].view(-1, PERIOD, part.shape[1]) == first).all()), (what, at)
        assert torch.equal(part[whole:], first[:part.shape[0] - whole]), (what, at)
    return first


@pytest.mark.parametrize("k", [8, 7])
def test_half_a_billion_rows(k):
    m, n = (1 << 29) + 1129, 8
    print(f"linear m={m} n={n} k={k}", flush=True)
    c = case(PERIOD, n, k, torch.bfloat16, False, residual=False, seed=21)
    x = periodic(c["x"], m)
    out, p = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV), torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    B.echo_linear(x, on(c["w"]), out, bias=on(c["bias"]), act="relu", p=p,
                  workspace=space(B.echo_linear_workspace(m, n, k, act="relu")))
    torch.cuda.synchronize()
    want = R.linear_forward(c["x"], c["w"], c["bias"], None, "relu", False)
    R.close(same_everywhere(out, "out"), *want["out"], 2 * (k + 64), "out")
    kept = same_everywhere(p, "p")
    R.close(kept, *want["p"], k + 64, "p")
    print("backward", flush=True)
    dout = out.copy_(periodic(c["dout"], m))
    dx = torch.full((m, k), 7.0, dtype=torch.bfloat16, device=DEV)
    B.echo_linear_backward(dout, x, on(c["w"]), p, dx, None, act="relu",
                           workspace=space(B.echo_linear_backward_workspace(m, n, k, act="relu")))
    torch.cuda.synchronize()
    e = R.linear_backward(c["dout"], c["x"], c["w"], kept, "relu", False)["dx"]
    R.close(same_everywhere(dx, "dx"), e[0], e[1], n + 64, "dx")
