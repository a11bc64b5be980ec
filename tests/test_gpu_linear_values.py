"""Activations and slopes of the products on the GPU at the far ends of their
arguments, against binary64.

Each slope is read through one product: w is the identity and x's rows are not
used, so dx is dp, rounded to the type once (its second rounding changes nothing,
the other terms of its sum are zeros).  A slope or value is off by its
exponential's 2^-17 = 128 units of 2^-24, at most 1.2 of it for a slope, and by ten
roundings: 170 units of its own magnitude, which is |dout| for a slope and |dout| (1
+ |p|) for a gated product's value."""
import numpy as np
import pytest
import torch

import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from test_gpu_norm import DEV, on

pytestmark = pytest.mark.gpu
UNITS = 170


def ends(dt):
    """both signs of magnitudes from the smallest normal to the largest finite value"""
    top = 127 if dt is torch.bfloat16 else 15
    v = torch.cat([torch.zeros(1, dtype=torch.float64), 1.375 * 2.0 ** torch.arange(-top + 1, top + 1, 1.0, dtype=torch.float64),
                   torch.linspace(0.25, 12, 48, dtype=torch.float64)])
    return torch.cat([v, -v]).to(dt)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_slopes_at_the_far_ends(dt, act, gated):
    dt = R.TYPES[dt]
    print(f"slopes act={act} gated={gated} {dt}", flush=True)
    p = ends(dt)
    n, m = len(p), 3
    rows = 2 * n if gated else n
    dout = torch.full((m, n), 0.75, dtype=dt)
    up = torch.full((n,), 0.5, dtype=dt)
    kept = (torch.cat([p, up]) if gated else p).expand(m, rows).contiguous()
    w = torch.eye(rows, dtype=dt)
    dx = torch.empty(m, rows, dtype=dt, device=DEV)
    ws = torch.empty(B.echo_linear_backward_workspace(m, n, rows, act=act, gated=gated), dtype=torch.uint8, device=DEV)
    B.echo_linear_backward(on(dout), torch.zeros(m, rows, dtype=dt, device=DEV), on(w), on(kept), dx, None, act=act,
                           gated=gated, workspace=ws)
    torch.cuda.synchronize()
    value, slope = R.act(p.double().numpy(), act)
    d = np.full(n, 0.75)
    exact, magnitude = d * slope, d.copy()
    if gated:
        exact = np.concatenate([0.5 * exact, d * value])
        magnitude = np.concatenate([0.5 * d, d * (1 + np.abs(p.double().numpy()))])
    assert np.isfinite(exact).all()
    for r in range(m):
        R.close(dx[r], exact, magnitude, UNITS, f"row {r}")


def test_halfs_range_of_dp_follows_the_scale_of_dout():
    """dp is rounded to half: past its largest value infinite, under its normals short of
    digits, both moved into the range by a power of two on dout"""
    n = 16
    up = torch.tensor([2.0 ** 14, 2.0 ** 13, 2.0 ** -10, 2.0 ** -11] * (n // 4), dtype=torch.float16)
    odd = 1.0 + 2.0 ** -10  # the smallest half above 1
    kept = torch.cat([torch.ones(n, dtype=torch.float16), up])[None].contiguous()
    w = torch.cat([torch.eye(n), torch.zeros(n, n)]).to(torch.float16)
    ws = torch.empty(B.echo_linear_backward_workspace(1, n, n, gated=True), dtype=torch.uint8, device=DEV)

    def dx(scale):
        dout, got = torch.full((1, n), odd * scale, dtype=torch.float16), torch.empty(1, n, dtype=torch.float16, device=DEV)
        B.echo_linear_backward(on(dout), torch.zeros(1, n, dtype=torch.float16, device=DEV), on(w), on(kept), got, None,
                               gated=True, workspace=ws)
        torch.cuda.synchronize()
        return got.cpu().double()[0]

    exact = odd * up.double()
    large, small = up.double() > 1, up.double() < 1
    assert not bool(torch.isfinite(dx(2.0 ** 3)).any())               # dp of 2^17: infinite, and NaN times w's zeros
    assert torch.equal(dx(2.0 ** -2)[large], exact[large] * 2.0 ** -2)
    assert torch.equal(dx(2.0 ** -12)[small], up.double()[small] * 2.0 ** -12)  # the last digit is lost
    assert torch.equal(dx(1.0)[small], exact[small])
