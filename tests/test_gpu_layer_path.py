"""The layer operators and the all-reduce together, as examples/tp_layer.py runs
them: one layer's forward and backward against a binary64 run that takes the
all-reduce's own results as given (its parity with the oracle has its own
tests), so only the operators' roundings lie between.

Bounds.  Every tensor passed on is rounded once to bfloat16 (half a unit is
2^-8 of the value, 2^-9 on the average): z, p, a and x forward, da, dp and dz
backward, so a result that stands on r such roundings in a row differs by about
sqrt(r) 2^-9 of its root mean square; 2^-6 is 4 times that for r = 4.  The
all-reduce itself rounds to sevenths of a group's largest of 128 values, which for
normal ones is about 2.8 of their deviation: 0.4 / sqrt(12) = 0.12 of it in
every part and once more in the sum, together 0.16 of the sum's; 0.25 holds it."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -6


def off(got, want):
    got = got.double()
    return float((got - want).square().mean().sqrt() / want.square().mean().sqrt())


@pytest.mark.parametrize("tokens,hidden,inner,ranks", [(64, 512, 192, 4), (8, 1024, 128, 8), (1, 512, 64, 2),
                                                       (96, 256, 100, 3)])
def test_layers_forward_and_backward(tokens, hidden, inner, ranks):
    import tp_layer

    print(f"tp_layer tokens={tokens} hidden={hidden} inner={inner} ranks={ranks}", flush=True)
    blocks, out = tp_layer.run(tokens, hidden, inner, ranks)
    torch.cuda.synchronize()
    first, last = blocks
    d = lambda t: t.double()  # noqa: E731
    rms = lambda h: h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731

    # forward of the second layer, from the first layer's reduced output
    h = d(first.h) + d(first.y)
    assert off(last.h, h) < NEAR
    assert off(last.z, rms(h)) < NEAR
    total = 0
    for r in range(ranks):
        p = d(last.z) @ d(last.up[r]).T
        a = torch.nn.functional.silu(p[:, :inner]) * p[:, inner:]
        assert off(last.p[r], p) < NEAR and off(last.a[r], a) < NEAR
        x = a @ d(last.down[r]).T
        assert off(last.x[r], x) < NEAR
        total = total + x
    # the 4-bit all-reduce: codes of +-7 around groups of 128, two roundings
    assert off(last.y, total) < 0.25

    # backward of the second layer by automatic differentiation
    z = d(last.z).requires_grad_(True)
    up = [d(w).requires_grad_(True) for w in last.up]
    down = [d(w).requires_grad_(True) for w in last.down]
    y = 0
    for r in range(ranks):
        p = z @ up[r].T
        y = y + (torch.nn.functional.silu(p[:, :inner]) * p[:, inner:]) @ down[r].T
    y.backward(d(out["grad"]))
    for r in range(ranks):
        assert off(last.dup[r], up[r].grad) < NEAR and off(last.ddown[r], down[r].grad) < NEAR
    assert torch.isfinite(out["dh"].float()).all() and float(out["dh"].float().abs().max()) > 0
    # the gradient that reaches the stream, with the quantized gradient of z between
    hh = h.clone().requires_grad_(True)
    (rms(hh) * z.grad).sum().backward()
    want = d(out["grad"]) + hh.grad
    assert off(first_dh(last, out), want) < 0.25


def first_dh(last, out):
    """the second layer's gradient of its stream, run again from what it kept"""
    import tp_layer

    reduce = tp_layer.AllReduce(out["grad"].numel(), last.ranks)
    dh, _ = last.backward(out["grad"], out["grad"], reduce)
    torch.cuda.synchronize()
    return dh
