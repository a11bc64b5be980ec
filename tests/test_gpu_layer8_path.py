"""The 8-bit operators together with the norms and the all-reduce, as
examples/tp_layer.py --eight-bit runs them: one layer forward and backward against
binary64 on the codes and scales that the layer kept.

Bounds.  p, a and x are sums of products of exact values (but for what the matrix
cores cut, 2^-16 of the result) rounded once to bfloat16; a result on r such
roundings in a row differs by about sqrt(r) 2^-9 of its root mean square, and 2^-6 is
4 times that for r = 4 (test_gpu_layer_path.py).  z, p and a against their 8-bit
forms: a code's rounding is at most 2^-4 of the value, 2^-5 / sqrt 3 on the average of
an even spread, with values below a block's normal codes adding less; 2^-4 holds the
root mean square."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
NEAR, CODED = 2.0 ** -6, 2.0 ** -4


def off(got, want):
    got = got.double()
    return float((got - want).square().mean().sqrt() / want.square().mean().sqrt())


def value(kept, parts=1):
    """what codes and scales stand for, binary64 (blocks along the rows)"""
    codes, scales = kept
    cols = codes.shape[1] // parts
    out = []
    for c, s in zip(codes.double().split(cols, 1), scales.double().chunk(parts, 1)):
        out.append(c * s.repeat_interleave(128, 1)[:, :cols])
    return torch.cat(out, 1)


def weight(kept, parts=1):
    codes, scales = kept
    rows = codes.shape[0] // parts
    out = []
    for c, s in zip(codes.double().split(rows), scales.double().chunk(parts)):
        out.append(c * s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :codes.shape[1]])
    return torch.cat(out)


@pytest.mark.parametrize("tokens,hidden,inner,ranks", [(64, 512, 192, 4), (8, 1024, 128, 8), (1, 512, 64, 2),
                                                       (96, 256, 100, 3), (300, 640, 333, 2)])
def test_layers_forward_and_backward(tokens, hidden, inner, ranks):
    import tp_layer

    if tokens * hidden % (128 * ranks):
        pytest.skip("the all-reduce takes whole groups for each rank")
    print(f"tp_layer eight-bit tokens={tokens} hidden={hidden} inner={inner} ranks={ranks}", flush=True)
    blocks, out = tp_layer.run(tokens, hidden, inner, ranks, kind=tp_layer.Layer8)
    torch.cuda.synchronize()
    first, last = blocks
    h = first.h.double() + first.y.double()
    assert off(last.h, h) < NEAR
    rms = lambda h: h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    assert off(last.z, rms(h)) < NEAR
    z = value(last.z8)
    assert off(z, last.z.double()) < CODED
    total = 0
    for r in range(ranks):
        up, down = weight(last.up8[r], 2), weight(last.down8[r])
        assert off(up, last.up[r].double()) < CODED and off(down, last.down[r].double()) < CODED
        p = z @ up.T
        assert off(value(last.p8[r], 2), p) < CODED + NEAR
        a = torch.nn.functional.silu(p[:, :inner]) * p[:, inner:]
        assert off(value(last.a8[r]), a) < CODED + NEAR
        x = value(last.a8[r]) @ down.T
        assert off(last.x[r], x) < NEAR
        total = total + x
    assert off(last.y, total) < 0.25  # the 4-bit all-reduce

    # the second layer's gradients from its checkpoints, by the formulas
    grad = out["grad"].double()
    dz = 0
    for r in range(ranks):
        p, a = value(last.p8[r], 2), value(last.a8[r])
        gate, up = p[:, :inner], p[:, inner:]
        da = grad @ last.down[r].double()
        s = torch.sigmoid(gate)
        dp = torch.cat([da * up * (s + gate * s * (1 - s)), da * gate * s], 1)
        assert off(last.ddown[r], grad.T @ a) < NEAR and off(last.dup[r], dp.T @ z) < NEAR
        dz = dz + dp @ last.up[r].double()
    assert torch.isfinite(out["dh"].float()).all() and float(out["dh"].float().abs().max()) > 0
    hh = h.clone().requires_grad_(True)
    (rms(hh) * dz).sum().backward()
    reduce = tp_layer.AllReduce(out["grad"].numel(), last.ranks)
    dh, _ = last.backward(out["grad"], out["grad"], reduce)
    torch.cuda.synchronize()
    assert off(dh, grad + hh.grad) < 0.25


def test_checkpoints_hold_less_than_half_the_bytes():
    import tp_layer

    kept = tp_layer.Layer8.space_for(torch.empty(256, 1024, device="meta"))
    assert sum(t.untyped_storage().nbytes() for t in kept) < 0.52 * 256 * 1024 * 2


def test_a_captured_layer_gives_the_eager_results():
    import tp_layer

    layer = tp_layer.Layer8(64, 512, 192, 2, 5)
    reduce = tp_layer.AllReduce(64 * 512, 2)
    h = torch.randn(64, 512, device="cuda", dtype=torch.bfloat16)
    layer.forward(h, None, reduce)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(h, None, reduce)
    torch.cuda.current_stream().wait_stream(side)
    want = [layer.x[r].clone() for r in range(2)] + [layer.p8[1][1].clone(), layer.a8[0][0].float()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(h, None, reduce)
    for _ in range(3):
        for t in (*layer.x, layer.p, layer.a, layer.p8[1][1], layer.z):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [layer.x[0], layer.x[1], layer.p8[1][1], layer.a8[0][0].float()]
        assert all(torch.equal(g, w) for g, w in zip(got, want))
