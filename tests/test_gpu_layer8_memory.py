"""What examples/tp_layer.py --eight-bit holds for the backward pass: z, p and a in 8 bits, 33
bytes for 64 of theirs (a byte an element and four for each 128), and their 16-bit forms
once for all layers."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
TOKENS, HIDDEN, INNER, RANKS = 96, 512, 384, 2


def tensors(v):
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (list, tuple)):
        for q in v:
            yield from tensors(q)


def held(layer):
    return [t for v in vars(layer).values() for t in tensors(v)]


def test_checkpoints_take_33_bytes_for_64():
    import tp_layer

    (layer, _), _ = tp_layer.run(TOKENS, HIDDEN, INNER, RANKS, kind=tp_layer.Layer8)
    kept = [*layer.z8, *(t for q in layer.p8 + layer.a8 for t in q)]
    size = sum(t.untyped_storage().nbytes() for t in kept)
    assert size * 64 == 33 * 2 * TOKENS * (HIDDEN + RANKS * 3 * INNER)


def test_16_bit_forms_are_held_once():
    import tp_layer

    blocks, _ = tp_layer.run(TOKENS, HIDDEN, INNER, RANKS, layers=3, kind=tp_layer.Layer8)
    wide = [t for b in blocks for t in held(b) if t.dtype is torch.bfloat16 and tuple(t.shape) in
            ((TOKENS, INNER), (TOKENS, 2 * INNER))]
    assert len({t.data_ptr() for t in wide}) == 2  # p and a of one rank
    assert len({b.z.data_ptr() for b in blocks}) == 1


def test_gradients_do_not_meet_the_shared_forms():
    """a layer's gradients after another layer's forward pass has overwritten z, p and a"""
    import tp_layer

    def gradients(spoil):
        layer = tp_layer.Layer8(TOKENS, HIDDEN, INNER, RANKS, 3)
        gen = torch.Generator(device="cuda").manual_seed(1)
        h, y, grad = (torch.randn(TOKENS, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
        there, back = (tp_layer.AllReduce(TOKENS * HIDDEN, RANKS) for _ in range(2))
        layer.forward(h, y, there)
        if spoil:
            for t in (layer.z, layer.p, layer.a):
                t.fill_(float("nan"))
        dh, dy = layer.backward(grad, grad, back)
        torch.cuda.synchronize()
        return [dh, dy, *layer.dup, *layer.ddown]

    for a, b in zip(gradients(False), gradients(True)):
        assert torch.equal(a, b)
