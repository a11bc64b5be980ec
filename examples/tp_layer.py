"""A tensor-parallel MLP block with its all-reduce, one GPU playing every rank.

Each rank holds a slice of the block's weights.  Forward, per layer and rank:

    echo_norm      h <- h + y, z = rms(h): the residual add of the block before
                   and this block's norm in one pass
    echo_linear    a = silu(z Wg^T) * (z Wu^T): column-parallel, gated
    echo_linear    x = a Wd^T: row-parallel, this rank's part of the sum
    all-reduce     y = sum over ranks of x, carried in 4-bit codes: echo_encode on
                   every rank, echo_reduce_shard of each chunk, echo_decode, and
                   echo_update of the rank's averages off the critical path

Backward, per layer and rank: echo_linear_backward of both products, the
all-reduce of the gradient of z, and echo_norm_backward.

With --eight-bit the products read 8-bit floating point (echo_pack8, echo_linear8),
and each layer keeps z, p and a for its backward pass in 8 bits only
(echo_linear_backward8): 33 bytes for 64 of theirs, a byte an element and a scale for
each 128.  Their 16-bit forms are there once for all layers.

    python examples/tp_layer.py --tokens 1024 --hidden 4096 --inner 1792 --ranks 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from error_compensated_bit_echo_amd import binding as echo  # noqa: E402

DEV = "cuda:0"
BF16 = torch.bfloat16


def empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device=DEV)


class AllReduce:
    """The 4-bit all-reduce of one call sequence over `ranks` logical ranks."""

    def __init__(self, n, ranks):
        self.n, self.ranks, self.chunk = n, ranks, n // ranks
        self.avg = [(empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)) for _ in range(ranks)]
        self.states = [echo.echo_state_init(f, s, n, ranks, r) for r, (f, s) in enumerate(self.avg)]
        self.codes = [empty(n // 2, dtype=torch.uint8) for _ in range(ranks)]
        self.scales = [empty(n // 128, dtype=torch.float32) for _ in range(ranks)]
        self.codes2, self.scales2 = empty(n // 2, dtype=torch.uint8), empty(n // 128, dtype=torch.float32)
        self.e2 = [empty(self.chunk, dtype=torch.float32) for _ in range(ranks)]

    def __call__(self, parts, y):
        """y <- the sum of the ranks' parts as every rank receives it"""
        c, s = self.chunk // 2, self.chunk // 128
        for st, x, codes, scales in zip(self.states, parts, self.codes, self.scales):
            echo.echo_encode(st, x, codes, scales)
        for j in range(self.ranks):
            echo.echo_reduce_shard([q[j * c:(j + 1) * c] for q in self.codes], [q[j * s:(j + 1) * s] for q in self.scales],
                                   self.codes2[j * c:(j + 1) * c], self.scales2[j * s:(j + 1) * s], None, self.e2[j],
                                   chunk_n=self.chunk)
        echo.echo_decode(self.codes2, self.scales2, y, n=self.n)
        for r, st in enumerate(self.states):
            echo.echo_update(st, parts[r], self.codes[r], self.scales[r], self.e2[r])


class Layer:
    """One block's weights, dealt to the ranks, and what its backward pass needs."""

    def __init__(self, tokens, hidden, inner, ranks, seed, beside=None):
        """`beside`: another layer of the same sizes"""
        gen = torch.Generator(device=DEV).manual_seed(seed)
        draw = lambda *s: (torch.randn(*s, generator=gen, device=DEV) * s[-1] ** -0.5).to(BF16)  # noqa: E731
        self.up = [draw(2 * inner, hidden) for _ in range(ranks)]    # gate rows, then up rows
        self.down = [draw(hidden, inner) for _ in range(ranks)]
        self.norm = torch.ones(hidden, dtype=BF16, device=DEV)
        self.ranks, self.inner = ranks, inner
        self.h, self.y = empty(tokens, hidden), empty(tokens, hidden)
        self.stats = empty(4, tokens, dtype=torch.float32)
        self.kept(tokens, hidden, beside)
        self.x = [empty(tokens, hidden) for _ in range(ranks)]
        space = lambda *a, **k: empty(echo.echo_linear_workspace(*a, **k), dtype=torch.uint8)  # noqa: E731
        self.ws_up = space(tokens, inner, hidden, act="silu", gated=True)
        self.ws_down = space(tokens, hidden, inner)

    def kept(self, tokens, hidden, beside):
        """what the forward pass keeps of z, p and a"""
        self.z = empty(tokens, hidden)
        self.p = [empty(tokens, 2 * self.inner) for _ in range(self.ranks)]
        self.a = [empty(tokens, self.inner) for _ in range(self.ranks)]

    def forward(self, h, y, reduce):
        """h, the stream, and y, the block before's output (None for the first)"""
        if y is None:
            self.h.copy_(h)
            echo.echo_norm(h, None, None, self.z, pre="rms", w_pre=self.norm, stats=self.stats)
        else:
            echo.echo_norm(h, y, self.h, self.z, pre="rms", w_pre=self.norm, stats=self.stats)
        for r in range(self.ranks):
            echo.echo_linear(self.z, self.up[r], self.a[r], act="silu", gated=True, p=self.p[r], workspace=self.ws_up)
            echo.echo_linear(self.a[r], self.down[r], self.x[r], workspace=self.ws_down)
        reduce(self.x, self.y)
        return self.h, self.y

    def backward(self, dh, dy, reduce):
        """Gradients of the stream and of the block before's output, for dh
        (gradient of the stream behind the norm) and dy (of this block's
        output); each rank's weight gradients stay in self.dup, self.ddown."""
        tokens, hidden = dy.shape
        self.dup, self.ddown = [torch.empty_like(w) for w in self.up], [torch.empty_like(w) for w in self.down]
        self.dnorm = torch.empty_like(self.norm)
        dz = [torch.empty_like(dy) for _ in range(self.ranks)]
        da = empty(tokens, self.inner)
        need = max(self.products_workspace(tokens, hidden), echo.echo_norm_backward_workspace(tokens, hidden))
        ws = empty(need, dtype=torch.uint8)
        self.products_backward(dy, da, dz, ws)
        total = torch.empty_like(dy)
        reduce(dz, total)
        out_h, out_y = torch.empty_like(dh), torch.empty_like(dy)
        echo.echo_norm_backward(total, dh, self.h, None, self.stats, out_h, out_y, pre="rms", w_pre=self.norm,
                                dw_pre=self.dnorm, workspace=ws)
        return out_h, out_y

    def products_backward(self, dy, da, dz, ws):
        """every rank's dz and weight gradients; da is one rank's at a time"""
        for r in range(self.ranks):
            echo.echo_linear_backward(dy, self.a[r], self.down[r], None, da, self.ddown[r], workspace=ws)
            echo.echo_linear_backward(da, self.z, self.up[r], self.p[r], dz[r], self.dup[r], act="silu", gated=True,
                                      workspace=ws)

    def products_workspace(self, tokens, hidden):
        return max(echo.echo_linear_backward_workspace(tokens, hidden, self.inner),
                   echo.echo_linear_backward_workspace(tokens, self.inner, hidden, act="silu", gated=True))


class Layer8(Layer):
    """The same block with its products in 8-bit floating point, and 8-bit checkpoints."""

    def __init__(self, tokens, hidden, inner, ranks, seed, beside=None):
        super().__init__(tokens, hidden, inner, ranks, seed, beside)
        self.up8 = [self.pack(w, blocks=True, parts=2) for w in self.up]
        self.down8 = [self.pack(w, blocks=True) for w in self.down]
        self.ws_up = empty(echo.echo_linear8_workspace(tokens, inner, hidden, act="silu", gated=True), dtype=torch.uint8)
        self.ws_down = empty(echo.echo_linear8_workspace(tokens, hidden, inner), dtype=torch.uint8)

    def kept(self, tokens, hidden, beside):
        # z, and p and a of one rank at a time, are packed as soon as they are there
        self.z, self.p, self.a = (beside.z, beside.p, beside.a) if beside else (
            empty(tokens, hidden), empty(tokens, 2 * self.inner), empty(tokens, self.inner))
        self.z8 = self.space_for(self.z)
        self.p8 = [self.space_for(self.p, parts=2) for _ in range(self.ranks)]
        self.a8 = [self.space_for(self.a) for _ in range(self.ranks)]

    @staticmethod
    def space_for(x, **how):
        """codes and scales of a tensor like x"""
        return echo.codes8_empty(*x.shape), empty(*echo.scales8_shape(*x.shape, **how), dtype=torch.float32)

    def pack(self, x, **how):
        kept = self.space_for(x, **how)
        echo.echo_pack8(x, *kept, **how)
        return kept

    def forward(self, h, y, reduce):
        if y is None:
            self.h.copy_(h)
            echo.echo_norm(h, None, None, self.z, pre="rms", w_pre=self.norm, stats=self.stats)
        else:
            echo.echo_norm(h, y, self.h, self.z, pre="rms", w_pre=self.norm, stats=self.stats)
        echo.echo_pack8(self.z, *self.z8)
        for r in range(self.ranks):
            echo.echo_linear8(*self.z8, *self.up8[r], self.a, act="silu", gated=True, p=self.p, workspace=self.ws_up)
            echo.echo_pack8(self.p, *self.p8[r], parts=2)
            echo.echo_pack8(self.a, *self.a8[r])
            echo.echo_linear8(*self.a8[r], *self.down8[r], self.x[r], workspace=self.ws_down)
        reduce(self.x, self.y)
        return self.h, self.y

    def products_backward(self, dy, da, dz, ws):
        for r in range(self.ranks):
            echo.echo_linear_backward8(dy, *self.a8[r], self.down[r], None, None, da, self.ddown[r], workspace=ws)
            echo.echo_linear_backward8(da, *self.z8, self.up[r], *self.p8[r], dz[r], self.dup[r], act="silu", gated=True,
                                       workspace=ws)

    def products_workspace(self, tokens, hidden):
        return max(echo.echo_linear_backward8_workspace(tokens, hidden, self.inner),
                   echo.echo_linear_backward8_workspace(tokens, self.inner, hidden, act="silu", gated=True))


def run(tokens, hidden, inner, ranks, layers=2, steps=1, seed=0, kind=Layer):
    """`steps` forward and backward passes of a few layers; returns the layers
    and the last step's tensors"""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    h0 = torch.randn(tokens, hidden, generator=gen, device=DEV).to(BF16)
    grad = (1e-3 * torch.randn(tokens, hidden, generator=gen, device=DEV)).to(BF16)
    blocks = []
    for k in range(layers):
        blocks.append(kind(tokens, hidden, inner, ranks, seed + 1 + k, beside=blocks[0] if blocks else None))
    # one call sequence each way: the averages are carried from layer to layer
    there, back = AllReduce(tokens * hidden, ranks), AllReduce(tokens * hidden, ranks)
    for _ in range(steps):
        h, y = h0, None
        for block in blocks:
            h, y = block.forward(h, y, there)
        # the loss is linear in the stream behind the last block, h + y
        dh, dy = grad, grad
        for block in reversed(blocks):
            dh, dy = block.backward(dh, dy, back)
    return blocks, {"h0": h0, "grad": grad, "h": h, "y": y, "dh": dh}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=1792, help="columns of the inner product on one rank")
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--eight-bit", action="store_true", help="products and checkpoints in 8-bit floating point")
    args = ap.parse_args()
    kind = Layer8 if args.eight_bit else Layer
    run(args.tokens, args.hidden, args.inner, args.ranks, args.layers, kind=kind)
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    _, out = run(args.tokens, args.hidden, args.inner, args.ranks, args.layers, kind=kind)
    end.record()
    torch.cuda.synchronize()
    print(f"{args.layers} layers, {args.tokens} tokens x {args.hidden}, {args.ranks} ranks of {args.inner} on one GPU: "
          f"{begin.elapsed_time(end):.2f} ms forward and backward, set-up among it; "
          f"|y| {float(out['y'].float().norm()):.4f}, |dh| {float(out['dh'].float().norm()):.6f}")


if __name__ == "__main__":
    main()
