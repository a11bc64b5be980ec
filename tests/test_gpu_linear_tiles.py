"""The large tiles of echo_linear and echo_linear_backward on the GPU against
binary64: forward, dx and dw, plain and gated, both types, with and without splits,
tiles cut by the last row and the last column, contractions that end inside a step,
operands whose rows are followed by NaN.  tests/test_linear_plan.py holds the shapes to
their tiles.

Forward, every element by the bounds of test_gpu_linear; all outputs by the norm of
every row and column (layer_sums), which a lost row or step would break."""
import pytest
import torch

import layer_reference as R
import layer_sums as S
from error_compensated_bit_echo_amd import binding as B
from linear_tile_cases import CASES
from test_gpu_linear import space
from test_gpu_norm import DEV, guarded, untouched

pytestmark = pytest.mark.gpu


def followed_by_nan(t):
    """t in rows of an aligned pitch with NaN behind them"""
    rows, cols = t.shape
    buf = torch.full((rows, (cols + 15) // 8 * 8), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, :cols] = t
    return buf[:, :cols]


def run(m, n, k, dt, act, gated, forward, backward, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    rand = lambda *s, spread=1.0: (spread * torch.randn(*s, generator=gen, device=DEV)).to(dt)  # noqa: E731
    rows = 2 * n if gated else n
    plain = act == "none" and not gated
    x, w = followed_by_nan(rand(m, k)), followed_by_nan(rand(rows, k, spread=k ** -0.5))
    if k % 8:  # rows that no direct load takes: the call copies them
        x, w = (x, w) if not forward else (x.contiguous(), w.contiguous())
    if forward:
        bias, residual = rand(rows, spread=0.3), rand(m, n)
        ob, out = guarded(m, n, dt, n + 8)
        pb, p = guarded(m, rows, dt)
        B.echo_linear(x, w, out, bias=bias, residual=residual, act=act, gated=gated, p=p,
                      workspace=space(B.echo_linear_workspace(m, n, k, act=act, gated=gated)))
        torch.cuda.synchronize()
        want = S.forward(x, w, bias, residual, act, gated)
        for name, t, roundings in (("out", out, 2 * (k + 64)), ("p", p, k + 64)):
            S.elements(t, *want[name], roundings, name)
            S.near(t, want[name][0], 1, name)
        untouched(ob, out, "out")
        untouched(pb, p, "p")
    if backward:
        dout, p = followed_by_nan(rand(m, n)), None if plain else rand(m, rows)
        outs = {"dx": guarded(m, k, dt), "dw": guarded(rows, k, dt), "dbias": guarded(1, rows, dt)}
        B.echo_linear_backward(dout, x, w, p, outs["dx"][1], outs["dw"][1], dbias=outs["dbias"][1][0], act=act,
                               gated=gated, workspace=space(B.echo_linear_backward_workspace(m, n, k, act=act, gated=gated)))
        torch.cuda.synchronize()
        want = S.backward(dout, x, w, p, act, gated)
        for name, (buf, t) in outs.items():
            S.near(t, want[name], 1 if plain or name == "dbias" else 2, name)
            untouched(buf, t, name)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("name", list(CASES))
def test_large_tiles(name, dt):
    m, n, k, act, gated, product, tile, split = CASES[name]
    print(f"tile {name}: m={m} n={n} k={k} {dt} {act} gated={gated}", flush=True)
    run(m, n, k, R.TYPES[dt], act, gated, product == "out", product != "out")
