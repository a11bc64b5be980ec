"""echo_linear and echo_linear_backward on the GPU against binary64: both types,
every activation and gate, sizes around the tiles and steps of the kernels, odd
sizes, pitches and addresses, single rows, empty sides, NaN, streams and graphs.

Bounds.  A sum over c adds its products in some fixed order, so at most c
binary32 roundings of terms of magnitude |x| |w|; the matrix cores add a few at a
time and a random walk stays far below, but the bound used is the proved one,
c + 64 (64 for bias, activation and residual: exponentials are good to 2^-17 =
128 units of 2^-24 where they are that large, and such terms are small beside the
sum's magnitude, or their own share is added by the reference).  The backward
products read dp rounded to the type: half a unit of each term more."""
import numpy as np
import pytest
import torch

import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from test_gpu_norm import DEV, guarded, on, rand, untouched

pytestmark = pytest.mark.gpu


def case(m, n, k, dt, gated=False, bias=True, residual=True, seed=0):
    gen = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    rows = 2 * n if gated else n
    return {"x": rand(gen, m, k, dt=dt), "w": rand(gen, rows, k, dt=dt, spread=max(k, 1) ** -0.5),
            "bias": rand(gen, rows, dt=dt, spread=0.3) if bias else None,
            "residual": rand(gen, m, n, dt=dt) if residual else None, "dout": rand(gen, m, n, dt=dt)}


def space(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def forward(c, act, gated, keep=True, shift=0, pads=(0, 0, 0)):
    m, k = c["x"].shape
    rows = c["w"].shape[0]
    n = rows // 2 if gated else rows
    dt = c["x"].dtype
    _, x = guarded(m, k, dt, k + pads[0], shift)
    _, w = guarded(rows, k, dt, k + pads[1], shift)
    ob, out = guarded(m, n, dt, n + pads[2], shift)
    pb, p = guarded(m, rows, dt)
    x.copy_(c["x"])
    w.copy_(c["w"])
    B.echo_linear(x, w, out, bias=on(c["bias"]), residual=on(c["residual"]), act=act, gated=gated,
                  p=p if keep else None, workspace=space(B.echo_linear_workspace(m, n, k, act=act, gated=gated)))
    torch.cuda.synchronize()
    want = R.linear_forward(c["x"], c["w"], c["bias"], c["residual"], act, gated)
    R.close(out, *want["out"], 2 * (k + 64), "out")
    untouched(ob, out, "out")
    if keep:
        R.close(p, *want["p"], k + 64, "p")
        untouched(pb, p, "p")
    return out, p


def backward(c, act, gated, p, want=("dx", "dw", "dbias"), shift=0, pads=(0, 0, 0)):
    m, k = c["x"].shape
    rows = c["w"].shape[0]
    n = rows // 2 if gated else rows
    dt = c["x"].dtype
    plain = act == "none" and not gated
    _, x = guarded(m, k, dt, k + pads[0], shift)
    _, w = guarded(rows, k, dt, k + pads[1], shift)
    _, dout = guarded(m, n, dt, n + pads[2], shift)
    x.copy_(c["x"])
    w.copy_(c["w"])
    dout.copy_(c["dout"])
    outs = {"dx": guarded(m, k, dt), "dw": guarded(rows, k, dt), "dbias": guarded(1, rows, dt)}
    give = {q: (v[0] if q == "dbias" else v) if q in want else None for q, (_, v) in outs.items()}
    B.echo_linear_backward(dout, x, w, None if plain else p, give["dx"], give["dw"], dbias=give["dbias"], act=act,
                           gated=gated, workspace=space(B.echo_linear_backward_workspace(m, n, k, act=act, gated=gated)))
    torch.cuda.synchronize()
    exact = R.linear_backward(c["dout"], c["x"], c["w"], p, act, gated)
    length = {"dx": rows, "dw": m, "dbias": m}
    for q in want:
        v = outs[q][1]
        e, magnitude = exact[q][0].reshape(v.shape), exact[q][1].reshape(v.shape)
        if q != "dbias" and not plain:  # dp's rounding, in units of 2^-24
            magnitude = magnitude + exact[q][2] * (R.HALF_ULP[dt] / R.EPS32 / (length[q] + 64))
            if dt == torch.float16:     # dp below the type's normals
                other = c["w"] if q == "dx" else c["x"]
                magnitude = magnitude + R.TINY[dt] / R.EPS32 * other.double().abs().sum(0).numpy()[None, :] / (length[q] + 64)
        R.close(v, e, magnitude, length[q] + 64, q)
    for q, (buf, v) in outs.items():
        untouched(buf, v if q in want else v[:0], q)
    return {q: outs[q][1] for q in want}


SIZES = [(1, 1, 1), (1, 8, 64), (1, 300, 1000), (3, 5, 7), (16, 64, 32), (17, 33, 63), (31, 100, 72), (33, 65, 129),
         (64, 64, 64), (65, 130, 200), (100, 257, 96), (128, 128, 128), (129, 127, 130), (200, 96, 256),
         (255, 384, 65), (257, 260, 191), (2, 1030, 520), (300, 20, 777)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_sizes(m, n, k, dt, gated):
    print(f"linear m={m} n={n} k={k} {dt} gated={gated}", flush=True)
    act = "silu" if gated else "none"
    c = case(m, n, k, R.TYPES[dt], gated)
    _, p = forward(c, act, gated)
    backward(c, act, gated, p)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activations(act, gated):
    for dt in ("bf16", "f16"):
        print(f"linear act={act} gated={gated} {dt}", flush=True)
        c = case(70, 90, 80, R.TYPES[dt], gated, seed=1)
        c["w"] = (c["w"].float() * 3).to(R.TYPES[dt])  # sums out to the flat ends
        _, p = forward(c, act, gated)
        backward(c, act, gated, p)


@pytest.mark.parametrize("m,n,k", [(2600, 1003, 40), (1300, 5, 41), (900, 9, 1001), (700, 78, 5)])
def test_many_odd_rows(m, n, k):
    """rows that end inside a vector, and rows under one, in runs of several rows
    and in whole steps along the contraction"""
    for gated, act in ((False, "none"), (False, "gelu"), (True, "silu")):
        print(f"linear m={m} n={n} k={k} {act} gated={gated}", flush=True)
        c = case(m, n, k, torch.float16, gated, seed=13)
        _, p = forward(c, act, gated)
        backward(c, act, gated, p)


@pytest.mark.parametrize("m,n,k", [(1025, 2056, 136), (2050, 1032, 72), (4100, 520, 80), (70, 8200, 64),
                                   (6000, 136, 4104), (513, 100, 9000)])
def test_many_tiles(m, n, k):
    print(f"linear m={m} n={n} k={k}", flush=True)
    for gated, act in ((False, "gelu_tanh"), (True, "silu")):
        c = case(m, n, k, torch.bfloat16, gated, seed=2)
        _, p = forward(c, act, gated)
        backward(c, act, gated, p)
    c = case(m, n, k, torch.bfloat16, False, bias=False, residual=False, seed=3)
    forward(c, "none", False, keep=False)
    backward(c, "none", False, None)


@pytest.mark.parametrize("shift,pads", [(0, (8, 16, 8)), (1, (0, 0, 0)), (0, (3, 0, 1)), (3, (5, 2, 7))])
def test_pitches_and_odd_addresses(shift, pads):
    for m, n, k, gated in ((70, 72, 136, False), (5, 40, 264, True), (200, 131, 77, False), (300, 64, 128, True)):
        print(f"linear m={m} n={n} k={k} shift={shift} pads={pads}", flush=True)
        c = case(m, n, k, torch.bfloat16, gated, seed=4)
        act = "silu" if gated else "gelu"
        _, p = forward(c, act, gated, shift=shift, pads=pads)
        backward(c, act, gated, p, shift=shift, pads=pads)
        backward(c, "none", False, None, shift=shift, pads=pads) if not gated else None


def test_gradients_asked_for_alone():
    c = case(90, 56, 120, torch.bfloat16, False, seed=5)
    _, p = forward(c, "silu", False)
    both = backward(c, "silu", False, p)
    for q in ("dx", "dw", "dbias"):
        alone = backward(c, "silu", False, p, want=(q,))
        assert torch.equal(alone[q], both[q]), q
    backward(c, "none", False, None, want=("dbias",))


def test_residual_in_place():
    c = case(130, 72, 96, torch.bfloat16, False, seed=6)
    out, _ = forward(c, "gelu", False)
    r = on(c["residual"])
    B.echo_linear(on(c["x"]), on(c["w"]), r, bias=on(c["bias"]), residual=r, act="gelu",
                  workspace=space(B.echo_linear_workspace(130, 72, 96, act="gelu")))
    torch.cuda.synchronize()
    assert torch.equal(r, out)


@pytest.mark.parametrize("m,n,k", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0)])
def test_empty_sides(m, n, k):
    """no rows, no outputs, no inputs: sums over nothing are zeros"""
    c = case(m, n, k, torch.bfloat16, False, seed=7)
    e = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    out, p = e(m, n), e(m, n)
    B.echo_linear(on(c["x"]), on(c["w"]), out, bias=on(c["bias"]), residual=on(c["residual"]), act="silu", p=p,
                  workspace=space(B.echo_linear_workspace(m, n, k, act="silu")))
    want = R.linear_forward(c["x"], c["w"], c["bias"], c["residual"], "silu", False)
    R.close(out, *want["out"], 64, "out")
    dx, dw, db = e(m, k), e(n, k), e(n)
    B.echo_linear_backward(on(c["dout"]), on(c["x"]), on(c["w"]), p, dx, dw, dbias=db, act="silu",
                           workspace=space(B.echo_linear_backward_workspace(m, n, k, act="silu")))
    torch.cuda.synchronize()
    if n == 0 or m == 0:
        for t in (dx, dw, db):
            assert not t.numel() or float(t.abs().max()) == 0


def test_nan_stays_in_its_row_and_column():
    m, n, k = 140, 150, 200
    for gated in (False, True):
        c = case(m, n, k, torch.bfloat16, gated, residual=False, seed=8)
        act = "silu" if gated else "gelu"
        out, p = forward(c, act, gated)
        x, w = c["x"].clone(), c["w"].clone()
        x[17, 3], w[21, 5] = float("nan"), float("nan")
        got = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
        B.echo_linear(on(x), on(w), got, bias=on(c["bias"]), act=act, gated=gated,
                      workspace=space(B.echo_linear_workspace(m, n, k, act=act, gated=gated)))
        torch.cuda.synchronize()
        rows, cols = [i for i in range(m) if i != 17], [j for j in range(n) if j != 21]
        assert bool(torch.isnan(got[17]).all()) and bool(torch.isnan(got[:, 21]).all())
        assert torch.equal(got[rows][:, cols], out[rows][:, cols])


def test_padding_may_hold_nan():
    """what lies between the rows of a pitched operand never reaches a sum"""
    for m, n, k in ((40, 70, 100), (40, 70, 104), (3, 70, 104), (200, 200, 136)):
        c = case(m, n, k, torch.bfloat16, False, bias=False, residual=False, seed=9)
        dirty = {}
        for q, (r, cols) in {"x": (m, k), "w": (n, k), "dout": (m, n)}.items():
            buf = torch.full((r, cols + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
            buf[:, :cols] = on(c[q])
            dirty[q] = buf[:, :cols]
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        outs = []
        for t in (dirty, {q: on(c[q]) for q in dirty}):
            out, dx, dw = e(m, n), e(m, k), e(n, k)
            B.echo_linear(t["x"], t["w"], out, workspace=space(B.echo_linear_workspace(m, n, k)))
            B.echo_linear_backward(t["dout"], t["x"], t["w"], None, dx, dw,
                                   workspace=space(B.echo_linear_backward_workspace(m, n, k)))
            outs.append((out, dx, dw))
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert bool(torch.isfinite(a.float()).all()) and torch.equal(a, b)


def test_same_bits_on_every_call_and_on_another_stream():
    c = case(700, 264, 520, torch.bfloat16, True, seed=10)
    out, p = forward(c, "silu", True)
    first = backward(c, "silu", True, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, _ = forward(c, "silu", True)
        again = backward(c, "silu", True, p)
    assert torch.equal(out, out2)
    for q in first:
        assert torch.equal(first[q], again[q]), q


@pytest.mark.parametrize("m", [1, 48, 500])
def test_captured_products_replay(m):
    """forward and backward in a HIP graph, replayed with other inputs between"""
    n, k = 160, 1096
    c = {q: on(v) for q, v in case(m, n, k, torch.bfloat16, True, seed=11).items()}
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    out, p, dx, dw, db = e(m, n), e(m, 2 * n), e(m, k), e(2 * n, k), e(2 * n)
    fw = space(B.echo_linear_workspace(m, n, k, act="silu", gated=True))
    bw = space(B.echo_linear_backward_workspace(m, n, k, act="silu", gated=True))

    def step():
        B.echo_linear(c["x"], c["w"], out, bias=c["bias"], residual=c["residual"], act="silu", gated=True, p=p,
                      workspace=fw)
        B.echo_linear_backward(c["dout"], c["x"], c["w"], p, dx, dw, dbias=db, act="silu", gated=True, workspace=bw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        c["x"].copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(r)).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (out, p, dx, dw, db)]
        for v in (out, p, dx, dw, db, fw, bw):
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (out, p, dx, dw, db)):
            assert torch.equal(a, b), f"replay {r}"


def test_rows_far_apart():
    """row offsets beyond 2^32 bytes: rows of a pitch of 2^21 elements, the last
    at 4.4 GB"""
    m, n, k, ld = 1060, 72, 136, 1 << 21
    c = case(m, n, k, torch.bfloat16, False, bias=False, residual=False, seed=12)
    big = torch.empty((m - 1) * ld + 256, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((m, k), (ld, 1))
    x.copy_(c["x"])
    out, dw = torch.empty(m, n, dtype=torch.bfloat16, device=DEV), torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    B.echo_linear(x, on(c["w"]), out, workspace=space(B.echo_linear_workspace(m, n, k)))
    B.echo_linear_backward(on(c["dout"]), x, on(c["w"]), None, None, dw,
                           workspace=space(B.echo_linear_backward_workspace(m, n, k)))
    torch.cuda.synchronize()
    R.close(out, *R.linear_forward(c["x"], c["w"], None, None, "none", False)["out"], 2 * (k + 64), "out")
    e = R.linear_backward(c["dout"], c["x"], c["w"], None, "none", False)["dw"]
    R.close(dw, e[0], e[1], m + 64, "dw")


def test_differences_of_the_forward_call():
    """dx and dw along a direction against a central difference of the forward
    call: outputs of order 1 rounded to half's 2^-11 over a step of 2^-3 leave
    the difference good to about 1e-2 of the gradient's magnitude"""
    m, n, k = 24, 40, 64
    c = case(m, n, k, torch.float16, False, bias=False, residual=False, seed=13)
    _, p = forward(c, "silu", False)
    got = backward(c, "silu", False, p)
    dout = c["dout"].double()

    def objective(x, w):
        out = torch.empty(m, n, dtype=torch.float16, device=DEV)
        B.echo_linear(on(x), on(w), out, act="silu", workspace=space(B.echo_linear_workspace(m, n, k, act="silu")))
        torch.cuda.synchronize()
        return float((out.cpu().double() * dout).sum())

    gen = torch.Generator().manual_seed(3)
    for name, at in (("x", c["x"]), ("w", c["w"])):
        way = torch.randn(at.shape, generator=gen) * (1.0 if name == "x" else k ** -0.5)
        step = 2.0 ** -3
        up, down = (at.float() + step * way).half(), (at.float() - step * way).half()
        args = {"x": c["x"], "w": c["w"]}
        diff = objective(**{**args, name: up}) - objective(**{**args, name: down})
        g = got["d" + name].cpu().double()
        moved = up.double() - down.double()
        along, size = float((g * moved).sum()), float((g.abs() * moved.abs()).sum())
        assert abs(diff - along) <= 2e-2 * size, (name, diff, along, size)
