"""echo_linear_backward8 on the GPU against binary64: both types, activations and gates,
odd sizes, pitches, outputs left out, empty sides, NaN, streams and graphs.

Bounds as in the tests of echo_linear_backward: dp rounded to the type in the terms of
dx and dw, sums of c terms; x unpacked to the type is exact for scales that are powers
of two, and one rounding more in the terms of dw for others."""
import numpy as np
import pytest
import torch

import fp8_reference as F
import layer_reference as R
import layer_sums as S
from error_compensated_bit_echo_amd import binding as B
from test_gpu_linear8 import operand, scales_of, space
from test_gpu_norm import DEV, guarded, on, rand, untouched

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def case(m, n, k, dt, act, gated, fmt="e4m3", scales="pow2", seed=0, extra=(0, 0)):
    gen = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    rows, parts = (2 * n, 2) if gated else (n, 1)
    c = {"dt": dt, "act": act, "gated": gated, "p": None, "sp": None, "pv": None, "scales": scales}
    c["x"], xr = operand(m, k, fmt, gen, extra[0])
    c["sx"] = scales_of(scales, F.scales_shape(m, k, False, 1), gen) * 0.25
    c["xv"] = F.values(xr, c["sx"].double().numpy(), fmt)
    c["w"] = rand(gen, rows, k, dt=dt, spread=max(k, 1) ** -0.5)
    c["dout"] = rand(gen, m, n, dt=dt)
    if act != "none" or gated:
        c["p"], pr = operand(m, rows, "e4m3", gen, extra[1])
        c["sp"] = scales_of(scales, F.scales_shape(m, rows, False, parts), gen) * 0.25
        c["pv"] = F.values(pr, c["sp"].double().numpy(), "e4m3", False, parts)
    return c


def backward(c, want=("dx", "dw", "dbias"), pads=(0, 0), shift=0, sums=True):
    (m, k), rows, dt = c["x"].shape, c["w"].shape[0], c["dt"]
    n = rows // 2 if c["gated"] else rows
    _, w = guarded(rows, k, dt, k + pads[0], shift)
    _, dout = guarded(m, n, dt, n + pads[1], shift)
    w.copy_(c["w"])
    dout.copy_(c["dout"])
    outs = {"dx": guarded(m, k, dt), "dw": guarded(rows, k, dt), "dbias": guarded(1, rows, dt)}
    give = {q: (v[0] if q == "dbias" else v) if q in want else None for q, (_, v) in outs.items()}
    print(f"linear_backward8 m={m} n={n} k={k} {dt} {c['act']} gated={c['gated']} {want}", flush=True)
    ws = space(B.echo_linear_backward8_workspace(m, n, k, act=c["act"], gated=c["gated"]))
    B.echo_linear_backward8(dout, c["x"], on(c["sx"]), w, c["p"], on(c["sp"]), give["dx"], give["dw"], dbias=give["dbias"],
                            act=c["act"], gated=c["gated"], workspace=ws)
    torch.cuda.synchronize()
    pv = None if c["pv"] is None else torch.from_numpy(c["pv"])
    exact = R.linear_backward(c["dout"], torch.from_numpy(c["xv"]), c["w"], pv, c["act"], c["gated"])
    length = {"dx": rows, "dw": m, "dbias": m}
    roundings = {"dx": 0 if c["pv"] is None else 1, "dw": (0 if c["pv"] is None else 1) + (c["scales"] != "pow2"), "dbias": 0}
    half = R.HALF_ULP[dt] / R.EPS32
    for q in want:
        buf, v = outs[q]
        e, magnitude = exact[q][0].reshape(v.shape), exact[q][1].reshape(v.shape)
        if q != "dbias" and roundings[q]:  # each rounding of a factor of the terms, in units of 2^-24
            magnitude = magnitude + roundings[q] * 1.01 * half / (length[q] + 64) * exact[q][2].reshape(v.shape)
        R.close(v, e, magnitude, length[q] + 64, q)
        untouched(buf, v, q)
        if sums and length[q] >= 64:
            S.near(v, torch.from_numpy(e), 1 + roundings[q], q)
    return {q: outs[q][1] for q in want}


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", True), ("gelu", False), ("gelu_tanh", True), ("relu", False)])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 16, 40), (64, 128, 64), (130, 72, 200), (33, 137, 129), (300, 7, 259), (257, 264, 24)])
def test_shapes(m, n, k, act, gated, dt):
    backward(case(m, n, k, dt, act, gated))


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("scales", ["pow2", "any"])
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", True)])
def test_formats_and_scales(fmt, scales, act, gated):
    # (e5m2 holds values past half's precision but not, at these scales, past its range)
    for dt in TYPES:
        backward(case(200, 96, 300, dt, act, gated, fmt, scales))


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias")])
@pytest.mark.parametrize("act,gated,n,k", [("none", False, 40, 72), ("none", False, 41, 73), ("silu", True, 41, 73)])
def test_outputs_left_out(want, act, gated, n, k):
    c = case(90, n, k, torch.bfloat16, act, gated)
    if "dw" not in want:
        every = backward(c)
        few = backward(c, want)
        assert all(torch.equal(few[q], every[q]) for q in want)
        m, rows = 90, c["w"].shape[0]
        # x's tensors are named by their shape and not read
        dx = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
        B.echo_linear_backward8(on(c["dout"]), c["x"], on(c["sx"]) * float("nan"), on(c["w"]), c["p"], on(c["sp"]), dx, None,
                                act=act, gated=gated, workspace=space(B.echo_linear_backward8_workspace(m, n, k, act=act, gated=gated)))
        assert torch.equal(dx, every["dx"]) and rows == (2 * n if gated else n)
    else:
        backward(c, want)


@pytest.mark.parametrize("act,gated", [("none", False), ("gelu", True)])
def test_pitches_and_addresses(act, gated):
    for extra, pads, shift in (((16, 32), (5, 3), 1), ((0, 48), (8, 8), 0)):
        backward(case(77, 90, 333, torch.bfloat16, act, gated, extra=extra), pads=pads, shift=shift)


@pytest.mark.parametrize("m,n,k", [(0, 8, 8), (4, 0, 8), (4, 8, 0)])
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", True)])
def test_empty_sides(m, n, k, act, gated):
    got = backward(case(m, n, k, torch.bfloat16, act, gated), sums=False)
    if m == 0:
        assert float(got["dw"].float().abs().sum()) == 0 and float(got["dbias"].float().abs().sum()) == 0


@pytest.mark.parametrize("dt", TYPES)
def test_long_sums(dt):
    backward(case(6000, 130, 70, dt, "silu", True))
    backward(case(5003, 131, 71, dt, "gelu", False))


def test_nan_stays_where_the_formulas_let_it_reach():
    c = case(100, 64, 96, torch.bfloat16, "silu", False)
    c["x"].view(torch.uint8)[7, 30] = 0x7F
    c["p"].view(torch.uint8)[9, 20] = 0x7F
    ws = space(B.echo_linear_backward8_workspace(100, 64, 96, act="silu"))
    dx, dw = torch.empty(100, 96, dtype=torch.bfloat16, device=DEV), torch.empty(64, 96, dtype=torch.bfloat16, device=DEV)
    db = torch.empty(64, dtype=torch.bfloat16, device=DEV)
    B.echo_linear_backward8(on(c["dout"]), c["x"], on(c["sx"]), on(c["w"]), c["p"], on(c["sp"]), dx, dw, dbias=db, act="silu",
                            workspace=ws)
    nx, nw = torch.isnan(dx).cpu(), torch.isnan(dw).cpu()
    assert bool(nx[9].all()) and not bool(nx[torch.arange(100) != 9].any())
    assert bool(nw[20].all()) and bool(nw[:, 30].all())
    rest = nw[torch.arange(64) != 20][:, torch.arange(96) != 30]
    assert not bool(rest.any())
    assert torch.isnan(db).cpu().tolist() == [j == 20 for j in range(64)]


def test_gradients_against_differences():
    """dw and dx of a linear loss against central differences of the formula in binary64"""
    c = case(6, 9, 33, torch.float16, "gelu", True, seed=4)
    # p as the checkpoint has it, as if it were x w^T plus what the rounding added
    x, w = torch.from_numpy(c["xv"]), c["w"].double()
    rest = torch.from_numpy(c["pv"]) - x @ w.T
    dout = c["dout"].double()

    def loss(x, w):
        p = x @ w.T + rest
        return float((torch.nn.functional.gelu(p[:, :9]) * p[:, 9:] * dout).sum())

    got = backward(c, sums=False)
    h = 1e-5
    for name, at in (("dx", [(0, 0), (5, 32), (2, 17)]), ("dw", [(0, 0), (17, 32), (8, 5), (9, 11)])):
        for i, j in at:
            e = torch.zeros_like(x if name == "dx" else w)
            e[i, j] = h
            d = (loss(x + e, w) - loss(x - e, w) if name == "dx" else loss(x, w + e) - loss(x, w - e)) / (2 * h)
            scale = float(got[name].double().abs().max())
            assert abs(float(got[name][i, j]) - d) <= 2.0 ** -8 * scale, (name, i, j)


def test_streams_and_graph():
    c = case(200, 72, 136, torch.bfloat16, "silu", True)
    want = {q: v.clone() for q, v in backward(c).items()}
    t = {q: on(c[q]) for q in ("dout", "sx", "w", "sp")}
    dx, dw = torch.empty(200, 136, dtype=torch.bfloat16, device=DEV), torch.empty(144, 136, dtype=torch.bfloat16, device=DEV)
    db = torch.empty(144, dtype=torch.bfloat16, device=DEV)
    ws = space(B.echo_linear_backward8_workspace(200, 72, 136, act="silu", gated=True))

    def run():
        B.echo_linear_backward8(t["dout"], c["x"], t["sx"], t["w"], c["p"], t["sp"], dx, dw, dbias=db, act="silu", gated=True,
                                workspace=ws)

    def same():
        torch.cuda.synchronize()
        return torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"]) and torch.equal(db, want["dbias"].view(-1))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for o in (dx, dw, db, ws):
            o.zero_()
        graph.replay()
        assert same()


@pytest.mark.parametrize("gated", [False, True])
def test_offsets_past_32_bits(gated):
    """codes of p past 2^31 bytes, dout and dp past 2^32: the first and last rows have a
    gradient, and sums over all rows add nothing of the others (a zero rounds nothing, so
    the bounds are of the rows that have one)"""
    m, n, k, some = 131200, 8264 if gated else 16520, 16, 96
    c = case(2 * some, n, k, torch.bfloat16, "relu", gated)

    def grown(t):
        big = torch.zeros(m, t.shape[1], dtype=t.dtype, device=DEV)
        big[:some], big[-some:] = t[:some], t[some:]
        return big

    def codes(t):
        big = B.codes8_empty(m, t.shape[1])
        big.view(torch.uint8).zero_()
        big.view(torch.uint8)[:some], big.view(torch.uint8)[-some:] = t.view(torch.uint8)[:some], t.view(torch.uint8)[some:]
        return big

    rows = c["w"].shape[0]
    dx, dw = torch.empty(m, k, dtype=c["dt"], device=DEV), torch.empty(rows, k, dtype=c["dt"], device=DEV)
    db = torch.empty(rows, dtype=c["dt"], device=DEV)
    print(f"linear_backward8 m={m} n={n} k={k} gated={gated}", flush=True)
    B.echo_linear_backward8(grown(on(c["dout"])), codes(c["x"]), grown(on(c["sx"])), on(c["w"]), codes(c["p"]), grown(on(c["sp"])),
                            dx, dw, dbias=db, act="relu", gated=gated,
                            workspace=space(B.echo_linear_backward8_workspace(m, n, k, act="relu", gated=gated)))
    torch.cuda.synchronize()
    exact = R.linear_backward(c["dout"], torch.from_numpy(c["xv"]), c["w"], torch.from_numpy(c["pv"]), "relu", gated)
    half = R.HALF_ULP[c["dt"]] / R.EPS32
    for q, v, length in (("dx", torch.cat([dx[:some], dx[-some:]]), rows), ("dw", dw, 2 * some), ("dbias", db, 2 * some)):
        e, magnitude = exact[q][:2]
        if q != "dbias":
            magnitude = magnitude + 1.01 * half / (length + 64) * exact[q][2]
        R.close(v, e, magnitude, length + 64, q)
    assert not dx[some:-some].any()
