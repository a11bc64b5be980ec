"""echo_linear8 on the GPU against binary64: both types, both formats of x, every
activation and gate, scales that are powers of two, others and both in one row,
sizes around the tiles and blocks, odd sizes with anything behind a row's end,
pitches, single rows, empty sides, NaN, streams and graphs.

Bounds.  fp8_reference.products has what the matrix cores' sums of eight products
lose; every other addition is off by at most one unit of 2^-23 of the magnitude of
the terms: 2 (c + 64) units of 2^-24, the 64 for the scales' product, bias,
activation and residual (as in the tests of echo_linear).  That bound grows with the
sum, so layer_sums.near also holds every row and column by its norm: one rounding
to the type, and for what is cut 2^-12.  (A cut is below 2^-13 of the largest of
eight products, for normal values within 4 of their root mean square, so 2^-11 of
it; uniform below that, 1 / sqrt 3; and only products below 2^-7 of the largest
lose anything, less than 0.4 of them: 2^-11 sqrt(.4 / 3) < 2^-12, of either sign.)"""
import numpy as np
import pytest
import torch

import fp8_reference as F
import layer_reference as R
import layer_sums as S
from error_compensated_bit_echo_amd import binding as B
from test_gpu_norm import DEV, guarded, on, rand, untouched

pytestmark = pytest.mark.gpu


def scales_of(kind, shape, gen):
    """"pow2", "any", or "mixed": powers of two but for some of the later blocks"""
    s = torch.exp2(torch.randint(-6, 3, shape, generator=gen).float())
    if kind == "pow2":
        return s
    other = s * (0.5 + torch.rand(shape, generator=gen))
    if kind == "any":
        return other
    late = torch.rand(shape, generator=gen) < 0.2
    late[:, :shape[1] // 2] = False
    return torch.where(late, other, s)


def operand(rows, cols, fmt, gen, extra=0):
    """(codes on the GPU in rows of a pitch filled with NaN, their bytes)"""
    pitch = (cols + 15) // 16 * 16 + extra
    raw = torch.randn(rows, cols, generator=gen).to(F.FORMATS[fmt])
    buf = torch.full((max(rows, 1), pitch), 0x7F, dtype=torch.uint8, device=DEV)
    buf[:rows, :cols] = raw.view(torch.uint8).to(DEV)
    return buf[:rows, :cols].view(F.FORMATS[fmt]), raw.view(torch.uint8).numpy()


def case(m, n, k, dt, gated=False, fmt="e4m3", scales="pow2", bias=True, residual=True, seed=0, extra=(0, 0)):
    gen = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    rows, parts = (2 * n, 2) if gated else (n, 1)
    x, xr = operand(m, k, fmt, gen, extra[0])
    w, wr = operand(rows, k, "e4m3", gen, extra[1])
    sx = scales_of(scales, F.scales_shape(m, k, False, 1), gen)
    sw = scales_of("pow2" if scales == "mixed" else scales, F.scales_shape(rows, k, True, parts), gen) * max(k, 1) ** -0.5
    if scales != "any":
        sw = torch.exp2(torch.round(torch.log2(sw)))
    return {"x": x, "w": w, "sx": sx, "sw": sw, "xr": xr, "wr": wr, "fmt": fmt,
            "bias": rand(gen, rows, dt=dt, spread=0.3) if bias else None,
            "residual": rand(gen, m, n, dt=dt) if residual else None, "dt": dt, "gated": gated}


def space(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def forward(c, act, keep=True, pad=0, sums=True, stream=None):
    (m, k), rows, dt, gated = c["x"].shape, c["w"].shape[0], c["dt"], c["gated"]
    n = rows // 2 if gated else rows
    ob, out = guarded(m, n, dt, n + pad, 1 if pad else 0)
    pb, p = guarded(m, rows, dt)
    print(f"linear8 m={m} n={n} k={k} {dt} {act} gated={gated} {c['x'].dtype}", flush=True)
    B.echo_linear8(c["x"], on(c["sx"]), c["w"], on(c["sw"]), out, bias=on(c["bias"]), residual=on(c["residual"]), act=act,
                   gated=gated, p=p if keep else None, workspace=space(B.echo_linear8_workspace(m, n, k, act=act, gated=gated)))
    torch.cuda.synchronize()
    units = 2 * (k + 64)
    want = F.linear_forward(c["xr"], c["sx"].double().numpy(), c["fmt"], c["wr"], c["sw"].double().numpy(), c["bias"],
                            c["residual"], act, gated, units)
    R.close(out, *want["out"], units, "out")
    untouched(ob, out, "out")
    if keep:
        R.close(p, *want["p"], units, "p")
        untouched(pb, p, "p")
    if sums and keep and k >= 64:
        S.near(p, torch.from_numpy(want["p"][0]), 1 + 2.0 ** -12 / R.HALF_ULP[dt], "p")
    return out, p


TYPES = [torch.bfloat16, torch.float16]
SMALL = [(1, 16, 128), (1, 1, 1), (16, 24, 256), (3, 130, 200), (16, 7, 1000), (5, 264, 4096), (2, 33, 16), (1, 1792, 4096)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", SMALL)
def test_few_rows(m, n, k, gated, dt):
    forward(case(m, n, k, dt, gated), "silu" if gated else "none")
    forward(case(m, n, k, dt, gated, fmt="e5m2", scales="any", seed=1), "gelu")


@pytest.mark.parametrize("k", [1023, 1920, 2047, 2048, 2049, 2177, 4095, 4097])
@pytest.mark.parametrize("gated", [False, True])
def test_few_rows_of_every_share_of_blocks(gated, k):
    forward(case(11, 40, k, torch.bfloat16, gated, scales="any"), "silu" if gated else "none")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", [(17, 16, 128), (64, 64, 128), (65, 63, 127), (63, 65, 129), (128, 128, 256), (129, 200, 384),
                                   (100, 1, 640), (40, 130, 1001), (300, 260, 33), (256, 96, 16), (77, 31, 1)])
def test_tiles(m, n, k, gated, dt):
    forward(case(m, n, k, dt, gated), "silu" if gated else "none")
    forward(case(m, n, k, dt, gated, scales="any", seed=1), "gelu_tanh")


@pytest.mark.parametrize("act", list(B.ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [4, 70])
def test_activations(m, gated, act):
    forward(case(m, 72, 300, torch.bfloat16, gated), act)
    forward(case(m, 72, 300, torch.float16, gated, bias=False, residual=False), act, keep=False)


@pytest.mark.parametrize("scales", ["pow2", "any", "mixed"])
@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("m,n,k,gated", [(200, 264, 1200, False), (200, 140, 1200, True), (12, 264, 1200, False), (12, 140, 1200, True)])
def test_scales(m, n, k, gated, fmt, scales):
    forward(case(m, n, k, torch.bfloat16, gated, fmt, scales), "silu" if gated else "none")


def test_scales_of_every_size():
    """powers of two to the ends of their range, a subnormal one, 0 and -1: what the matrix
    cores cannot apply is applied beside them"""
    for bad in (0.0, -1.0, 2.0 ** -127, 2.0 ** -126, 2.0 ** 100, 3.0):
        for m in (8, 80):
            c = case(m, 48, 512, torch.bfloat16, bias=False, residual=False)
            c["sx"][m // 2, 2] = bad
            c["sx"][1, 1] = bad
            forward(c, "none", sums=False)


@pytest.mark.parametrize("m", [9, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_pitches(m, gated):
    forward(case(m, 90, 333, torch.bfloat16, gated, extra=(16, 64)), "silu", pad=5)
    forward(case(m, 90, 320, torch.float16, gated, extra=(48, 0)), "none", pad=8)


@pytest.mark.parametrize("m", [6, 90])
def test_in_place_residual(m):
    c = case(m, 64, 256, torch.bfloat16)
    want, _ = forward(c, "none")
    out = on(c["residual"]).clone()
    B.echo_linear8(c["x"], on(c["sx"]), c["w"], on(c["sw"]), out, bias=on(c["bias"]), residual=out,
                   workspace=space(B.echo_linear8_workspace(m, 64, 256)))
    assert torch.equal(out, want)


@pytest.mark.parametrize("m,n,k", [(1000, 520, 96), (4100, 2060, 64)])
def test_in_place_residual_of_many_tiles(m, n, k):
    """rows and columns at odd addresses, whose last tiles are cut both ways"""
    c = case(m, n, k, torch.float16)
    w, room = (c["w"], on(c["sw"])), space(B.echo_linear8_workspace(m, n, k, act="relu"))
    want = torch.empty(m, n, dtype=torch.float16, device=DEV)
    B.echo_linear8(c["x"], on(c["sx"]), *w, want, bias=on(c["bias"]), residual=on(c["residual"]), act="relu", workspace=room)
    buf, out = guarded(m, n, torch.float16, n + 3, 1)
    out.copy_(c["residual"])
    B.echo_linear8(c["x"], on(c["sx"]), *w, out, bias=on(c["bias"]), residual=out, act="relu", workspace=room)
    assert torch.equal(out, want)
    untouched(buf, out, "out")


@pytest.mark.parametrize("m,n,k", [(0, 8, 8), (4, 0, 8), (4, 8, 0), (40, 8, 0)])
def test_empty_sides(m, n, k):
    forward(case(m, n, k, torch.bfloat16), "silu", sums=False)


@pytest.mark.parametrize("m", [7, 100])
@pytest.mark.parametrize("fmt", F.FORMATS)
def test_nan_spoils_its_row_only(m, fmt):
    c = case(m, 200, 700, torch.bfloat16, fmt=fmt, bias=False, residual=False)
    ok, _ = forward(c, "none")
    ok = ok.clone()
    c["x"].view(torch.uint8)[3, 650] = 0x7F
    out = torch.empty_like(ok)
    ws = space(B.echo_linear8_workspace(m, 200, 700))
    B.echo_linear8(c["x"], on(c["sx"]), c["w"], on(c["sw"]), out, workspace=ws)
    assert bool(torch.isnan(out[3]).all())
    rest = torch.arange(m, device=DEV) != 3
    assert torch.equal(out[rest], ok[rest])
    c["x"].view(torch.uint8)[3, 650] = 0
    c["sx"][5, 2] = float("nan")
    B.echo_linear8(c["x"], on(c["sx"]), c["w"], on(c["sw"]), out, workspace=ws)
    assert bool(torch.isnan(out[5]).all()) and bool(torch.isfinite(out[torch.arange(m, device=DEV) != 5].float()).all())


def test_splits_and_their_join():
    """long contractions over few tiles"""
    for m, n, k, gated in ((256, 512, 16384, False), (192, 130, 16389, True), (500, 257, 9000, False)):
        assert B.echo_linear8_workspace(m, n, k, gated=gated) > 0
        forward(case(m, n, k, torch.bfloat16, gated), "silu" if gated else "none")
        forward(case(m, n, k, torch.float16, gated, scales="mixed"), "gelu")


def test_same_bits_again():
    for m in (5, 300):
        c = case(m, 320, 2048, torch.bfloat16, scales="mixed")
        a, _ = forward(c, "none")
        b, _ = forward(c, "none")
        assert torch.equal(a, b)


def test_streams_and_graph():
    c = case(200, 136, 900, torch.bfloat16, scales="mixed")
    d = case(3, 136, 900, torch.bfloat16, seed=2)
    want = [forward(q, "silu")[0].clone() for q in (c, d)]
    side = torch.cuda.Stream()
    outs = [torch.empty_like(w) for w in want]
    args = [(q["x"], on(q["sx"]), q["w"], on(q["sw"]), o, on(q["bias"]), on(q["residual"]),
             space(B.echo_linear8_workspace(*o.shape, 900))) for q, o in zip((c, d), outs)]

    def run():
        for x, sx, w, sw, o, b, r, ws in args:
            B.echo_linear8(x, sx, w, sw, o, bias=b, residual=r, act="silu", workspace=ws)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.randn(100, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_gradient_of_x_in_8_bits():
    """dx = dp w by the same call, on the packed gradient and the transposed weights"""
    gen = torch.Generator().manual_seed(3)
    m, n, k = 70, 256, 200
    w = rand(gen, n, k, dt=torch.bfloat16, spread=k ** -0.5).to(DEV)
    dp = rand(gen, m, n, dt=torch.bfloat16, spread=1e-3).to(DEV)
    w8, sw = B.codes8_empty(n, k), torch.empty(B.scales8_shape(n, k, blocks=True), device=DEV)
    wt, st = B.codes8_empty(k, n), torch.empty(B.scales8_shape(k, n, blocks=True), device=DEV)
    B.echo_pack8(w, w8, sw, blocks=True, codes_t=wt, scales_t=st)
    d8, sd = B.codes8_empty(m, n, torch.float8_e5m2), torch.empty(B.scales8_shape(m, n), device=DEV)
    B.echo_pack8(dp, d8, sd)
    dx = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    B.echo_linear8(d8, sd, wt, st, dx, workspace=space(B.echo_linear8_workspace(m, k, n)))
    torch.cuda.synchronize()
    raw = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()  # noqa: E731
    units = 2 * (n + 64)
    want, magnitude = F.products(raw(d8), sd.cpu().double().numpy(), "e5m2", raw(wt), st.cpu().double().numpy(), 1, units)
    R.close(dx, want, magnitude, units, "dx")
    # and by the weights as they were packed
    dv = F.values(raw(d8), sd.cpu().double().numpy(), "e5m2")
    np.testing.assert_allclose(want, dv @ F.values(raw(w8), sw.cpu().double().numpy(), "e4m3", True), rtol=1e-9, atol=1e-12)


def test_refusals_with_tensors():
    c = case(20, 32, 64, torch.bfloat16, bias=False, residual=False)
    out = torch.empty(20, 32, dtype=torch.bfloat16, device=DEV)
    sx, sw = on(c["sx"]), on(c["sw"])
    for args, match in (((c["x"], sx, c["w"].contiguous().view(torch.uint8), sw, out), "w"),
                        ((c["x"], sx.double(), c["w"], sw, out), "sx"), ((c["x"], sx, c["w"], sw.t().expand(2, 1), out), "sw"),
                        ((c["x"], sx, c["w"], sw, out.float()), "out"), ((c["x"], sx, c["w"], sw, out[:, :16]), "out"),
                        ((c["x"][:, :8], sx, c["w"], sw, out), "w")):
        with pytest.raises(ValueError, match=match):
            B.echo_linear8(*args)
    with pytest.raises(ValueError, match="p"):
        B.echo_linear8(c["x"], sx, c["w"], sw, out, p=torch.empty(20, 30, dtype=torch.bfloat16, device=DEV))
