"""echo_norm and echo_norm_backward on the GPU against binary64: types, row
lengths around every row shape, norm kinds, gates, pitches, odd addresses, rows
that hold inf or NaN, single and missing tokens, streams and graphs.

Roundings on the longest path: a row's sum adds at most 16 elements in a thread,
6 steps over the lanes and 16 wavefronts (38), a norm takes two such sums and
about ten operations, and the second norm stands on the first: 128 bounds it.
A parameter's gradient adds at most 8 rows in a wavefront, 4 of those, and 32
runs of at most 32 partial sums on terms with the errors above: 256."""
import pytest
import torch

import layer_reference as R
from error_compensated_bit_echo_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROUNDINGS, SUM_ROUNDINGS = 128, 256


def rand(gen, *shape, dt=torch.float32, at=0.0, spread=1.0):
    return (at + spread * torch.randn(*shape, generator=gen)).to(dt)


def guarded(T, H, dt, ld=None, shift=0):
    """a [T, H] view of pitch ld, `shift` elements into a buffer of a sentinel"""
    ld = ld or H
    buf = torch.full((max(T, 1) * ld + shift + 64,), 7.0, dtype=dt, device=DEV)
    view = buf[shift:shift + T * ld].view(T, ld)[:, :H] if T else torch.empty(0, H, dtype=dt, device=DEV)
    return buf, view


def untouched(buf, view, what):
    """nothing outside the view was written"""
    mask = torch.ones_like(buf, dtype=torch.bool)
    if view.numel():
        off = view.storage_offset()
        mask.as_strided(view.shape, view.stride(), off).fill_(False)
    assert bool((buf[mask] == 7.0).all()), f"{what}: written outside its rows"


def case(T, H, dt, sdt, post, pre, groups, seed=0, mean=0.0):
    gen = torch.Generator().manual_seed(seed * 1000003 + T * 131 + H)
    c = {"h": rand(gen, T, H, dt=sdt, at=mean), "y": rand(gen, T, H, dt=dt, spread=0.5)}
    for k, kind in (("post", post), ("pre", pre)):
        c["w_" + k] = rand(gen, H, dt=dt, at=1.0, spread=0.2) if kind != "none" else None
        c["b_" + k] = rand(gen, H, dt=dt, spread=0.2) if kind == "layer" else None
    c["gate"] = rand(gen, groups, H, dt=dt, at=0.5, spread=0.4) if groups else None
    c["dz"] = rand(gen, T, H, dt=dt) if pre != "none" else None
    c["dh_out"] = rand(gen, T, H, dt=sdt)
    return c


def on(t):
    return None if t is None else t.to(DEV)


def check_forward(c, post, pre, scale=0.75, eps=1e-5, roundings=ROUNDINGS):
    T, H = c["h"].shape
    want = R.norm_forward(c["h"], c["y"], post, c["w_post"], c["b_post"], c["gate"], scale, pre, c["w_pre"],
                          c["b_pre"], eps)
    hb, h_out = guarded(T, H, c["h"].dtype)
    zb, z = guarded(T, H, c["y"].dtype)
    stats = torch.full((4, T), 7.0, device=DEV)
    B.echo_norm(on(c["h"]), on(c["y"]), h_out, z if pre != "none" else None, post=post, w_post=on(c["w_post"]),
                b_post=on(c["b_post"]), gate=on(c["gate"]), scale=scale, pre=pre, w_pre=on(c["w_pre"]),
                b_pre=on(c["b_pre"]), eps=eps, stats=stats)
    torch.cuda.synchronize()
    R.close(h_out, *want["h_out"], roundings, "h_out")
    if pre != "none":
        R.close(z, *want["z"], roundings, "z")
    untouched(hb, h_out, "h_out")
    untouched(zb, z, "z")
    exact, magnitude = want["stats"]
    if pre == "none":  # planes of a norm that is none: 0 and 1
        exact[2], exact[3] = 0, 1
    R.close(stats, exact, magnitude, roundings, "stats")
    return h_out, stats


def check_backward(c, post, pre, h_out, stats, scale=0.75, in_place=False):
    T, H = c["h"].shape
    dt, sdt = c["y"].dtype, c["h"].dtype
    want = R.norm_backward(c["dz"], c["dh_out"], h_out, c["y"], stats, post, c["w_post"], c["b_post"],
                           c["gate"], scale, pre, c["w_pre"])
    dhb, dh = guarded(T, H, sdt)
    dyb, dy = guarded(T, H, dt)
    if in_place:
        dh.copy_(on(c["dh_out"]))
    G = 0 if c["gate"] is None else c["gate"].shape[0]
    outs = {n: guarded(1, H, dt) for n, k in (("dw_post", post), ("db_post", post), ("dw_pre", pre), ("db_pre", pre))
            if k != "none"}
    if G:
        outs["dgate"] = guarded(G, H, dt)
    ws = torch.empty(B.echo_norm_backward_workspace(T, H, G), dtype=torch.uint8, device=DEV)
    args = dict(post=post, w_post=on(c["w_post"]), b_post=on(c["b_post"]), gate=on(c["gate"]), scale=scale,
                pre=pre, w_pre=on(c["w_pre"]), workspace=ws,
                **{n: (v if n == "dgate" else v[0]) for n, (_, v) in outs.items()})
    B.echo_norm_backward(on(c["dz"]), dh if in_place else on(c["dh_out"]), h_out, on(c["y"]), stats, dh, dy, **args)
    torch.cuda.synchronize()
    R.close(dh, *want["dh"], ROUNDINGS, "dh")
    R.close(dy, *want["dy"], ROUNDINGS, "dy")
    untouched(dhb, dh, "dh")
    untouched(dyb, dy, "dy")
    for n, (buf, v) in outs.items():
        exact, magnitude = want[n]
        R.close(v, exact.reshape(v.shape), magnitude.reshape(v.shape), SUM_ROUNDINGS, n)
        untouched(buf, v, n)
    return {"dh": dh, "dy": dy, **{n: v for n, (_, v) in outs.items()}}


TYPE_PAIRS = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]
# around the row shapes: one wavefront (to 512, to 1024), up to eight (to 4096),
# up to sixteen (to 8192, to 16384); lengths that are no multiple of 8
LENGTHS = [(1, 1), (3, 7), (5, 64), (9, 511), (6, 512), (7, 513), (5, 1024), (3, 1025), (3, 2048), (2, 2051),
           (1, 4096), (2, 4097), (2, 8192), (2, 8195), (1, 16384), (3, 16381)]


@pytest.mark.parametrize("T,H", LENGTHS)
@pytest.mark.parametrize("dt,sdt", TYPE_PAIRS)
def test_row_lengths_and_types(dt, sdt, T, H):
    print(f"norm T={T} H={H} {dt} stream {sdt}", flush=True)
    post, pre = ("layer", "rms") if H % 2 else ("rms", "layer")
    c = case(T, H, R.TYPES[dt], R.TYPES[sdt], post, pre, 1)
    h_out, stats = check_forward(c, post, pre)
    check_backward(c, post, pre, h_out, stats)


@pytest.mark.parametrize("groups", [0, 1, 2, 8, 24])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_norm_kinds_and_gates(post, pre, groups):
    for H in (100, 1030):  # a wavefront per row and four: whole groups, parts of groups, single rows
        print(f"norm T=24 H={H} {post}/{pre} groups={groups}", flush=True)
        c = case(24, H, torch.bfloat16, torch.float32, post, pre, groups, seed=3)
        h_out, stats = check_forward(c, post, pre)
        check_backward(c, post, pre, h_out, stats)


@pytest.mark.parametrize("T,H,groups", [(2050, 1032, 1025), (5000, 72, 1250), (5000, 72, 625), (4099, 40, 1),
                                        (3000, 1536, 3)])
def test_many_rows(T, H, groups):
    """workgroups that walk several rows: whole gate rows inside a workgroup's
    walk and gate rows over many workgroups"""
    print(f"norm T={T} H={H} groups={groups}", flush=True)
    c = case(T, H, torch.bfloat16, torch.bfloat16, "rms", "rms", groups, seed=4)
    h_out, stats = check_forward(c, "rms", "rms")
    check_backward(c, "rms", "rms", h_out, stats)


@pytest.mark.parametrize("T,H,groups", [(1030, 4100, 515), (600, 8200, 300), (520, 4104, 2), (770, 8195, 1)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_many_long_rows(T, H, groups, kind):
    """several rows to a workgroup of more than eight wavefronts, whose sums over
    the rows stand in LDS; with biases' gradients (layer) and without"""
    print(f"norm T={T} H={H} groups={groups} {kind}", flush=True)
    c = case(T, H, torch.float16, torch.float32, kind, kind, groups, seed=5)
    h_out, stats = check_forward(c, kind, kind)
    check_backward(c, kind, kind, h_out, stats)


def test_mean_far_from_zero_costs_no_digits():
    c = case(8, 1000, torch.float32, torch.float32, "none", "layer", 0, mean=300.0)
    check_forward(c, "none", "layer")


@pytest.mark.parametrize("shift,ld", [(0, 200), (1, 203), (3, 777)])
def test_pitches_and_odd_addresses(shift, ld):
    T, H = 11, 195
    c = case(T, H, torch.bfloat16, torch.bfloat16, "rms", "layer", 0, seed=5)
    want = R.norm_forward(c["h"], c["y"], "rms", c["w_post"], None, None, 0.75, "layer", c["w_pre"], c["b_pre"], 1e-5)
    hb, h = guarded(T, H, torch.bfloat16, ld, shift)
    yb, y = guarded(T, H, torch.bfloat16, ld + 2, shift)
    _, w = guarded(1, H, torch.bfloat16, None, shift)
    h.copy_(c["h"])
    y.copy_(c["y"])
    w.copy_(c["w_pre"][None])
    zb, z = guarded(T, H, torch.bfloat16, None, shift)
    stats = torch.empty(4, T, device=DEV)
    B.echo_norm(h, y, h, z, post="rms", w_post=on(c["w_post"]), scale=0.75, pre="layer", w_pre=w[0],
                b_pre=on(c["b_pre"]), eps=1e-5, stats=stats)  # in place: h_out is h
    torch.cuda.synchronize()
    R.close(h, *want["h_out"], ROUNDINGS, "h in place")
    R.close(z, *want["z"], ROUNDINGS, "z")
    untouched(hb, h, "h")
    untouched(zb, z, "z")
    untouched(yb, y, "y")
    back = R.norm_backward(c["dz"], c["dh_out"], h, c["y"], stats, "rms", c["w_post"], None, None, 0.75, "layer",
                           c["w_pre"])
    dyb, dy = guarded(T, H, torch.bfloat16, None, shift)
    dh = on(c["dh_out"])
    B.echo_norm_backward(on(c["dz"]), dh, h, y, stats, dh, dy, post="rms", w_post=on(c["w_post"]), scale=0.75,
                         pre="layer", w_pre=w[0])
    torch.cuda.synchronize()
    R.close(dh, *back["dh"], ROUNDINGS, "dh in place")
    R.close(dy, *back["dy"], ROUNDINGS, "dy")
    untouched(dyb, dy, "dy")


def test_first_norm_without_a_block_output():
    c = case(5, 300, torch.bfloat16, torch.float32, "none", "rms", 0)
    z = torch.empty(5, 300, dtype=torch.bfloat16, device=DEV)
    B.echo_norm(on(c["h"]), None, None, z, pre="rms", w_pre=on(c["w_pre"]), eps=1e-6)
    want = R.norm_forward(c["h"], None, "none", None, None, None, 1.0, "rms", c["w_pre"], None, 1e-6)
    R.close(z, *want["z"], ROUNDINGS, "z")


def test_no_tokens():
    H = 96
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    B.echo_norm(e(0, H), e(0, H), e(0, H), e(0, H), pre="rms", w_pre=w)
    dw, dg = torch.full_like(w, 7.0), torch.full((3, H), 7.0, dtype=torch.bfloat16, device=DEV)
    B.echo_norm_backward(e(0, H), None, e(0, H), e(0, H), torch.empty(4, 0, device=DEV), e(0, H), e(0, H),
                         gate=torch.ones(3, H, dtype=torch.bfloat16, device=DEV), pre="rms", w_pre=w, dw_pre=dw,
                         dgate=dg)
    torch.cuda.synchronize()
    assert float(dw.abs().max()) == 0 and float(dg.abs().max()) == 0  # sums over nothing


def test_inf_and_nan_stay_in_their_rows():
    T, H = 12, 640
    for bad in (float("nan"), float("inf")):
        c = case(T, H, torch.bfloat16, torch.float32, "rms", "layer", 1, seed=6)
        clean = {k: (v.clone() if v is not None else None) for k, v in c.items()}
        c["y"][4, 17] = bad
        outs = []
        for d in (c, clean):
            z = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            h_out = torch.empty(T, H, device=DEV)
            B.echo_norm(on(d["h"]), on(d["y"]), h_out, z, post="rms", w_post=on(d["w_post"]), gate=on(d["gate"]),
                        pre="layer", w_pre=on(d["w_pre"]), b_pre=on(d["b_pre"]))
            outs.append((h_out, z))
        torch.cuda.synchronize()
        keep = [r for r in range(T) if r != 4]
        for got, want in zip(*outs):
            assert torch.equal(got[keep], want[keep])
            assert bool(torch.isnan(got[4]).any())


def test_same_bits_on_every_call_and_on_another_stream():
    c = case(700, 1024, torch.bfloat16, torch.bfloat16, "rms", "rms", 1, seed=8)
    h_out, stats = check_forward(c, "rms", "rms")
    first = check_backward(c, "rms", "rms", h_out, stats)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = check_backward(c, "rms", "rms", h_out, stats, in_place=True)
    for n in first:
        assert torch.equal(first[n], again[n]), n


def test_captured_norms_replay():
    """forward and backward in a HIP graph, replayed with other inputs between"""
    T, H = 64, 1024
    c = case(T, H, torch.bfloat16, torch.bfloat16, "none", "rms", 0, seed=9)
    t = {k: on(v) for k, v in c.items()}
    h_out, z, dh, dy = (torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    stats = torch.empty(4, T, device=DEV)
    dw = torch.empty(H, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(B.echo_norm_backward_workspace(T, H), dtype=torch.uint8, device=DEV)

    def step():
        B.echo_norm(t["h"], t["y"], h_out, z, pre="rms", w_pre=t["w_pre"], stats=stats)
        B.echo_norm_backward(t["dz"], t["dh_out"], h_out, t["y"], stats, dh, dy, pre="rms", w_pre=t["w_pre"],
                             dw_pre=dw, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        t["y"].copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (h_out, z, stats, dh, dy, dw)]
        for v in (h_out, z, stats, dh, dy, dw):
            v.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (h_out, z, stats, dh, dy, dw)):
            assert torch.equal(a, b), f"replay {k}"


def test_differences_of_the_forward_call():
    """the backward call's dh, dy along a direction against a central difference
    of the forward call itself (binary32, so a step of 2^-6 is where the
    difference's own error, step^2 and rounding / step, is smallest)"""
    T, H, scale = 4, 256, 0.5
    c = case(T, H, torch.float32, torch.float32, "layer", "rms", 2, seed=12)
    h_out, stats = check_forward(c, "layer", "rms", scale=scale)
    got = check_backward(c, "layer", "rms", h_out, stats, scale=scale)
    dz, dh_out = c["dz"].double(), c["dh_out"].double()

    def objective(h, y):
        a, b = torch.empty(T, H, device=DEV), torch.empty(T, H, device=DEV)
        B.echo_norm(on(h), on(y), a, b, post="layer", w_post=on(c["w_post"]), b_post=on(c["b_post"]),
                    gate=on(c["gate"]), scale=scale, pre="rms", w_pre=on(c["w_pre"]), b_pre=None, eps=1e-5)
        torch.cuda.synchronize()
        return float((a.cpu().double() * dh_out).sum() + (b.cpu().double() * dz).sum())

    gen = torch.Generator().manual_seed(2)
    step = 2.0 ** -6
    for name in ("h", "y"):
        way = torch.randn(T, H, generator=gen)
        at = {"h": c["h"], "y": c["y"]}
        up = objective(**{k: (v + step * way if k == name else v) for k, v in at.items()})
        down = objective(**{k: (v - step * way if k == name else v) for k, v in at.items()})
        along = float((got["d" + name].cpu().double() * way.double()).sum())
        size = float((got["d" + name].cpu().double().abs() * way.double().abs()).sum())
        assert abs((up - down) / (2 * step) - along) <= 4e-3 * size, name
