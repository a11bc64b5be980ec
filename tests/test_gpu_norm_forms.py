"""The forms of echo_norm_backward on the GPU against binary64: with and without a
post norm or gate, with and without the biases' gradients, over every row shape, each
with rows of whole vectors and of short last ones, several rows to a workgroup.

Row shapes.  Without a post norm and a gate: a wavefront with one vector a lane to 512
elements and two to 1024, up to eight wavefronts to 4096, up to sixteen to 8192 and
with two vectors past that; with one of them two vectors begin past 8192 only and a
wavefront holds rows to 512.  Bounds: those of test_gpu_norm for every element, with
sums over at most 40 rows in a wavefront's run, four runs side by side and 32 runs of
32 partial sums behind it; and every row and column by its norm (layer_sums)."""
import pytest
import torch

import layer_sums as S
from error_compensated_bit_echo_amd import binding as B
from layer_reference import TYPES
from test_gpu_norm import DEV, ROUNDINGS, SUM_ROUNDINGS, TYPE_PAIRS, guarded, untouched

pytestmark = pytest.mark.gpu

# tokens: more than one row to a workgroup
SHAPES = [(4500, 5), (4500, 512), (4500, 509), (4200, 1024), (4200, 1021), (1100, 2048), (1100, 2051), (600, 4096),
          (600, 4093), (530, 8192), (530, 8189), (300, 16384), (300, 16381)]


def case(T, H, dt, sdt, post, pre, groups, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + T * 131 + H)
    rand = lambda *s, t=dt, at=0.0, spread=1.0: (at + spread * torch.randn(*s, generator=gen, device=DEV)).to(t)  # noqa: E731
    c = {"h": rand(T, H, t=sdt), "y": rand(T, H, spread=0.5), "dh_out": rand(T, H, t=sdt),
         "dz": rand(T, H) if pre != "none" else None, "gate": rand(groups, H, at=0.5, spread=0.4) if groups else None}
    for k, kind in (("post", post), ("pre", pre)):
        c["w_" + k] = rand(H, at=1.0, spread=0.2) if kind != "none" else None
        c["b_" + k] = rand(H, spread=0.2) if kind == "layer" else None
    h_out, stats = torch.empty_like(c["h"]), torch.empty(4, T, device=DEV)
    z = torch.empty(T, H, dtype=dt, device=DEV) if pre != "none" else None
    B.echo_norm(c["h"], c["y"], h_out, z, post=post, w_post=c["w_post"], b_post=c["b_post"], gate=c["gate"], scale=0.75,
                pre=pre, w_pre=c["w_pre"], b_pre=c["b_pre"], eps=1e-5, stats=stats)
    return {**c, "h_out": h_out, "stats": stats}


def gradients(c, post, pre, sums, y=True, dy=True):
    """{name: (buffer, view)} of a call that asks for `sums`, dh and dy"""
    T, H = c["h"].shape
    dt = c["y"].dtype
    outs = {"dh": guarded(T, H, c["h"].dtype)}
    if dy:
        outs["dy"] = guarded(T, H, dt)
    for n in sums:
        outs[n] = guarded(c["gate"].shape[0] if n == "dgate" else 1, H, dt)
    size = B.echo_norm_backward_workspace(T, H, 0 if c["gate"] is None else c["gate"].shape[0])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if sums else None  # NaN in every word
    B.echo_norm_backward(c["dz"], c["dh_out"], c["h_out"] if pre != "none" else None, c["y"] if y else None, c["stats"],
                         outs["dh"][1], outs["dy"][1] if dy else None, post=post, w_post=c["w_post"], b_post=c["b_post"],
                         gate=c["gate"], scale=0.75, pre=pre, w_pre=c["w_pre"], workspace=ws,
                         **{n: (v if n == "dgate" else v[0]) for n, (_, v) in outs.items() if n in sums})
    torch.cuda.synchronize()
    return outs


def check(c, post, pre, sums, **kw):
    outs = gradients(c, post, pre, sums, **kw)
    want = S.norm_backward(c["dz"], c["dh_out"], c["h_out"], c["y"], c["stats"], post, c["w_post"], c["b_post"],
                           c["gate"], 0.75, pre, c["w_pre"])
    for n, (buf, v) in outs.items():
        exact, magnitude = (t.reshape(v.shape) for t in want[n])
        S.elements(v, exact, magnitude, SUM_ROUNDINGS if n in sums else ROUNDINGS, n)
        if v.shape[1] >= 64:
            S.near(v, exact, 1, n)
        untouched(buf, v, n)


def wanted(post, pre, biases, gate=False):
    sums = [f"d{v}_{k}" for k, kind in (("post", post), ("pre", pre)) if kind != "none" for v in ("wb" if biases else "w")]
    return sums + (["dgate"] if gate else [])


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dt,sdt", TYPE_PAIRS)
def test_a_pre_norm_alone(dt, sdt, T, H):
    """no post norm, no gate: the backward pass of a pre-norm model"""
    for pre, biases in (("rms", False), ("layer", True), ("layer", False)):
        print(f"norm T={T} H={H} {dt} stream {sdt} none/{pre} biases={biases}", flush=True)
        check(case(T, H, TYPES[dt], TYPES[sdt], "none", pre, 0, seed=1), "none", pre, wanted("none", pre, biases))


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dt,sdt", TYPE_PAIRS)
def test_norms_on_both_sides(dt, sdt, T, H):
    """gates of one row, of rows over whole workgroups and in parts, of a row per
    token, and none; with the biases' gradients and without"""
    for post, pre, biases, groups in (("rms", "rms", False, 0), ("rms", "rms", False, 1), ("layer", "layer", True, T // 2),
                                      ("layer", "rms", False, 2), ("rms", "layer", True, T)):
        print(f"norm T={T} H={H} {dt} stream {sdt} {post}/{pre} biases={biases} groups={groups}", flush=True)
        check(case(T, H, TYPES[dt], TYPES[sdt], post, pre, groups, seed=2), post, pre, wanted(post, pre, biases, groups > 0))


@pytest.mark.parametrize("T,H", [(33000, 256), (33000, 1024), (20000, 4096), (20000, 2051)])
@pytest.mark.parametrize("post,pre,groups", [("none", "rms", 0), ("rms", "rms", 8)])
def test_long_runs_of_rows(post, pre, groups, T, H):
    """as a training step has them: the sums over many rows lose none"""
    print(f"norm T={T} H={H} {post}/{pre} groups={groups}", flush=True)
    check(case(T, H, torch.bfloat16, torch.bfloat16, post, pre, groups, seed=4), post, pre,
          wanted(post, pre, False, groups > 0))


@pytest.mark.parametrize("H", [512, 1021, 4096, 8189, 16384])
def test_outputs_asked_for_alone(H):
    """no sums and no workspace, one sum, no dy, a gate without its gradient and
    without y"""
    T = 300
    for post, pre, groups in (("none", "rms", 0), ("rms", "layer", 2), ("none", "none", 2), ("layer", "none", 0)):
        print(f"norm T={T} H={H} {post}/{pre} groups={groups}", flush=True)
        c = case(T, H, torch.bfloat16, torch.float32, post, pre, groups, seed=3)
        check(c, post, pre, [])
        check(c, post, pre, [], dy=False)
        for one in wanted(post, pre, True, groups > 0):
            check(c, post, pre, [one])
        if post == "none":
            check(c, post, pre, [] if pre == "none" else ["dw_pre"], y=False)
