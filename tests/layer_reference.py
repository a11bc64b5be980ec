"""The layer operators in binary64, straight from their formulas, on the CPU,
each with the magnitude of the terms that its sums add up.

A result r of the library is held to |r - exact| <= u |exact| + k 2^-24 M + tiny:
u is half a unit in the last place of the output's type (its one rounding), M
the magnitude of the terms, k the number of binary32 roundings on the longest
path to the result (a sum of n terms in any fixed order has at most its depth of
them), and tiny half the smallest subnormal of the type."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
EPS32 = 2.0 ** -24


def close(got, exact, magnitude, roundings, what):
    """got (a tensor of its own type) against binary64, by the bound above"""
    dt = got.dtype
    g = got.detach().cpu().double().numpy()
    exact, magnitude = np.asarray(exact, np.float64), np.asarray(magnitude, np.float64)
    assert g.shape == exact.shape, (what, g.shape, exact.shape)
    room = HALF_ULP[dt] * np.abs(exact) + roundings * EPS32 * magnitude + TINY[dt]
    finite = np.isfinite(exact)
    if dt == torch.float16:  # beyond the largest half: the type's infinity
        finite &= np.abs(exact) < 65504
    bad = finite & ~(np.abs(g - exact) <= room)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[:3].tolist()}: "
                           f"{g[bad][:3]} for {exact[bad][:3]}, room {room[bad][:3]}")
    nan = np.isnan(exact)
    assert np.isnan(g[nan]).all(), f"{what}: NaN expected"


def _d(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _norm(v, va, kind, w, b, eps, stats=None):
    """N(v), its magnitude, mean, rstd; va is the magnitude of v's own terms"""
    T, H = v.shape
    if kind == "none":
        return v, va, np.zeros(T), np.ones(T)
    if stats is None:
        mean = v.mean(1) if kind == "layer" else np.zeros(T)
        rstd = 1 / np.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)
    else:
        mean, rstd = stats
    spread = va + (va.mean(1) if kind == "layer" else np.zeros(T))[:, None]
    w1 = np.ones(H) if w is None else w
    b1 = np.zeros(H) if b is None else b
    hat = (v - mean[:, None]) * rstd[:, None]
    return hat * w1 + b1, spread * rstd[:, None] * np.abs(w1) + np.abs(b1), mean, rstd


def norm_forward(h, y, post, w_post, b_post, gate, scale, pre, w_pre, b_pre, eps):
    """{name: (exact, magnitude)} of echo_norm's outputs"""
    h, w_post, b_post, w_pre, b_pre, g = map(_d, (h, w_post, b_post, w_pre, b_pre, gate))
    T, H = h.shape
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    m1, r1 = np.zeros(T), np.ones(T)
    h2, a2 = h, np.abs(h)
    if y is not None:
        y = _d(y)
        u, ua, m1, r1 = _norm(y, np.abs(y), post, w_post, b_post, eps)
        if g is not None:
            rows = np.arange(T) // (T // g.shape[0]) if T else np.zeros(0, int)
            u, ua = u * g[rows], ua * np.abs(g[rows])
        h2, a2 = h + scale * u, np.abs(h) + abs(scale) * ua
    z, za, m2, r2 = _norm(h2, a2, pre, w_pre, b_pre, eps)
    stats = np.stack([m1, r1, m2, r2])
    ya = np.abs(y).mean(1) if y is not None and H else np.zeros(T)
    # a mean's terms are the row's; a reciprocal deviation's relative error is the row's spread's
    rel = lambda v, va, r: r * np.maximum(1, (va ** 2).mean(1) * r * r)  # noqa: E731
    sa = np.stack([ya, r1 if y is None else rel(y, np.abs(y), r1), a2.mean(1), rel(h2, a2, r2)])
    return {"h_out": (h2, a2), "z": (z, za), "stats": (stats, sa)}


def _norm_back(d, da, v, kind, w, mean, rstd):
    """gradient of v for the gradient d of N(v), with magnitudes; and the
    normalized row with its own"""
    H = v.shape[1]
    if kind == "none":
        return d, da, v, np.abs(v)
    w1 = np.ones(H) if w is None else w
    hat = (v - mean[:, None]) * rstd[:, None]
    hata = (np.abs(v) + np.abs(mean)[:, None]) * rstd[:, None]
    g, ga = d * w1, da * np.abs(w1)
    s, sa = g - hat * (g * hat).mean(1, keepdims=True), ga + hata * (ga * hata).mean(1, keepdims=True)
    if kind == "layer":
        s, sa = s - g.mean(1, keepdims=True), sa + ga.mean(1, keepdims=True)
    return s * rstd[:, None], sa * rstd[:, None], hat, hata


def norm_backward(dz, dh_out, h_out, y, stats, post, w_post, b_post, gate, scale, pre, w_pre):
    """{name: (exact, magnitude)} of echo_norm_backward's outputs"""
    dz, dh_out, h_out, y, st, w_post, b_post, w_pre, g = map(
        _d, (dz, dh_out, h_out, y, stats, w_post, b_post, w_pre, gate))
    some = next(t for t in (dz, dh_out, y) if t is not None)
    T, H = some.shape
    scale = float(np.float32(scale))
    dh = np.zeros((T, H)) if dh_out is None else dh_out
    dha, out = np.abs(dh), {}
    if pre != "none":
        back, ba, hat, hata = _norm_back(dz, np.abs(dz), h_out, pre, w_pre, st[2], st[3])
        dh, dha = dh + back, dha + ba
        out["dw_pre"] = ((dz * hat).sum(0), (np.abs(dz) * hata).sum(0))
        out["db_pre"] = (dz.sum(0), np.abs(dz).sum(0))
    out["dh"] = (dh, dha)
    du, dua = scale * dh, abs(scale) * dha
    if y is None:
        out["dy"] = (du, dua)
        return out
    if g is not None:
        u, ua, _, _ = _norm(y, np.abs(y), post, w_post, b_post, 0.0,
                            None if post == "none" else (st[0], st[1]))
        if post != "none":
            ua = ua + np.abs(st[0] * st[1])[:, None]
        G = g.shape[0]
        out["dgate"] = ((du * u).reshape(G, -1, H).sum(1), (dua * ua).reshape(G, -1, H).sum(1))
        rows = np.arange(T) // (T // G) if T else np.zeros(0, int)
        du, dua = du * g[rows], dua * np.abs(g[rows])
    dy, dya, hat, hata = _norm_back(du, dua, y, post, w_post, st[0] if st is not None else None,
                                    st[1] if st is not None else None)
    out["dy"] = (dy, dya)
    if post != "none":
        out["dw_post"] = ((du * hat).sum(0), (dua * hata).sum(0))
        out["db_post"] = (du.sum(0), dua.sum(0))
    return out


# ---- products ---------------------------------------------------------------------

def act(p, kind):
    """(value, slope) of an activation in binary64"""
    from scipy.special import erfc, expit
    if kind == "relu":
        return np.maximum(p, 0), (p > 0).astype(np.float64)
    if kind == "silu":
        s = expit(p)
        return p * s, s * (1 + p * expit(-p))
    if kind == "gelu":
        c = erfc(-p / np.sqrt(2)) / 2
        return p * c, c + p * np.exp(-p * p / 2) / np.sqrt(2 * np.pi)
    if kind == "gelu_tanh":
        a = np.sqrt(8 / np.pi) * (p + 0.044715 * p ** 3)
        s = expit(a)
        return p * s, s + p * s * expit(-a) * np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * p * p)
    return p, np.ones_like(p)


def linear_forward(x, w, bias, residual, kind, gated):
    """{name: (exact, magnitude)} of echo_linear's outputs.  An activation's
    value changes by at most 1.2 of what its argument changes by (the largest
    slope of the five is below 1.13)."""
    x, w, bias, residual = map(_d, (x, w, bias, residual))
    p, pa = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        p, pa = p + bias, pa + np.abs(bias)
    if gated:
        n = p.shape[1] // 2
        v, va = act(p[:, :n], kind)[0], 1.2 * pa[:, :n]
        out, oa = v * p[:, n:], va * np.abs(p[:, n:]) + np.abs(v) * pa[:, n:] + va * pa[:, n:] * EPS32
    else:
        out, oa = act(p, kind)[0], 1.2 * pa
    if residual is not None:
        out, oa = out + residual, oa + np.abs(residual)
    return {"out": (out, oa), "p": (p, pa)}


def linear_backward(dout, x, w, p, kind, gated):
    """{name: (exact, magnitude, magnitude rounded to the operands' type)}:
    the products read dp rounded once to the type, which adds its half unit of
    every term"""
    d, x, w, p = map(_d, (dout, x, w, p))
    if gated:
        n = d.shape[1]
        v, s = act(p[:, :n], kind)
        dp = np.concatenate([d * p[:, n:] * s, d * v], 1)
    else:
        dp = d if kind == "none" else d * act(p, kind)[1]
    da = np.abs(dp)
    if kind != "none" or gated:
        # what a slope or value is off by: 2^-17 of its exponentials' share, at
        # most 1.2 of it, as multiples of 2^-24
        reach = np.abs(d) if not gated else np.concatenate([np.abs(d * p[:, n:]), np.abs(d) * (1 + np.abs(p[:, :n]))], 1)
        da = da + 8 * reach
    return {"dx": (dp @ w, da @ np.abs(w), np.abs(dp) @ np.abs(w)),
            "dw": (dp.T @ x, da.T @ np.abs(x), np.abs(dp).T @ np.abs(x)),
            "dbias": (dp.sum(0), da.sum(0))}
