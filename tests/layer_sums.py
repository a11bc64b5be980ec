"""What a product's or a sum's error may be as a whole: a check beside the bound of
every element, which grows with the length of the sum and so lets a lost row pass.

An output of one rounding is off by at most u of itself, u half a unit of its type, so
a row or column of outputs differs from the exact one by at most u of its norm.  Each
further rounding that all terms of a sum carry (dp's to the operands' type) adds a
random walk of at most u of the result.  binary32 accumulation and exponentials are
far below the 2^-12 that is added for them.  One row of m lost from a sum over m
independent terms changes its norm by about 1 / sqrt(m)."""
from __future__ import annotations

import torch

import layer_reference as R


def _far(got, exact, dim):
    err, size = (got - exact).square().sum(dim).sqrt(), exact.square().sum(dim).sqrt()
    return err / size.clamp(min=1e-300)


def near(got, exact, roundings, what, u=None):
    """every row and every column of got (its own type) to binary64, by the norm"""
    u = R.HALF_ULP[got.dtype] if u is None else u
    room = roundings * u + 2.0 ** -12
    g, e = got.double(), exact.to(got.device).reshape(got.shape)
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    for dim in range(g.dim()):
        # a short row has one element that may be close to 0
        if g.shape[dim] >= 16:
            far = _far(g, e, dim)
            assert float(far.max()) <= room, (f"{what}: summed over dimension {dim}, place {int(far.argmax())} is off by "
                                              f"{float(far.max()):.5f} of its norm, room {room:.5f}")


def elements(got, exact, magnitude, roundings, what):
    """the bound of layer_reference.close, where the tensors are"""
    dt = got.dtype
    g = got.double()
    room = R.HALF_ULP[dt] * exact.abs() + roundings * R.EPS32 * magnitude + R.TINY[dt]
    bad = ~((g - exact).abs() <= room)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[:3].tolist()}"


def act(p, kind):
    """(value, slope) of an activation, binary64 tensors"""
    if kind == "relu":
        return p.clamp(min=0), (p > 0).double()
    if kind == "silu":
        s = torch.sigmoid(p)
        return p * s, s * (1 + p * torch.sigmoid(-p))
    if kind == "gelu":
        c = torch.erfc(-p / 2 ** 0.5) / 2
        return p * c, c + p * torch.exp(-p * p / 2) / (2 * torch.pi) ** 0.5
    if kind == "gelu_tanh":
        a = (8 / torch.pi) ** 0.5 * (p + 0.044715 * p ** 3)
        s = torch.sigmoid(a)
        return p * s, s + p * s * torch.sigmoid(-a) * (8 / torch.pi) ** 0.5 * (1 + 3 * 0.044715 * p * p)
    return p, torch.ones_like(p)


def forward(x, w, bias, residual, kind, gated):
    """{name: (exact, magnitude)}, binary64, where the tensors are"""
    x, w = x.double(), w.double()
    p, pa = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        p, pa = p + bias.double(), pa + bias.double().abs()
    if gated:
        n = p.shape[1] // 2
        v = act(p[:, :n], kind)[0]
        out, oa = v * p[:, n:], 1.2 * pa[:, :n] * p[:, n:].abs() + v.abs() * pa[:, n:] + 1.2 * pa[:, :n] * pa[:, n:] * R.EPS32
    else:
        out, oa = act(p, kind)[0], 1.2 * pa
    if residual is not None:
        out, oa = out + residual.double(), oa + residual.double().abs()
    return {"out": (out, oa), "p": (p, pa)}


def backward(dout, x, w, p, kind, gated):
    """{name: exact}, binary64, where the tensors are"""
    d, x, w = dout.double(), x.double(), w.double()
    if gated:
        n = d.shape[1]
        v, s = act(p.double()[:, :n], kind)
        dp = torch.cat([d * p.double()[:, n:] * s, d * v], 1)
    else:
        dp = d if kind == "none" else d * act(p.double(), kind)[1]
    return {"dx": dp @ w, "dw": dp.T.contiguous() @ x, "dbias": dp.sum(0)}


def _norm_back(d, da, v, kind, w, mean, rstd):
    """gradient of v for the gradient d of N(v), with magnitudes; the normalized row
    with its own"""
    if kind == "none":
        return d, da, v, v.abs()
    hat = (v - mean[:, None]) * rstd[:, None]
    hata = (v.abs() + mean.abs()[:, None]) * rstd[:, None]
    g, ga = (d, da) if w is None else (d * w, da * w.abs())
    s, sa = g - hat * (g * hat).mean(1, keepdim=True), ga + hata * (ga * hata).mean(1, keepdim=True)
    if kind == "layer":
        s, sa = s - g.mean(1, keepdim=True), sa + ga.mean(1, keepdim=True)
    return s * rstd[:, None], sa * rstd[:, None], hat, hata


def norm_backward(dz, dh_out, h_out, y, stats, post, w_post, b_post, gate, scale, pre, w_pre):
    """{name: (exact, magnitude)} of echo_norm_backward's outputs, binary64, where the
    tensors are"""
    dz, dh_out, h_out, y, st, w_post, b_post, w_pre, g = (
        None if t is None else t.double() for t in (dz, dh_out, h_out, y, stats, w_post, b_post, w_pre, gate))
    T, H = next(t for t in (dz, dh_out, y) if t is not None).shape
    scale = float(torch.tensor(scale, dtype=torch.float32))
    dh = torch.zeros_like(dz) if dh_out is None else dh_out
    dha, out = dh.abs(), {}
    if pre != "none":
        back, ba, hat, hata = _norm_back(dz, dz.abs(), h_out, pre, w_pre, st[2], st[3])
        dh, dha = dh + back, dha + ba
        out["dw_pre"] = ((dz * hat).sum(0), (dz.abs() * hata).sum(0))
        out["db_pre"] = (dz.sum(0), dz.abs().sum(0))
    out["dh"] = (dh, dha)
    du, dua = scale * dh, abs(scale) * dha
    if g is not None:
        G = g.shape[0]
        if y is not None:
            u, ua = y, y.abs()
            if post != "none":
                u, ua = (y - st[0][:, None]) * st[1][:, None], (y.abs() + st[0].abs()[:, None]) * st[1][:, None]
                u, ua = (u, ua) if w_post is None else (u * w_post, ua * w_post.abs())
                u, ua = (u, ua) if b_post is None else (u + b_post, ua + b_post.abs())
            out["dgate"] = ((du * u).view(G, -1, H).sum(1), (dua * ua).view(G, -1, H).sum(1))
        of_row = torch.arange(T, device=g.device) // (T // G)
        du, dua = du * g[of_row], dua * g[of_row].abs()
    if post == "none":
        out["dy"] = (du, dua)
        return out
    dy, dya, hat, hata = _norm_back(du, dua, y, post, w_post, st[0], st[1])
    out["dy"] = (dy, dya)
    out["dw_post"] = ((du * hat).sum(0), (dua * hata).sum(0))
    out["db_post"] = (du.sum(0), dua.sum(0))
    return out
