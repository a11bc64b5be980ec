"""The layer operators beside the all-reduce, as they are timed and compared.

Two operators, forward and backward, stand on both sides of a tensor-parallel
all-reduce: the norms before and after a block with its gate and residual
scale (echo_norm, echo_norm_backward), and the matrix product with bias,
activation and residual in its epilogue (echo_linear, echo_linear_backward).

Where `own` is false `run` computes them in their plain form, in binary32 and
rounded once at the end; where it is true, with the library's calls.

A case's fields
  norms      tokens, hidden, dtype ("bf16", "f16", "f32"), stream (type of the
             residual stream: dtype or "f32"), post / pre ("none", "rms",
             "layer"), groups (rows of the gate, 0: no gate; token t uses row
             t // (tokens / groups)), scale, eps, train (statistics kept)
  products   m rows, n outputs, k inputs, dtype, act, gated, bias, residual,
             train (the product before the activation is kept)
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _norm(name, op, tokens, hidden, dtype="bf16", stream="bf16", post="none", pre="rms", groups=0,
          scale=1.0, eps=1e-6, train=False):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "dtype": dtype, "stream": stream,
            "post": post, "pre": pre, "groups": groups, "scale": scale, "eps": eps, "train": train}


def _linear(name, op, m, n, k, dtype="bf16", act="none", gated=False, bias=False, residual=False,
            train=False):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "train": train}


def listed():
    return [
        # serving one sequence: the residual add and pre-norm of a single token
        _norm("norm_token", "norm", 1, 4096),
        # a decode step of 256 sequences at hidden 4096, sandwich norms, binary32 stream, gate per channel
        _norm("norm_decode", "norm", 256, 4096, stream="f32", post="rms", groups=1, scale=0.5),
        # a prefill of 8192 tokens at hidden 4096
        _norm("norm_prefill", "norm", 8192, 4096, train=True),
        # the training site of 8 x 4096 tokens at hidden 1024, backward
        _norm("norm_train_grad", "norm_grad", 32768, 1024, train=True),
        # layer norms on both sides, one gate row for each of 8 sequences, an odd hidden size, backward
        _norm("norm_odd_grad", "norm_grad", 8 * 509, 2051, dtype="f16", stream="f32", post="layer",
              pre="layer", groups=8, scale=0.7, eps=1e-5, train=True),
        # serving one sequence: the gated up-projection of one token, one rank of eight
        _linear("linear_token", "linear", 1, 1792, 4096, act="silu", gated=True),
        # a decode step of 256 sequences: the down-projection of one rank with its residual
        _linear("linear_decode", "linear", 256, 4096, 1792, residual=True),
        # a prefill of 8192 tokens: the gated up-projection of one rank
        _linear("linear_prefill", "linear", 8192, 1792, 4096, act="silu", gated=True),
        # the product that follows a 1 GB all-reduce: 131072 tokens
        _linear("linear_large", "linear", 131072, 1792, 4096),
        # rows, columns and inputs that are no multiple of anything
        _linear("linear_odd", "linear", 1237, 777, 1001, dtype="f16", act="gelu", bias=True,
                residual=True, train=True),
        # the training site of 8 x 4096 tokens at hidden 1024: one rank's gated projection, backward
        _linear("linear_train_grad", "linear_grad", 32768, 384, 1024, act="silu", gated=True, train=True),
        # a projection with bias and GELU over 8192 tokens, backward
        _linear("linear_gelu_grad", "linear_grad", 8192, 1792, 4096, dtype="f16", act="gelu_tanh", bias=True,
                train=True),
    ]


def _spread(rng, lo, hi):
    """a whole number whose logarithm is spread evenly over [lo, hi]"""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """a feature size: mostly a multiple of 64 or of 8, at times anything"""
    n = _spread(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    if rng.random() < 0.45:
        grad = rng.random() < 0.5
        hidden = _size(rng, 64, 8192)
        tokens = _spread(rng, 1, min(32768, (8192 * 4096) // hidden))
        groups = rng.choice((0, 0, 1, 2))
        if groups == 2:  # a few sequences with a gate row each
            groups = rng.choice((2, 3, 8))
            tokens = max(1, tokens // groups) * groups
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        return _norm("", "norm_grad" if grad else "norm", tokens, hidden, dtype=dtype,
                     stream=rng.choice((dtype, "f32")), post=rng.choice(("none", "rms", "layer")),
                     pre=rng.choice(("rms", "layer")), groups=groups, scale=rng.choice((1.0, 0.5, 0.2)),
                     eps=rng.choice((1e-6, 1e-5)), train=grad or rng.random() < 0.5)
    grad = rng.random() < 0.4
    n, k = _size(rng, 32, 8192), _size(rng, 32, 8192)
    gated = rng.random() < 0.4
    act = rng.choice(("silu", "gelu", "gelu_tanh")) if gated else \
        rng.choice(("none", "none", "relu", "gelu", "gelu_tanh", "silu"))
    most = 131072 * 1792 * 4096 // (n * k * (2 if gated else 1) * (2 if grad else 1))
    room = (1 << 29) // (n * (3 if gated else 2) + k)  # rows whose tensors stay within the largest case's
    m = _spread(rng, 1, max(1, min(131072, most, room)))
    return _linear("", "linear_grad" if grad else "linear", m, n, k, dtype=rng.choice(("bf16", "f16")),
                   act=act, gated=gated, bias=rng.random() < 0.4, residual=not grad and rng.random() < 0.4,
                   train=grad or rng.random() < 0.3)


# ---- inputs -------------------------------------------------------------------

def _hidden_states(gen, rows, cols, spread=1.0, peak=20.0):
    """activations with a scale per channel and one channel in a thousand far larger"""
    v = torch.randn(rows, cols, generator=gen, device=DEV)
    c = torch.exp(torch.randn(cols, generator=gen, device=DEV) * 0.5) * spread
    c = torch.where(torch.rand(cols, generator=gen, device=DEV) < 0.001, c * peak, c)
    return v * c


def _gradients(gen, rows, cols):
    """heavy-tailed gradients of order 1e-3 (a normal over the root of a mean of three squares, cut at 64)"""
    z = torch.randn(rows, cols, generator=gen, device=DEV)
    s = torch.zeros_like(z)
    for _ in range(3):
        s += torch.randn(rows, cols, generator=gen, device=DEV).square()
    return torch.clamp(z / torch.sqrt(s / 3), -64, 64) * 1e-3


def _norm_inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    T, H, G = case["tokens"], case["hidden"], case["groups"]
    t, ts = TYPES[case["dtype"]], TYPES[case["stream"]]
    vec = lambda c, s: (c + s * torch.randn(H, generator=gen, device=DEV)).to(t)  # noqa: E731
    i = {"h": _hidden_states(gen, T, H).to(ts), "y": _hidden_states(gen, T, H, 0.5).to(t)}
    i["w_post"] = vec(1.0, 0.1) if case["post"] != "none" else None
    i["b_post"] = vec(0.0, 0.1) if case["post"] == "layer" else None
    i["w_pre"] = vec(1.0, 0.1) if case["pre"] != "none" else None
    i["b_pre"] = vec(0.0, 0.1) if case["pre"] == "layer" else None
    i["gate"] = (0.5 + 0.3 * torch.randn(G, H, generator=gen, device=DEV)).to(t) if G else None
    if case["op"] == "norm_grad":
        h_out, _, stats = _norm_plain(case, i, keep=True)
        i["h_out"], i["stats"] = h_out, stats
        i["dz"] = _gradients(gen, T, H).to(t)
        i["dh_out"] = _gradients(gen, T, H).to(ts)
        del i["h"]
    return i


def _linear_inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["dtype"]]
    rows = 2 * n if case["gated"] else n
    i = {"x": _hidden_states(gen, m, k, peak=8.0).to(t)}
    i["w"] = (torch.randn(rows, k, generator=gen, device=DEV) / math.sqrt(k)).to(t)
    i["bias"] = (0.2 * torch.randn(rows, generator=gen, device=DEV)).to(t) if case["bias"] else None
    i["residual"] = torch.randn(m, n, generator=gen, device=DEV).to(t) if case["residual"] else None
    if case["op"] == "linear_grad":
        i["p"] = None
        if case["act"] != "none" or case["gated"]:
            p = i["x"].float() @ i["w"].float().t()
            i["p"] = (p if i["bias"] is None else p + i["bias"].float()).to(t)
        i["dout"] = _gradients(gen, m, n).to(t)
    return i


def prepare(case, seed):
    i = (_norm_inputs if case["op"].startswith("norm") else _linear_inputs)(case, seed)
    state = {"case": case, "in": i}
    if own:
        state["call"] = (_norm_buffers if case["op"].startswith("norm") else _linear_buffers)(case, i)
    return state


# ---- the plain form: binary32, rounded once at the end --------------------------

def _f(v):
    return None if v is None else v.float()


def _plain_norm_of(v, kind, w, b, eps):
    """(normed rows, mean, reciprocal deviation)"""
    if kind == "none":
        return v, None, None
    mean = v.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    rstd = 1.0 / torch.sqrt(c.square().mean(dim=1, keepdim=True) + eps)
    out = c * rstd * w
    return (out if b is None else out + b), mean[:, 0], rstd[:, 0]


def _rows(gate, tokens):
    """the gate's row of each token"""
    return gate.repeat_interleave(tokens // gate.shape[0], dim=0)


def _norm_plain(case, i, keep):
    h, y = _f(i["h"]), _f(i["y"])
    T = case["tokens"]
    u, m1, r1 = _plain_norm_of(y, case["post"], _f(i["w_post"]), _f(i["b_post"]), case["eps"])
    if i["gate"] is not None:
        u = u * _rows(_f(i["gate"]), T)
    h2 = h + case["scale"] * u
    z, m2, r2 = _plain_norm_of(h2, case["pre"], _f(i["w_pre"]), _f(i["b_pre"]), case["eps"])
    stats = None
    if keep:
        zero, one = torch.zeros(T, device=h.device), torch.ones(T, device=h.device)
        stats = torch.stack([zero if m1 is None else m1, one if r1 is None else r1,
                             zero if m2 is None else m2, one if r2 is None else r2])
    return h2.to(TYPES[case["stream"]]), z.to(TYPES[case["dtype"]]), stats


def _plain_norm_grad_of(d, v, kind, w, mean, rstd):
    """(gradient of v, of the weight, of the bias) for the gradient d of the normed rows"""
    if kind == "none":
        return d, None, None
    hat = (v - mean[:, None]) * rstd[:, None]
    g = d * w
    s = g - hat * (g * hat).mean(dim=1, keepdim=True)
    if kind == "layer":
        s = s - g.mean(dim=1, keepdim=True)
    return s * rstd[:, None], (d * hat).sum(dim=0), d.sum(dim=0)


def _norm_grad_plain(case, i):
    t, ts, T = TYPES[case["dtype"]], TYPES[case["stream"]], case["tokens"]
    st, y, h2, gate = i["stats"], _f(i["y"]), _f(i["h_out"]), _f(i["gate"])
    back, dw2, db2 = _plain_norm_grad_of(_f(i["dz"]), h2, case["pre"], _f(i["w_pre"]), st[2], st[3])
    dh = _f(i["dh_out"]) + back
    du, dgate = case["scale"] * dh, None
    if gate is not None:
        u = y if case["post"] == "none" else (y - st[0][:, None]) * st[1][:, None] * _f(i["w_post"])
        if i["b_post"] is not None:
            u = u + _f(i["b_post"])
        dgate = (du * u).view(gate.shape[0], -1, case["hidden"]).sum(dim=1)
        du = du * _rows(gate, T)
    dy, dw1, db1 = _plain_norm_grad_of(du, y, case["post"], _f(i["w_post"]), st[0], st[1])
    out = {"dh": dh.to(ts), "dy": dy.to(t), "dgate": dgate, "dw_post": dw1, "dw_pre": dw2,
           "db_post": db1 if case["post"] == "layer" else None,
           "db_pre": db2 if case["pre"] == "layer" else None}
    return {n: (v if n in ("dh", "dy") else v.to(t)) for n, v in out.items() if v is not None}


def _plain_act(p, act):
    if act == "relu":
        return torch.where(p > 0, p, torch.zeros_like(p))
    if act == "silu":
        return p / (1 + torch.exp(-p))
    if act == "gelu":
        return 0.5 * p * (1 + torch.erf(p * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * p * (1 + torch.tanh(math.sqrt(2 / math.pi) * (p + 0.044715 * p * p * p)))
    return p


def _plain_act_slope(p, act):
    if act == "relu":
        return (p > 0).to(p.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-p))
        return s * (1 + p * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(p * math.sqrt(0.5))) + p * torch.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (p + 0.044715 * p * p * p))
        return 0.5 * (1 + th) + 0.5 * p * (1 - th * th) * c * (1 + 3 * 0.044715 * p * p)
    return torch.ones_like(p)


def _linear_plain(case, i):
    t, n = TYPES[case["dtype"]], case["n"]
    p = _f(i["x"]) @ _f(i["w"]).t()
    if i["bias"] is not None:
        p = p + _f(i["bias"])
    if case["gated"]:
        out = _plain_act(p[:, :n], case["act"]) * p[:, n:]
    else:
        out = _plain_act(p, case["act"])
    if i["residual"] is not None:
        out = out + _f(i["residual"])
    return {"out": out.to(t), "p": p.to(t)} if case["train"] else {"out": out.to(t)}


def _linear_grad_plain(case, i):
    t, n, d = TYPES[case["dtype"]], case["n"], _f(i["dout"])
    if case["gated"]:
        p = _f(i["p"])
        d = torch.cat([d * p[:, n:] * _plain_act_slope(p[:, :n], case["act"]),
                       d * _plain_act(p[:, :n], case["act"])], dim=1)
    elif case["act"] != "none":
        d = d * _plain_act_slope(_f(i["p"]), case["act"])
    out = {"dx": (d @ _f(i["w"])).to(t), "dw": (d.t() @ _f(i["x"])).to(t)}
    if case["bias"]:
        out["dbias"] = d.sum(dim=0).to(t)
    return out


# ---- the library's calls --------------------------------------------------------

def _like(v):
    return None if v is None else torch.empty_like(v)


def _norm_buffers(case, i):
    from error_compensated_bit_echo_amd import binding as echo

    T, H, t, ts = case["tokens"], case["hidden"], TYPES[case["dtype"]], TYPES[case["stream"]]
    new = lambda dt: torch.empty(T, H, dtype=dt, device=DEV)  # noqa: E731
    if case["op"] == "norm":
        return {"h_out": new(ts), "z": new(t),
                "stats": torch.empty(4, T, device=DEV) if case["train"] else None}
    size = echo.echo_norm_backward_workspace(T, H, case["groups"])
    return {"dh": new(ts), "dy": new(t), "dgate": _like(i["gate"]), "dw_post": _like(i["w_post"]),
            "db_post": _like(i["b_post"]), "dw_pre": _like(i["w_pre"]), "db_pre": _like(i["b_pre"]),
            "workspace": torch.empty(size, dtype=torch.uint8, device=DEV)}


def _linear_buffers(case, i):
    from error_compensated_bit_echo_amd import binding as echo

    m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["dtype"]]
    if case["op"] == "linear":
        size = echo.echo_linear_workspace(m, n, k, gated=case["gated"])
        b = {"out": torch.empty(m, n, dtype=t, device=DEV)}
        b["p"] = torch.empty(m, i["w"].shape[0], dtype=t, device=DEV) if case["train"] else None
    else:
        size = echo.echo_linear_backward_workspace(m, n, k, act=case["act"], gated=case["gated"])
        b = {"dx": _like(i["x"]), "dw": _like(i["w"]), "dbias": _like(i["bias"])}
    b["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return b


def _own(state):
    from error_compensated_bit_echo_amd import binding as echo

    case, i, b = state["case"], state["in"], state["call"]
    if case["op"] == "norm":
        echo.echo_norm(i["h"], i["y"], b["h_out"], b["z"], post=case["post"], w_post=i["w_post"],
                       b_post=i["b_post"], gate=i["gate"], scale=case["scale"], pre=case["pre"],
                       w_pre=i["w_pre"], b_pre=i["b_pre"], eps=case["eps"], stats=b["stats"])
    elif case["op"] == "norm_grad":
        echo.echo_norm_backward(i["dz"], i["dh_out"], i["h_out"], i["y"], i["stats"], b["dh"], b["dy"],
                                post=case["post"], w_post=i["w_post"], b_post=i["b_post"], gate=i["gate"],
                                scale=case["scale"], pre=case["pre"], w_pre=i["w_pre"],
                                dw_post=b["dw_post"], db_post=b["db_post"], dgate=b["dgate"],
                                dw_pre=b["dw_pre"], db_pre=b["db_pre"], workspace=b["workspace"])
    elif case["op"] == "linear":
        echo.echo_linear(i["x"], i["w"], b["out"], bias=i["bias"], residual=i["residual"], act=case["act"],
                         gated=case["gated"], p=b["p"], workspace=b["workspace"])
    else:
        echo.echo_linear_backward(i["dout"], i["x"], i["w"], i["p"], b["dx"], b["dw"], dbias=b["dbias"],
                                  act=case["act"], gated=case["gated"], workspace=b["workspace"])
    return {n: v for n, v in b.items() if v is not None and n != "workspace"}


def run(state):
    if own:
        return _own(state)
    case, i = state["case"], state["in"]
    if case["op"] == "norm":
        h_out, z, stats = _norm_plain(case, i, case["train"])
        return {"h_out": h_out, "z": z, "stats": stats} if case["train"] else {"h_out": h_out, "z": z}
    return {"norm_grad": _norm_grad_plain, "linear": _linear_plain,
            "linear_grad": _linear_grad_plain}[case["op"]](case, i)


# ---- work -------------------------------------------------------------------------

def work(case):
    if case["op"].startswith("norm"):
        e, s = TYPES[case["dtype"]].itemsize, TYPES[case["stream"]].itemsize
        TH, H, G = case["tokens"] * case["hidden"], case["hidden"], case["groups"]
        vectors = sum({"none": 0, "rms": 1, "layer": 2}[case[p]] for p in ("post", "pre")) + G
        stats = 16 * case["tokens"] if case["train"] else 0
        if case["op"] == "norm":  # y, h in; h', z out
            return {"bytes": TH * (2 * e + 2 * s) + vectors * H * e + stats, "flops": 12 * TH}
        # dz, dh', h', y in; dh, dy out
        return {"bytes": TH * (3 * e + 3 * s) + 2 * vectors * H * e + stats, "flops": 30 * TH}
    m, n, k = case["m"], case["n"], case["k"]
    rows = 2 * n if case["gated"] else n
    kept = m * rows if case["act"] != "none" or case["gated"] else 0
    extra = rows if case["bias"] else 0
    if case["op"] == "linear":
        extra += (m * n if case["residual"] else 0) + (m * rows if case["train"] else 0)
        return {"bytes": 2 * (m * k + rows * k + m * n + extra), "flops": 2 * m * rows * k}
    return {"bytes": 2 * (2 * m * k + 2 * rows * k + m * n + kept + extra), "flops": 4 * m * rows * k}


# ---- the definition in 64 bits -------------------------------------------------------

def _exact_moments(v, kind, eps):
    """mean and reciprocal deviation of each row of a binary64 matrix"""
    T = v.shape[0]
    if kind == "none":
        return v.new_zeros(T), v.new_ones(T)
    mean = v.sum(1) / v.shape[1] if kind == "layer" else v.new_zeros(T)
    return mean, (((v - mean[:, None]) ** 2).sum(1) / v.shape[1] + eps) ** -0.5


def _exact_norm(case, i):
    d = {n: (None if v is None else v.double()) for n, v in i.items()}
    T, H = d["h"].shape
    m1, r1 = _exact_moments(d["y"], case["post"], case["eps"])
    u = (d["y"] - m1[:, None]) * r1[:, None]
    if d["w_post"] is not None:
        u *= d["w_post"]
    if d["b_post"] is not None:
        u += d["b_post"]
    if d["gate"] is not None:
        G = d["gate"].shape[0]
        u = (u.view(G, T // G, H) * d["gate"].view(G, 1, H)).view(T, H)
    h2 = d["h"] + u * case["scale"]
    m2, r2 = _exact_moments(h2, case["pre"], case["eps"])
    z = (h2 - m2[:, None]) * r2[:, None]
    if d["w_pre"] is not None:
        z *= d["w_pre"]
    if d["b_pre"] is not None:
        z += d["b_pre"]
    if not case["train"]:
        return {"h_out": h2, "z": z}
    return {"h_out": h2, "z": z, "stats": torch.stack([m1, r1, m2, r2])}


def _exact_norm_back(g, hat, r, kind, w):
    """gradient of a norm's input from the gradient g of its output: the
    Jacobian of row v is rstd (I - [1 1^T] / H - hat hat^T / H) diag(w)"""
    if kind == "none":
        return g
    H = g.shape[1]
    gw = g * w
    along = (gw * hat).sum(1) / H
    flat = gw.sum(1) / H if kind == "layer" else 0 * along
    return (gw - flat[:, None] - hat * along[:, None]) * r[:, None]


def _exact_norm_grad(case, i):
    d = {n: (None if v is None else v.double()) for n, v in i.items()}
    T, H = d["y"].shape
    m1, r1, m2, r2 = d["stats"]
    hat1 = (d["y"] - m1[:, None]) * r1[:, None]
    hat2 = (d["h_out"] - m2[:, None]) * r2[:, None]
    out = {"dh": d["dh_out"] + _exact_norm_back(d["dz"], hat2, r2, case["pre"], d["w_pre"])}
    du = out["dh"] * case["scale"]
    if d["gate"] is not None:
        G = d["gate"].shape[0]
        u = hat1 if d["w_post"] is None else hat1 * d["w_post"]
        u = u if d["b_post"] is None else u + d["b_post"]
        out["dgate"] = torch.stack([(a * b).sum(0) for a, b in zip(du.chunk(G), u.chunk(G))])
        du = (du.view(G, T // G, H) * d["gate"].view(G, 1, H)).view(T, H)
    out["dy"] = _exact_norm_back(du, hat1, r1, case["post"], d["w_post"])
    if case["post"] != "none":
        out["dw_post"] = (du * hat1).sum(0)
    if case["post"] == "layer":
        out["db_post"] = du.sum(0)
    if case["pre"] != "none":
        out["dw_pre"] = (d["dz"] * hat2).sum(0)
    if case["pre"] == "layer":
        out["db_pre"] = d["dz"].sum(0)
    return out


def _exact_act(p, act):
    """activation and slope in binary64"""
    if act == "relu":
        return p.clamp(min=0), torch.sign(p).clamp(min=0)
    if act == "silu":
        s = torch.sigmoid(p)
        return p * s, s + p * s * torch.sigmoid(-p)
    if act == "gelu":
        cdf = torch.erfc(-p / 2 ** 0.5) / 2
        return p * cdf, cdf + p * torch.exp(-p * p / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":  # (1 + tanh a) / 2 = sigmoid(2 a)
        a = (8 / math.pi) ** 0.5 * (p + 0.044715 * p ** 3)
        s = torch.sigmoid(a)
        return p * s, s + p * s * torch.sigmoid(-a) * (8 / math.pi) ** 0.5 * (1 + 0.134145 * p ** 2)
    return p, torch.ones_like(p)


def _exact_linear(case, i):
    p = torch.mm(i["x"].double(), i["w"].double().T)
    if i["bias"] is not None:
        p += i["bias"].double()
    if case["gated"]:
        a, b = p.chunk(2, dim=1)
        out = _exact_act(a, case["act"])[0] * b
    else:
        out = _exact_act(p, case["act"])[0]
    if i["residual"] is not None:
        out = out + i["residual"].double()
    return {"out": out, "p": p} if case["train"] else {"out": out}


def _exact_linear_grad(case, i):
    g = i["dout"].double()
    if case["gated"]:
        a, b = i["p"].double().chunk(2, dim=1)
        value, slope = _exact_act(a, case["act"])
        g = torch.hstack([g * b * slope, g * value])
    elif case["act"] != "none":
        g = g * _exact_act(i["p"].double(), case["act"])[1]
    out = {"dx": torch.mm(g, i["w"].double()), "dw": torch.mm(g.T, i["x"].double())}
    if case["bias"]:
        out["dbias"] = g.sum(0)
    return out


def exact(case, seed):
    if case["op"].startswith("norm"):
        i = _norm_inputs(case, seed)
        return _exact_norm(case, i) if case["op"] == "norm" else _exact_norm_grad(case, i)
    i = _linear_inputs(case, seed)
    return _exact_linear(case, i) if case["op"] == "linear" else _exact_linear_grad(case, i)
