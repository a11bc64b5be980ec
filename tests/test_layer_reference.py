"""The binary64 references of the layer operators against differences and
torch's automatic derivatives (CPU only)."""
import numpy as np
import pytest
import torch

import layer_reference as R


def _leaf(gen, *shape, at=0.0, spread=1.0):
    return (at + spread * torch.randn(*shape, generator=gen, dtype=torch.float64)).requires_grad_(True)


@pytest.mark.parametrize("groups", [0, 1, 3, 6])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_norm_gradients_follow_the_forward_formula(post, pre, groups):
    gen = torch.Generator().manual_seed(11)
    T, H, scale, eps = 6, 9, 0.75, 2.0 ** -10
    h, y = _leaf(gen, T, H), _leaf(gen, T, H, at=0.3)
    vec = lambda kind: (_leaf(gen, H, at=1.0, spread=0.2), _leaf(gen, H)) if kind != "none" else (None, None)  # noqa: E731
    (w1, b1), (w2, b2) = vec(post), vec(pre)
    gate = _leaf(gen, groups, H) if groups else None
    dz = torch.randn(T, H, generator=gen, dtype=torch.float64) if pre != "none" else None
    dh_out = torch.randn(T, H, generator=gen, dtype=torch.float64)

    def norm(v, kind, w, b):
        if kind == "none":
            return v
        m = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        return (v - m) / torch.sqrt(((v - m) ** 2).mean(1, keepdim=True) + eps) * w + b

    def objective(h, y, w1, b1, w2, b2, gate):
        u = norm(y, post, w1, b1)
        if gate is not None:
            u = u * gate.repeat_interleave(T // groups, 0)
        h2 = h + scale * u
        s = (h2 * dh_out).sum()
        return s if pre == "none" else s + (norm(h2, pre, w2, b2) * dz).sum()

    leaves = {"dh": h, "dy": y, "dw_post": w1, "db_post": b1, "dw_pre": w2, "db_pre": b2, "dgate": gate}
    objective(h, y, w1, b1, w2, b2, gate).backward()
    f = R.norm_forward(h, y, post, w1, b1, gate, scale, pre, w2, b2, eps)
    stats = torch.from_numpy(f["stats"][0])
    got = R.norm_backward(dz, dh_out, torch.from_numpy(f["h_out"][0]), y, stats, post, w1, b1, gate, scale,
                          pre, w2)
    rng = np.random.default_rng(5)
    for name, leaf in leaves.items():
        if leaf is None:
            continue
        exact, magnitude = got[name]
        assert np.allclose(exact, leaf.grad.numpy(), rtol=1e-10, atol=1e-12), name
        assert (np.abs(exact) <= magnitude * (1 + 1e-9) + 1e-300).all(), name
        # a central difference along one random direction
        way = torch.from_numpy(rng.standard_normal(tuple(leaf.shape)))
        step = 1e-6
        at = {k: (v.detach() if v is not None else None) for k, v in leaves.items()}
        args = lambda s: [at[k] + s * way if k == name else at[k] for k in  # noqa: E731
                          ("dh", "dy", "dw_post", "db_post", "dw_pre", "db_pre", "dgate")]
        diff = float(objective(*args(step)) - objective(*args(-step))) / (2 * step)
        along = float((exact * way.numpy()).sum())
        assert abs(diff - along) <= 1e-7 * max(1.0, abs(along)), (name, diff, along)


def test_the_bound_is_tight_enough_to_see_a_wrong_value():
    got = torch.tensor([1.0, 2.0, 3.0])
    R.close(got, [1.0, 2.0, 3.0], [1.0, 2.0, 3.0], 4, "same")
    with pytest.raises(AssertionError):
        R.close(got, [1.0, 2.0, 3.0 + 3e-6], [1.0, 2.0, 3.0], 4, "off by 1e-6")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_gradients_follow_the_forward_formula(kind, gated):
    gen = torch.Generator().manual_seed(21)
    m, n, k = 5, 4, 7
    rows = 2 * n if gated else n
    x, w, bias = _leaf(gen, m, k), _leaf(gen, rows, k), _leaf(gen, rows)
    residual = torch.randn(m, n, generator=gen, dtype=torch.float64)
    dout = torch.randn(m, n, generator=gen, dtype=torch.float64)
    f = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu}[kind]
    p = x @ w.T + bias
    out = (f(p[:, :n]) * p[:, n:] if gated else f(p)) + residual
    got = R.linear_forward(x, w, bias, residual, kind, gated)
    assert np.allclose(got["out"][0], out.detach().numpy(), rtol=1e-12, atol=1e-13)
    (out * dout).sum().backward()
    back = R.linear_backward(dout, x, w, p, kind, gated)
    for name, leaf in (("dx", x), ("dw", w), ("dbias", bias)):
        assert np.allclose(back[name][0], leaf.grad.numpy(), rtol=1e-10, atol=1e-12), name
    # a central difference along one direction of x, of w and of bias
    rng = np.random.default_rng(8)
    for name in ("dx", "dw", "dbias"):
        at = {"dx": x.detach().numpy(), "dw": w.detach().numpy(), "dbias": bias.detach().numpy()}
        way, step = rng.standard_normal(at[name].shape), 1e-6

        def objective(s):
            v = {q: torch.from_numpy(a + s * way if q == name else a) for q, a in at.items()}
            o = R.linear_forward(v["dx"], v["dw"], v["dbias"], residual, kind, gated)["out"][0]
            return float((o * dout.numpy()).sum())

        diff, along = (objective(step) - objective(-step)) / (2 * step), float((back[name][0] * way).sum())
        assert abs(diff - along) <= 1e-6 * max(1.0, abs(along)), (name, diff, along)
