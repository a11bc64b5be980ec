"""The check of whole sums sees a mistake that the bound of every element lets pass:
rows lost from a long sum, planted in the reference (CPU only)."""
import pytest
import torch

import layer_reference as R
import layer_sums as S


@pytest.mark.parametrize("kind,gated", [("none", False), ("gelu_tanh", False), ("silu", True)])
@pytest.mark.parametrize("lost", [1, 8])
def test_lost_rows_are_seen(kind, gated, lost):
    gen = torch.Generator().manual_seed(3)
    m, n, k = 6000, 136, 48
    rows = 2 * n if gated else n
    rand = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    x, w, p, dout = rand(m, k), rand(rows, k), rand(m, rows), rand(m, n)
    exact = S.backward(dout, x, w, p, kind, gated)
    # as the library rounds: dp to the type for the products, outputs once
    for name in ("dw", "dbias"):
        S.near(exact[name].to(torch.bfloat16), exact[name], 1, name)
    short = dout.clone()
    short[m - lost:] = 0
    wrong = S.backward(short, x, w, p, kind, gated)
    for name in ("dw", "dbias"):
        with pytest.raises(AssertionError, match="off by"):
            S.near(wrong[name].to(torch.bfloat16), exact[name], 1 if name == "dbias" else 2, name)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_the_formulas_are_those_of_the_reference(kind, gated):
    gen = torch.Generator().manual_seed(5)
    m, n, k = 20, 12, 9
    rows = 2 * n if gated else n
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, bias, residual, dout, p = rand(m, k), rand(rows, k), rand(rows), rand(m, n), rand(m, n), rand(m, rows)
    a, b = S.forward(x, w, bias, residual, kind, gated), R.linear_forward(x, w, bias, residual, kind, gated)
    for name in ("out", "p"):
        assert torch.allclose(a[name][0], torch.from_numpy(b[name][0]), rtol=1e-12, atol=1e-13), name
        assert torch.allclose(a[name][1], torch.from_numpy(b[name][1]), rtol=1e-6), name
    a, b = S.backward(dout, x, w, p, kind, gated), R.linear_backward(dout, x, w, p, kind, gated)
    for name in ("dx", "dw", "dbias"):
        assert torch.allclose(a[name], torch.from_numpy(b[name][0]), rtol=1e-12, atol=1e-12), name


@pytest.mark.parametrize("groups", [0, 1, 4])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_the_norms_formulas_are_those_of_the_reference(post, pre, groups):
    gen = torch.Generator().manual_seed(6)
    T, H = 8, 11
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    vec = lambda kind: (rand(H), rand(H) if kind == "layer" else None) if kind != "none" else (None, None)  # noqa: E731
    h, y, dz, dh_out = rand(T, H), rand(T, H) + 0.3, rand(T, H), rand(T, H)
    (w1, b1), (w2, b2) = vec(post), vec(pre)
    gate = rand(groups, H) if groups else None
    f = R.norm_forward(h, y, post, w1, b1, gate, 0.75, pre, w2, b2, 1e-5)
    h_out, stats = torch.from_numpy(f["h_out"][0]), torch.from_numpy(f["stats"][0])
    args = (dz if pre != "none" else None, dh_out, h_out, y, stats, post, w1, b1, gate, 0.75, pre, w2)
    a, b = S.norm_backward(*args), R.norm_backward(*args)
    assert set(a) == set(b)
    for name in a:
        assert torch.allclose(a[name][0], torch.from_numpy(b[name][0]), rtol=1e-11, atol=1e-12), name
        assert (a[name][1] <= torch.from_numpy(b[name][1]) * (1 + 1e-9)).all(), name
