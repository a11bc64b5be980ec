"""echo_linear8 over more steps than its rings hold, by every tile (bounds as in
test_gpu_linear8.py), with the first scale that is no power of two behind the ring's first
turn; rows of NaN behind x's and w's last and of NaN scales behind theirs; and subnormal codes,
whose cut the header states."""
import pytest
import torch

import fp8_reference as F
import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from linear8_ring_cases import CASES
from linear8_tile_cases import CASES as TILE_CASES
from test_gpu_linear8 import case, forward, space
from test_gpu_norm import DEV, on

pytestmark = pytest.mark.gpu


def late(c, gen, rows=None):
    """from the tenth block on a part of x's scales (of `rows`, or a fifth of all) and, if of all,
    of w's from the twelfth are no powers of two"""
    sx, sw = c["sx"], c["sw"]
    at = torch.rand(sx.shape, generator=gen) < 0.2 if rows is None else torch.zeros(sx.shape, dtype=torch.bool)
    if rows is not None:
        at[rows] = True
    at[:, :9] = False
    c["sx"] = torch.where(at, sx * (0.5 + torch.rand(sx.shape, generator=gen)), sx)
    if rows is None:
        sw[:, 11:] *= 0.5 + torch.rand(sw[:, 11:].shape, generator=gen)
    return c


@pytest.mark.parametrize("name", list(CASES))
def test_rings(name):
    m, n, k, act, gated, scales = CASES[name][:6]
    c = case(m, n, k, torch.float16 if "64" in name else torch.bfloat16, gated, "e5m2" if "others" in name else "e4m3",
             "any" if scales == "any" else "pow2")
    gen = torch.Generator().manual_seed(m + k)
    if scales in ("late", "one"):
        late(c, gen, None if scales == "late" else [m // 3])
    forward(c, act)


BEHIND = {name: TILE_CASES[name][:6] for name in ("256", "256 gated", "128", "128 gated", "64", "64 gated", "128 alone", "64 alone",
                                                  "64 alone gated", "128 split gated")}
BEHIND["few rows"], BEHIND["few rows gated"] = (11, 70, 1000, "none", False, "any"), (3, 70, 1000, "silu", True, "any")


@pytest.mark.parametrize("name", list(BEHIND))
def test_nan_behind_the_last_rows_has_no_influence(name):
    """a tile of rows behind x, w (gated, behind the up rows) and their scales: NaN, or zeros"""
    m, n, k, act, gated, scales = BEHIND[name]
    c = case(m, n, k, torch.bfloat16, gated, "e4m3", scales, bias=False, residual=False)
    rows = c["w"].shape[0]
    ws, got = space(B.echo_linear8_workspace(m, n, k, act=act, gated=gated)), []
    for code, scale in ((0x00, 1.0), (0x7F, float("nan"))):
        give = {}
        for q in ("x", "w"):
            r, pitch = c[q].shape[0], (k + 15) // 16 * 16
            codes = torch.full((r + 300, pitch), code, dtype=torch.uint8, device=DEV)
            codes[:r, :k] = c[q].view(torch.uint8)
            s = c["s" + q]
            all_scales = torch.full((s.shape[0] + 300, s.shape[1]), scale, device=DEV)
            all_scales[:s.shape[0]] = on(s)
            give[q], give["s" + q] = codes[:r, :k].view(c[q].dtype), all_scales[:s.shape[0]]
        out, p = (torch.empty(m, q, dtype=torch.bfloat16, device=DEV) for q in (n, rows))
        print(f"linear8 {name} with {scale} behind", flush=True)
        B.echo_linear8(give["x"], give["sx"], give["w"], give["sw"], out, act=act, gated=gated, p=p, workspace=ws)
        torch.cuda.synchronize()
        got.append((out, p))
    assert bool(torch.isfinite(got[0][1].float()).all())
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("scales", ["pow2", "any"])
@pytest.mark.parametrize("m,n,k", [(7, 48, 640), (80, 130, 640), (300, 520, 333)])
def test_subnormal_codes(m, n, k, scales, fmt):
    """x subnormal throughout, and among eight neighbours a few far larger ones; w of all sizes"""
    gen = torch.Generator().manual_seed(m + k)
    for few in (0.0, 0.1):
        c = case(m, n, k, torch.float16, False, fmt, scales, bias=False, residual=False)
        top = 8 if fmt == "e4m3" else 4
        raw = torch.randint(0, top, (m, k), generator=gen) + torch.randint(0, 2, (m, k), generator=gen) * 128
        large = torch.rand(m, k, generator=gen) < few
        raw = torch.where(large, torch.randint(0x30, 0x50, (m, k), generator=gen), raw).to(torch.uint8)
        c["x"].view(torch.uint8).copy_(raw.to(DEV))
        c["xr"] = raw.numpy()
        c["sx"] = c["sx"] * 2.0 ** (6 if fmt == "e4m3" else 12)
        forward(c, "none", sums=False)


def test_the_cut_beside_a_subnormal_code():
    """a product of normal codes beside that of a subnormal one, which counts with the
    smallest normal exponent: each off by less than 2^(E - 13)"""
    x = torch.zeros(20, 128, dtype=torch.uint8)
    w = torch.zeros(20, 128, dtype=torch.uint8)
    # x 2^-9 by w 2^8: E = -6 + 8; and 1.5 2^-6 by 1.25 2^-5
    x[:, 0], w[:, 0] = 0x01, 0x78
    x[:, 1], w[:, 1] = 0x0C, 0x12
    values = F.table("e4m3")
    assert values[0x01] == 2.0 ** -9 and values[0x78] == 2.0 ** 8
    assert values[0x0C] * values[0x12] == 1.5 * 2.0 ** -6 * 1.25 * 2.0 ** -5
    exact = 0.5 + 1.875 * 2.0 ** -11
    for m in (4, 20):
        out = torch.empty(m, 20, dtype=torch.float16, device=DEV)
        e4 = torch.float8_e4m3fn
        B.echo_linear8(x[:m].to(DEV).view(e4), torch.ones(m, 1, device=DEV), w.to(DEV).view(e4), torch.ones(1, 1, device=DEV),
                       out, workspace=space(B.echo_linear8_workspace(m, 20, 128)))
        off = (out.double().cpu() - exact).abs().max()
        assert float(off) < 2 * 2.0 ** (2 - 13) + exact * R.HALF_ULP[torch.float16]
