"""echo_linear8 with scales of x and w whose product is below binary32's smallest normal
number, or its smallest: what the header says of them, by every tile and in few rows, with
such blocks all along a row and only at its end.

Bounds.  As in test_gpu_linear8.py, and the product of two scales rounded to a multiple of
2^-149 is off by at most 2^-150, once for each block, times the sum of the block's codes'
products: 2^-150 of the sum of their magnitudes over all blocks."""
import numpy as np
import pytest
import torch

import fp8_reference as F
import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from linear8_tile_cases import CASES
from test_gpu_linear8 import space
from test_gpu_norm import DEV, on

pytestmark = pytest.mark.gpu
SHAPES = {"one row": (1, 40, 1100, False), "few rows": (11, 72, 2300, False), "few rows gated": (16, 40, 1100, True),
          **{name: (c[0], c[1], c[2], c[4]) for name, c in CASES.items()}}


def codes_of(rows, cols, gen):
    """large positive codes (128 to 448), so that the sums of the smallest products are large"""
    raw = torch.randint(0x70, 0x7F, (rows, cols), generator=gen, dtype=torch.int32).to(torch.uint8)
    buf = torch.full((rows, (cols + 15) // 16 * 16), 0x7F, dtype=torch.uint8, device=DEV)
    buf[:, :cols] = raw.to(DEV)
    return buf[:, :cols].view(torch.float8_e4m3fn), raw.numpy()


def case(m, n, k, gated, kind):
    """"powers": all scales powers of two; "other": none; "late": blocks of powers of two, blocks
    of others, and behind them those whose products are small, the codes before them 0"""
    gen = torch.Generator().manual_seed(m * 31 + n * 17 + k)
    rows, parts = (2 * n, 2) if gated else (n, 1)
    kb, digits = -(-k // 128), 1.0 if kind == "powers" else 1.25
    x, xr = codes_of(m, k, gen)
    w, wr = codes_of(rows, k, gen)
    sw = torch.full(F.scales_shape(rows, k, True, parts), 2.0 ** -31 * (1.0 if kind == "powers" else 1.5))
    sx = torch.full((m, kb), digits)  # every third row's products are large enough
    for at, small in ((0, 2.0 ** -120), (2, 2.0 ** -118)):
        sx[at::3] = digits * small
    if kind == "late":
        first, second = kb // 3, 2 * (kb // 3)
        sw[:, :first], sw[:, first:second] = 2.0 ** -5, 1.5 * 2.0 ** -5
        sx[:, :first] /= 1.25
        for at in (0, 2):
            x.view(torch.uint8)[at::3, :second * 128] = 0
            xr[at::3, :second * 128] = 0
    return {"x": x, "w": w, "sx": sx, "sw": sw, "xr": xr, "wr": wr, "gated": gated}


def product(c, keep=True):
    """(out, p) with NONE as the activation"""
    (m, k), rows = c["x"].shape, c["w"].shape[0]
    n = rows // 2 if c["gated"] else rows
    out, p = (torch.empty(m, q, dtype=torch.bfloat16, device=DEV) for q in (n, rows))
    print(f"linear8 m={m} n={n} k={k} gated={c['gated']}", flush=True)
    B.echo_linear8(c["x"], on(c["sx"]), c["w"], on(c["sw"]), out, gated=c["gated"], p=p if keep else None,
                   workspace=space(B.echo_linear8_workspace(m, n, k, gated=c["gated"])))
    torch.cuda.synchronize()
    return out, p


@pytest.mark.parametrize("kind", ["powers", "other", "late"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_small_products_of_scales(name, kind):
    c = case(*SHAPES[name], kind)
    assert float(c["sx"][0, -1].double() * c["sw"][0, -1].double()) < 2.0 ** -149  # (what the case is for)
    out, p = product(c)
    units = 2 * (c["x"].shape[1] + 64)
    want, magnitude = F.products(c["xr"], c["sx"].double().numpy(), "e4m3", c["wr"], c["sw"].double().numpy(),
                                 2 if c["gated"] else 1, units)
    values = F.table("e4m3")
    lost = 2.0 ** -150 * (np.abs(values[c["xr"]]) @ np.abs(values[c["wr"]]).T)
    R.close(p, want, magnitude + lost / (units * R.EPS32), units, "p")
    if not c["gated"]:
        assert torch.equal(out, p)


@pytest.mark.parametrize("m,n,k", [(9, 40, 1100), (200, 130, 1100), (1270, 1270, 600), (4090, 4088, 330)])
def test_rows_do_not_meet_their_neighbours_scales(m, n, k):
    """a row whose products of scales are small leaves the others' sums as they were, where all
    scales are of one kind"""
    c = case(m, n, k, False, "other")
    c["sx"][:] = 1.25
    want = product(c, keep=False)[0].clone()
    c["sx"][m // 2] = 1.25 * 2.0 ** -119
    out = product(c, keep=False)[0]
    rest = torch.arange(m, device=DEV) != m // 2
    assert torch.equal(out[rest], want[rest])


@pytest.mark.parametrize("m", [5, 100])
def test_zero_beside_the_largest_scale(m):
    """0 times a scale near the end of binary32 is 0, whatever the codes' products"""
    gen = torch.Generator().manual_seed(m)
    x, _ = codes_of(m, 256, gen)
    w, _ = codes_of(130, 256, gen)
    sx, sw = torch.full((m, 2), 2.0 ** -20, device=DEV), torch.full((2, 2), 1.5 * 2.0 ** -140, device=DEV)
    sx[m // 2], sw[1] = 0.0, 1.5 * 2.0 ** 120
    out = torch.empty(m, 130, dtype=torch.bfloat16, device=DEV)
    B.echo_linear8(x, sx, w, sw, out, workspace=space(B.echo_linear8_workspace(m, 130, 256)))
    torch.cuda.synchronize()
    assert not bool(out[m // 2].any()) and bool(torch.isfinite(out.float()).all())
    assert bool((out[:m // 2, 128:] > 2.0 ** 100).all())
