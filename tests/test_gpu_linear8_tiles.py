"""Every tile of echo_linear8 against binary64 (bounds as in test_gpu_linear8.py), and
products past 32 bits of offsets."""
import numpy as np
import pytest
import torch

import fp8_reference as F
import layer_reference as R
from error_compensated_bit_echo_amd import binding as B
from linear8_tile_cases import CASES
from test_gpu_linear8 import case, forward, space
from test_gpu_norm import DEV, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(CASES))
def test_tile(name):
    m, n, k, act, gated, scales = CASES[name][:6]
    dt = torch.float16 if "64" in name else torch.bfloat16
    forward(case(m, n, k, dt, gated, "e5m2" if "gated" in name and "other" in name else "e4m3", scales), act)


@pytest.mark.parametrize("name", ["256", "128", "64", "128 alone", "64 alone"])
def test_rows_behind_the_last_one_have_no_influence(name):
    """x and w end at the end of their buffers but for the last row's filling, and hold NaN
    there; the same bits as without"""
    m, n, k, act, gated, scales = CASES[name][:6]
    c = case(m, n, k, torch.bfloat16, gated, "e4m3", scales, bias=False, residual=False)
    a, _ = forward(c, act, keep=False, sums=False)
    for name in ("x", "w"):
        rows, pitch = c[name].shape[0], (k + 15) // 16 * 16
        buf = torch.zeros(rows, pitch, dtype=torch.uint8, device=DEV)
        buf[:, :k] = c[name].view(torch.uint8)
        c[name] = buf[:, :k].view(c[name].dtype)
    b, _ = forward(c, act, keep=False, sums=False)
    assert torch.equal(a, b)


def windows(x, w, sx, sw, out, rows, k):
    """a few rows of a large product, exactly"""
    xr = x[rows].contiguous().view(torch.uint8).cpu().numpy()
    wr = w.contiguous().view(torch.uint8).cpu().numpy()
    units = 2 * (k + 64)
    p, pa = F.products(xr, sx[rows].cpu().double().numpy(), "e4m3", wr, sw.cpu().double().numpy(), 1, units)
    R.close(out[rows], p, pa, units, "out")


def test_offsets_past_32_bits():
    """more than 2^32 bytes of codes, and scales and outputs past 2^31 bytes of their own"""
    m, n, k = (1 << 22) + 77, 300, 1040
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GiB")
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(0, 120, (m, k), dtype=torch.uint8, device=DEV, generator=gen)
    x = torch.where(torch.rand(1, k, device=DEV, generator=gen) < 0.5, x, x | 0x80).view(torch.float8_e4m3fn)
    w = torch.randn(n, k, device=DEV, generator=gen).to(torch.float8_e4m3fn)
    sx = torch.exp2(torch.randint(-4, 4, (m, 9), device=DEV, generator=gen).float())
    sw = torch.exp2(torch.randint(-4, 4, (3, 9), device=DEV, generator=gen).float()) * 1.25
    out = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    B.echo_linear8(x, sx, w, sw, out, workspace=space(B.echo_linear8_workspace(m, n, k)))
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 255, 256, (1 << 21) - 1, 1 << 21, (1 << 32) // k, (1 << 32) // k + 1, m - 78, m - 77, m - 1], device=DEV)
    windows(x, w, sx, sw, out, rows, k)
    # and the unpacked rows there
    back = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    B.echo_unpack8(x, sx, back)
    want = F.values(x[rows].contiguous().view(torch.uint8).cpu().numpy(), sx[rows].cpu().double().numpy(), "e4m3")
    assert torch.equal(back[rows].cpu().double(), torch.from_numpy(want))
    again, scales = B.codes8_empty(m, k), torch.empty_like(sx)
    B.echo_pack8(back, again, scales)
    codes, s = F.pack(want, "e4m3", False, 1)
    assert (again[rows].contiguous().view(torch.uint8).cpu().numpy() == codes).all()
    assert np.array_equal(scales[rows].cpu().double().numpy(), s)


def test_a_gated_weight_past_31_bits():
    """up rows more than 2^31 bytes behind their gate's"""
    m, n, k = 40, (1 << 20), 2064
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GiB")
    gen = torch.Generator(device=DEV).manual_seed(2)
    w = torch.randint(0, 120, (2 * n, k), dtype=torch.uint8, device=DEV, generator=gen).view(torch.float8_e4m3fn)
    x = torch.randn(m, k, device=DEV, generator=gen).to(torch.float8_e4m3fn)
    sx = torch.exp2(torch.randint(-9, -4, (m, 17), device=DEV, generator=gen).float())
    sw = torch.exp2(torch.randint(-9, -4, (2 * n // 128, 17), device=DEV, generator=gen).float())
    cols = torch.tensor([0, 1, 127, 128, 31, 32, n // 2, n - 129, n - 1])
    xr = x.contiguous().view(torch.uint8).cpu().numpy()
    both = torch.cat([cols, cols + n])
    wv = F.table("e4m3")[w[both.to(DEV)].contiguous().view(torch.uint8).cpu().numpy()]
    wv = wv * np.repeat(sw[(both // 128).to(DEV)].cpu().double().numpy(), 128, 1)[:, :k]
    xv = F.values(xr, sx.cpu().double().numpy(), "e4m3")
    for rows in (m, 3):
        out = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
        ws = space(B.echo_linear8_workspace(rows, n, k, act="relu", gated=True))
        B.echo_linear8(x[:rows], sx[:rows], w, sw, out, act="relu", gated=True, workspace=ws)
        torch.cuda.synchronize()
        p, pa = xv[:rows] @ wv.T, np.abs(xv[:rows]) @ np.abs(wv).T
        half = len(cols)
        want = np.maximum(p[:, :half], 0) * p[:, half:]
        # a product's sums by 2^-10 of their magnitude (eight cuts of 2^-13 of the largest beside them)
        magnitude = (pa[:, :half] * np.abs(p[:, half:]) + np.abs(p[:, :half]) * pa[:, half:])
        R.close(out[:, cols.to(DEV)], want, magnitude, 2.0 ** 14 + 2 * (k + 64), "out")
