"""echo_unpack8 rounds code times scale to a 16-bit type once: scales that are no powers of
two, chosen so that the product, rounded to binary32, would lie halfway between two
neighbours of the type, which it does not itself.  Every element equal to the one rounding
of the exact product; and the product of echo_linear_backward8 that reads x unpacked."""
import numpy as np
import pytest
import torch

import fp8_reference as F
from error_compensated_bit_echo_amd import binding as B
from test_gpu_norm import DEV
from test_gpu_pack8 import codes_in, matrix_in

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LOW_BITS = {"bf16": 16, "f16": 13}  # of a binary32 number's that the type does not hold
# exponents of the halves: subnormal numbers of the type among them, and the largest
EXPONENTS = {"bf16": (-133, -130, -127, -126, -100, -20, -1, 0, 3, 60, 127), "f16": (-25, -24, -20, -15, -14, -3, 0, 5, 15)}
LEAST = {"bf16": (-126, -133), "f16": (-14, -24)}  # exponents of the smallest normal and subnormal number


def halfway(dtype, fmt, rng, each=6):
    """[(byte of a code, scale)]: the product in binary32 is halfway between two neighbours
    of the type, the exact one is not"""
    values = F.table(fmt)
    codes = [c for c in range(128) if np.isfinite(values[c]) and values[c] > 0]
    normal, smallest = LEAST[dtype]
    found = []
    for e in EXPONENTS[dtype]:
        unit = 2.0 ** (max(e, normal) + LOW_BITS[dtype] - 23)  # between neighbours of the type at 2^e
        have = 0
        for _ in range(4000):
            v = (np.floor(2.0 ** e * (1 + rng.random()) / unit) + 0.5) * unit
            byte = int(rng.choice(codes))
            if v / values[byte] > F.LARGEST_OF[torch.float32]:
                continue
            s = np.float32(v / values[byte])
            for s in (s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(np.inf))):
                if not np.isfinite(s):
                    continue
                product = float(s) * values[byte]
                if product != v and float(np.float32(product)) == v:
                    found.append((byte, s))
                    have += 1
                    break
            if have == each:
                break
    assert len(found) > 3 * len(EXPONENTS[dtype])
    return found


def twice(v, t):
    """by way of binary32"""
    top = F.LARGEST_OF[torch.float32]
    return F.rounded(np.where(np.isfinite(v), np.clip(v, -top, top), v).astype(np.float32).astype(np.float64), t)


def planted(rows, cols, blocks, parts, dtype, fmt):
    """bytes and scales with the products of halfway() in every block"""
    rng = np.random.default_rng(rows * 31 + cols)
    pool = halfway(dtype, fmt, rng)
    raw = rng.integers(0, 256, (rows, cols), dtype=np.uint8)
    scales = np.zeros(F.scales_shape(rows, cols, blocks, parts), np.float32)
    for at, (r, c, i, j) in enumerate(F.places(rows, cols, blocks, parts)):
        byte, scales[i, j] = pool[at % len(pool)]
        raw[r, c][rng.random(raw[r, c].shape) < 0.3] = byte
        if at % 3 == 0:
            scales[i, j] = -scales[i, j]
        if at % 7 == 6:  # and a power of two among them
            scales[i, j] = 0.25
    return raw, scales


SHAPES = [(130, 512, False, 1), (140, 1024, False, 2), (150, 333, False, 1), (128, 514, False, 2), (600, 1500, True, 1),
          (512, 1203, True, 2)]


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,blocks,parts", SHAPES)
def test_unpack_rounds_once(rows, cols, blocks, parts, dtype, fmt):
    t = TYPES[dtype]
    raw, scales = planted(rows, cols, blocks, parts, dtype, fmt)
    want = F.values(raw, scales.astype(np.float64), fmt, blocks, parts)
    exact = F.rounded(want, t)
    nan = torch.isnan(exact)
    assert int(((exact != twice(want, t)) & ~nan).sum()) > 20  # (what the shape is for)
    _, codes = codes_in(rows, cols, fmt, 16)
    codes.view(torch.uint8).copy_(torch.from_numpy(raw))
    _, out = matrix_in(torch.zeros(rows, cols, dtype=t), 3, 1)
    print(f"unpack {rows} x {cols} {dtype} {fmt} blocks={blocks} parts={parts}", flush=True)
    B.echo_unpack8(codes, torch.from_numpy(scales).to(DEV), out, blocks=blocks, parts=parts)
    torch.cuda.synchronize()
    got = out.cpu()
    assert torch.equal(torch.isnan(got), nan)
    off = (got != exact) & ~nan
    assert not bool(off.any()), f"{int(off.sum())} differ: {got[off][:4]} for {exact[off][:4]}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("k", [512, 300])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_reads_x_rounded_once(k, act, fmt, dtype):
    """dp is the identity, so a row of dw is a row of x as it was unpacked"""
    m, t = 128, TYPES[dtype]
    raw, scales = planted(m, k, False, 1, dtype, fmt)
    raw = np.where(np.isfinite(F.table(fmt)[raw]), raw, 0x38).astype(np.uint8)
    want = F.values(raw, scales.astype(np.float64), fmt)
    exact = F.rounded(want, t)
    normal = exact.abs() >= torch.finfo(t).tiny  # (of smaller ones the product is not this test's)
    assert int(((exact != twice(want, t)) & normal).sum()) > 20
    _, x = codes_in(m, k, fmt)
    x.view(torch.uint8).copy_(torch.from_numpy(raw))
    dout = torch.eye(m, dtype=t, device=DEV)
    p = sp = None
    if act != "none":  # a positive sum everywhere: slope 1
        p, sp = torch.full((m, m), 0x38, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn), torch.ones(m, 1, device=DEV)
    w, dw = torch.zeros(m, k, dtype=t, device=DEV), torch.empty(m, k, dtype=t, device=DEV)
    ws = torch.empty(B.echo_linear_backward8_workspace(m, m, k, act=act), dtype=torch.uint8, device=DEV)
    print(f"linear_backward8 m={m} k={k} {act} {dtype} {fmt}", flush=True)
    B.echo_linear_backward8(dout, x, torch.from_numpy(scales).to(DEV), w, p, sp, None, dw, act=act, workspace=ws)
    torch.cuda.synchronize()
    got = dw.cpu()
    off = (got != exact) & normal
    assert not bool(off.any()), f"{int(off.sum())} differ: {got[off][:4]} for {exact[off][:4]}"
