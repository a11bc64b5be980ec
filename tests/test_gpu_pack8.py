"""echo_pack8 and echo_unpack8 on the GPU against binary64: every byte and scale equal.
Types, formats, blocks, parts, transposed codes, odd sizes, pitches and addresses;
zeros, smallest and largest numbers, borders of the scale's rule, ties, NaN and inf;
streams, graphs, nothing written beside the rows."""
import numpy as np
import pytest
import torch

import fp8_reference as F
from error_compensated_bit_echo_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FILL = 0x5A  # a byte in every place that no call may write


def codes_in(rows, cols, fmt, extra=0):
    """a buffer of FILL and a [rows, cols] view of codes in it, rows 16 bytes aligned"""
    pitch = (cols + 15) // 16 * 16 + extra
    buf = torch.full((rows * pitch + 64,), FILL, dtype=torch.uint8, device=DEV)
    return buf, buf[:rows * pitch].view(rows, pitch)[:, :cols].view(F.FORMATS[fmt])


def scales_in(shape):
    buf = torch.full((shape[0] * shape[1] + 16,), 7.0, device=DEV)
    return buf, buf[:shape[0] * shape[1]].view(shape)


def matrix_in(x, extra=0, shift=0):
    """x on the GPU with a pitch, `shift` elements into its buffer"""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + extra) + shift + 8,), 3.0, dtype=x.dtype, device=DEV)
    v = buf[shift:shift + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(x)
    return buf, v


def bytes_of(codes):
    return codes.contiguous().view(torch.uint8).cpu().numpy()


def same_codes(got, want, fmt, what):
    values = F.table(fmt)
    nan = np.isnan(values[want])
    assert np.isnan(values[got[nan]]).all(), f"{what}: NaN expected"
    bad = (got != want) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} differ, first at {np.argwhere(bad)[0]}: {got[bad][:3]} for {want[bad][:3]}"


def beside(buf, view, what):
    """the bytes of buf outside the rows of view are FILL"""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[mask] == FILL).all()), f"{what}: written outside its rows"


def check_pack(x, fmt, blocks=False, parts=1, turned=False, extra=0, shift=0, pad=0):
    rows, cols = x.shape
    want, ws = F.pack(x.double().numpy(), fmt, blocks, parts)
    _, dx = matrix_in(x, pad, shift)
    cb, codes = codes_in(rows, cols, fmt, extra)
    sb, scales = scales_in(ws.shape)
    tb, turned_codes = codes_in(cols, rows, fmt, extra) if turned else (None, None)
    tsb, turned_scales = scales_in(ws.shape[::-1]) if turned else (None, None)
    print(f"pack {tuple(x.shape)} {x.dtype} {fmt} blocks={blocks} parts={parts} turned={turned}", flush=True)
    B.echo_pack8(dx, codes, scales, blocks=blocks, parts=parts, codes_t=turned_codes, scales_t=turned_scales)
    torch.cuda.synchronize()
    same_codes(bytes_of(codes), want, fmt, "codes")
    np.testing.assert_array_equal(scales.cpu().double().numpy(), ws)
    beside(cb, codes.view(torch.uint8), "codes")
    assert bool((sb[scales.numel():] == 7.0).all())
    if turned:
        same_codes(bytes_of(turned_codes), want.T, fmt, "codes_t")
        np.testing.assert_array_equal(turned_scales.cpu().double().numpy(), ws.T)
        beside(tb, turned_codes.view(torch.uint8), "codes_t")
        assert bool((tsb[scales.numel():] == 7.0).all())
    return codes, scales


def draw(rows, cols, dtype, seed=0):
    """values over many binades, a few columns far larger"""
    gen = torch.Generator().manual_seed(seed * 7919 + rows * 31 + cols)
    x = torch.randn(rows, cols, generator=gen) * torch.exp(torch.randn(cols, generator=gen))
    x[:, ::37] *= 50
    return x.to(dtype)


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,parts", [(1, 1, 1), (1, 4096, 1), (3, 7, 1), (5, 128, 1), (7, 129, 1), (9, 1000, 1),
                                             (33, 1001, 1), (4, 16384, 1), (6, 2, 2), (5, 256, 2), (8, 254, 2), (3, 2051 * 2, 2)])
def test_rows(rows, cols, parts, dtype, fmt):
    check_pack(draw(rows, cols, TYPES[dtype]), fmt, parts=parts)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("rows,cols,parts", [(1, 1, 1), (128, 128, 1), (127, 129, 1), (130, 7, 1), (260, 384, 1), (37, 300, 1),
                                             (256, 136, 2), (512, 131, 2)])
def test_blocks(rows, cols, parts, dtype, turned):
    check_pack(draw(rows, cols, TYPES[dtype], 1), "e4m3" if dtype != "f32" else "e5m2", True, parts, turned)


@pytest.mark.parametrize("rows,cols", [(2, 6), (260, 130), (26, 33)])
def test_blocks_of_two_parts_begin_anew(rows, cols):
    check_pack(draw(rows, cols, torch.bfloat16, 2), "e4m3", True, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift,pad,extra", [(1, 0, 16), (3, 5, 48), (0, 8, 0)])
def test_pitches_and_addresses(dtype, shift, pad, extra):
    x = draw(19, 515, TYPES[dtype], 3)
    check_pack(x, "e4m3", extra=extra, shift=shift, pad=pad)
    check_pack(x, "e4m3", True, 1, True, extra=extra, shift=shift, pad=pad)


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_borders(fmt, dtype):
    """a block's largest at and beside the rule's borders, from the smallest numbers to the largest"""
    t, top = TYPES[dtype], F.LARGEST[fmt]
    info = torch.finfo(t)
    at = [top * 2.0 ** e for e in range(-160, 130) if info.tiny * 2.0 ** -8 <= top * 2.0 ** e <= info.max]
    at += [info.max, info.tiny, info.smallest_normal * info.eps, 0.0]
    v = torch.tensor(at, dtype=torch.float64).to(t)
    around = torch.cat([v, torch.nextafter(v, torch.zeros_like(v)), torch.nextafter(v, torch.full_like(v, info.max))])
    gen = torch.Generator().manual_seed(5)
    x = (torch.rand(around.numel(), 128, generator=gen, dtype=torch.float64) * 2 - 1) * around.double()[:, None]
    x[:, 17] = around.double() * torch.where(torch.rand(around.numel(), generator=gen) < 0.5, -1.0, 1.0)
    x[:, 18], x[:, 19] = 0.0, -0.0
    check_pack(x.to(t), fmt)


@pytest.mark.parametrize("fmt", F.FORMATS)
def test_ties_go_to_the_even_code(fmt):
    values = F.table(fmt)
    ladder = np.unique(np.abs(values[np.isfinite(values)]))
    mid = (ladder[1:] + ladder[:-1]) / 2
    pad = -len(mid) % 127
    rows = np.concatenate([mid, np.zeros(pad)]).reshape(-1, 127)
    x = torch.from_numpy(np.concatenate([np.full((len(rows), 1), F.LARGEST[fmt]), rows], 1)).float()  # scale 1
    codes, scales = check_pack(torch.cat([x, -x]), fmt)
    assert bool((scales == 1).all())


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("blocks", [False, True])
def test_nan_and_inf_stay_where_they_are(fmt, dtype, blocks):
    x = draw(140, 300, TYPES[dtype], 4)
    x[0, 5], x[0, 7], x[0, 8] = float("nan"), float("inf"), -float("inf")
    x[3, 128:256] = float("nan")
    x[4, 256:] = float("inf")
    codes, scales = check_pack(x, fmt, blocks, turned=blocks)
    assert bool(torch.isfinite(scales).all())
    v = codes.float().cpu()
    assert torch.equal(torch.isnan(v) | torch.isinf(v), ~torch.isfinite(x.float()))


@pytest.mark.parametrize("fmt", F.FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,blocks,parts", [(1, 1, False, 1), (2, 256, False, 1), (5, 1001, False, 1), (3, 254, False, 2),
                                                    (4, 2, False, 2), (259, 130, True, 1), (262, 21, True, 2)])
def test_unpack(rows, cols, blocks, parts, dtype, fmt):
    """every code, scales that are powers of two and others"""
    gen = torch.Generator().manual_seed(rows + cols)
    raw = torch.randint(0, 256, (rows, cols), generator=gen, dtype=torch.int32).to(torch.uint8)
    raw.view(-1)[:256] = torch.arange(raw.numel(), dtype=torch.int32).to(torch.uint8)[:256]
    shape = F.scales_shape(rows, cols, blocks, parts)
    scales = torch.exp2(torch.randint(-20, 6, shape, generator=gen).float())
    scales = torch.where(torch.rand(shape, generator=gen) < 0.5, scales, scales * (1 + torch.rand(shape, generator=gen)))
    t = TYPES[dtype]
    _, codes = codes_in(rows, cols, fmt, 16)
    codes.view(torch.uint8).copy_(raw)
    ob, out = matrix_in(torch.zeros(rows, cols, dtype=t), 3, 1)
    print(f"unpack {rows} x {cols} {dtype} {fmt} blocks={blocks} parts={parts}", flush=True)
    B.echo_unpack8(codes, scales.to(DEV), out, blocks=blocks, parts=parts)
    torch.cuda.synchronize()
    want = F.values(raw.numpy(), scales.double().numpy(), fmt, blocks, parts)
    # code times scale is rounded to binary32 first where the scale is no power of two: for a 16-bit type
    # that second rounding moves a result by one unit at most where the first one made a tie
    exact = F.rounded(want.astype(np.float32).astype(np.float64), t)
    got = out.cpu()
    nan = torch.isnan(exact)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], exact[~nan])
    mask = torch.ones_like(ob, dtype=torch.bool)
    mask.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(False)
    mask[:1] = True
    assert bool((ob[mask] == 3.0).all()), "written outside its rows"


@pytest.mark.parametrize("dtype", TYPES)
def test_largest_numbers_come_back_finite(dtype):
    """a number next to the type's largest is rounded up by its code, past the type's range"""
    t = TYPES[dtype]
    top = torch.finfo(t).max
    x = torch.full((2, 128), top, dtype=t)
    x[1] = -top
    x[:, 5] = top / 3
    codes, scales = check_pack(x, "e4m3")
    out = torch.empty(2, 128, dtype=t, device=DEV)
    B.echo_unpack8(codes, scales, out)
    got = out.cpu().double()
    assert bool(torch.isfinite(got).all())
    assert bool(((got - x.double()).abs() <= x.double().abs() * 2.0 ** -4).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_code_times_scale_is_exact(dtype):
    """unpacked and packed again, codes and scales are the same"""
    t = TYPES[dtype]
    x = draw(40, 700, t, 6)
    codes, scales = check_pack(x, "e4m3")
    back = torch.empty(40, 700, dtype=t, device=DEV)
    B.echo_unpack8(codes, scales, back)
    want = F.values(bytes_of(codes), scales.cpu().double().numpy(), "e4m3")
    assert torch.equal(back.cpu().double(), torch.from_numpy(want))
    codes2 = B.codes8_empty(40, 700)
    scales2 = torch.empty_like(scales)
    B.echo_pack8(back, codes2, scales2)
    again = torch.empty_like(back)
    B.echo_unpack8(codes2, scales2, again)
    assert torch.equal(again, back)


def test_empty():
    for rows, cols in ((0, 64), (3, 0), (0, 0)):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
        codes, scales = B.codes8_empty(rows, cols), torch.empty(B.scales8_shape(rows, cols), device=DEV)
        B.echo_pack8(x, codes, scales)
        B.echo_unpack8(codes, scales, x)
    torch.cuda.synchronize()


def test_codes_in_rows_that_do_not_line_up_are_refused():
    x = torch.zeros(4, 33, dtype=torch.bfloat16, device=DEV)
    scales = torch.empty(4, 1, device=DEV)
    with pytest.raises(ValueError, match="16 bytes"):
        B.echo_pack8(x, torch.empty(4, 33, dtype=torch.float8_e4m3fn, device=DEV), scales)
    with pytest.raises(ValueError, match="16 bytes"):
        B.echo_pack8(x, torch.empty(8, 48, dtype=torch.float8_e4m3fn, device=DEV)[:4, 8:41], scales)
    with pytest.raises(ValueError):
        B.echo_pack8(x, torch.empty(4, 48, dtype=torch.uint8, device=DEV)[:, :33], scales)
    with pytest.raises(ValueError, match="scales"):
        B.echo_pack8(x, B.codes8_empty(4, 33), torch.empty(4, 2, device=DEV))
    with pytest.raises(ValueError, match="codes_t"):
        B.echo_pack8(x, B.codes8_empty(4, 33), torch.empty(1, 1, device=DEV), blocks=True,
                     codes_t=B.codes8_empty(33, 4, torch.float8_e5m2), scales_t=torch.empty(1, 1, device=DEV))


def test_stream_and_graph():
    x = draw(64, 640, torch.bfloat16, 7).to(DEV)
    codes, scales = B.codes8_empty(64, 640), torch.empty(64, 5, device=DEV)
    back = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.echo_pack8(x, codes, scales)
        B.echo_unpack8(codes, scales, back)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [bytes_of(codes), scales.clone(), back.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.echo_pack8(x, codes, scales)
        B.echo_unpack8(codes, scales, back)
    for turn in range(3):
        codes.view(torch.uint8).fill_(1)
        scales.zero_()
        back.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (bytes_of(codes) == want[0]).all() and torch.equal(scales, want[1]) and torch.equal(back, want[2])
    x.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    w, s = F.pack(x.cpu().double().numpy(), "e4m3", False, 1)
    same_codes(bytes_of(codes), w, "e4m3", "codes")


@pytest.mark.parametrize("cols,blocks", [(33000, False), (33280, False), (33000, True)])
def test_offsets_past_32_bits(cols, blocks):
    """a matrix of more than 2^31 elements, its first and last rows looked at: of odd
    length, of whole wavefronts, and in blocks of 128 x 128 with its transpose"""
    rows, some = 65664, 128
    top, end = draw(some, cols, torch.bfloat16, 1), draw(some, cols, torch.bfloat16, 2)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:some], x[-some:] = top.to(DEV), end.to(DEV)
    codes, scales = B.codes8_empty(rows, cols), torch.empty(B.scales8_shape(rows, cols, blocks=blocks), device=DEV)
    turned = [B.codes8_empty(cols, rows), torch.empty(tuple(scales.shape)[::-1], device=DEV)] if blocks else [None, None]
    print(f"pack {rows} x {cols} blocks={blocks}", flush=True)
    B.echo_pack8(x, codes, scales, blocks=blocks, codes_t=turned[0], scales_t=turned[1])
    back = torch.full_like(x, 1.0)
    B.echo_unpack8(codes, scales, back, blocks=blocks)
    torch.cuda.synchronize()
    high = 1 if blocks else some  # rows of scales
    for part, sel, ssel in ((top, slice(0, some), slice(0, high)), (end, slice(rows - some, rows), slice(-high, None))):
        want, ws = F.pack(part.double().numpy(), "e4m3", blocks, 1)
        same_codes(bytes_of(codes[sel]), want, "e4m3", "codes")
        np.testing.assert_array_equal(scales[ssel].cpu().double().numpy(), ws)
        if blocks:
            same_codes(bytes_of(turned[0].view(torch.uint8)[:, sel]), want.T, "e4m3", "codes_t")
            np.testing.assert_array_equal(turned[1][:, ssel].cpu().double().numpy(), ws.T)
        values = torch.from_numpy(F.values(want, ws, "e4m3", blocks)).to(torch.bfloat16)
        assert torch.equal(back[sel].cpu(), values)
    assert not back[some:-some].any()


def test_more_vectors_than_a_32_bit_division_counts():
    """2^31 vectors of eight and a few, two to a row"""
    rows, cols, last = (1 << 30) + 5, 9, 4099
    codes = torch.zeros(rows, 16, dtype=torch.uint8, device=DEV)
    raw = torch.randint(0, 120, (last, 16), generator=torch.Generator().manual_seed(3), dtype=torch.uint8)
    codes[-last:] = raw.to(DEV)
    scales = torch.ones(rows, 1, device=DEV)
    scales[-last:, 0] = torch.exp2(torch.arange(last, device=DEV) % 7 - 3.0)
    x = torch.ones(rows, cols, dtype=torch.float16, device=DEV)
    B.echo_unpack8(codes[:, :cols].view(torch.float8_e4m3fn), scales, x)
    torch.cuda.synchronize()
    want = F.values(raw[:, :cols].numpy(), scales[-last:].cpu().double().numpy(), "e4m3")
    assert torch.equal(x[-last:].cpu(), torch.from_numpy(want).half())
    assert not x[:-last].any()
