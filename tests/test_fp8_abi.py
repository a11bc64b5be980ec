"""The 8-bit operators' ABI without a GPU: include/echo_fp8.h and the library agree,
and every bad argument is refused before anything is launched."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

from error_compensated_bit_echo_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 32  # fake, well-aligned addresses: every call below is rejected


def test_library_exports_what_the_header_declares():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "echo_fp8.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(echo_\w+)\s*\(", src, re.M))
    raw = C.CDLL(B.LIB_PATH)
    assert names == set(B.EXPORTED_FP8)
    for name in names:
        assert hasattr(raw, name), name


C_CONSUMER = r"""
#include <stdio.h>
#include "echo_fp8.h"
int main(void) {
  echo_pack8_desc p = {0};
  echo_linear8_desc l = {0};
  if (echo_pack8(&p, 0, 0, 0, 0, 0, 0) != ECHO_ERR_TYPE) return 1; /* format 0 */
  p.format = ECHO_E4M3;
  if (echo_pack8(&p, 0, 0, 0, 0, 0, 0) != ECHO_ERR_SHAPE) return 2; /* parts 0 */
  p.parts = 1;
  if (echo_pack8(&p, 0, 0, 0, 0, 0, 0) != ECHO_SUCCESS) return 3; /* nothing to do */
  p.rows = 4; p.cols = 8;
  if (echo_unpack8(&p, 0, 0, 0, 0) != ECHO_ERR_INVALID_ARGUMENT) return 4;
  l.m = 4; l.n = 4; l.k = 4;
  if (echo_linear8_workspace(&l) != ECHO_ERR_TYPE) return 5;
  l.x_format = ECHO_E5M2; l.act = ECHO_ACT_SILU; l.gated = 1;
  if (echo_linear8_workspace(&l) < 0 || echo_linear_backward8_workspace(&l) <= 0) return 6;
  if (echo_linear8(&l, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != ECHO_ERR_INVALID_ARGUMENT) return 7;
  l.m = 0;
  if (echo_linear8(&l, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != ECHO_SUCCESS) return 8;
  puts("ok");
  return 0;
}
"""


def test_header_is_plain_c(tmp_path):
    """the header compiles as C11 and a program without Python links against it"""
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    (tmp_path / "c.c").write_text(C_CONSUMER)
    exe = str(tmp_path / "c")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(tmp_path / "c.c"), "-o", exe, B.LIB_PATH, "-L", os.path.join(rocm, "lib"), "-lamdhip64",
                    f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}:{os.path.join(rocm, 'lib')}"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.returncode


def matrix(R=256, K=64, ld_x=0, ld_c=0, ld_t=0, dt=0, fmt=3, blocks=0, parts=1):
    return B.EchoPack8DescC(R, K, ld_x, ld_c, ld_t, dt, fmt, blocks, parts)


def pack(d, x=A, codes=2 * A, scales=3 * A, codes_t=None, scales_t=None):
    return B.lib.echo_pack8(C.byref(d) if d else None, x, codes, scales, codes_t, scales_t, None)


def unpack(d, codes=2 * A, scales=3 * A, x=A):
    return B.lib.echo_unpack8(C.byref(d) if d else None, codes, scales, x, None)


def test_pack_rejections():
    for call in (pack, unpack):
        assert call(None) == -1
        for bad in (dict(R=-1), dict(K=-1), dict(K=(1 << 21) + 1), dict(R=(1 << 31) + 1), dict(R=(1 << 21) + 1, blocks=1),
                    dict(R=1 << 31, K=1 << 12), dict(ld_x=63), dict(ld_x=1 << 22), dict(ld_c=48), dict(ld_c=1 << 22),
                    dict(parts=0), dict(parts=3), dict(K=65, parts=2), dict(R=255, blocks=1, parts=2)):
            assert call(matrix(**bad)) == -2, bad
        for bad in (dict(dt=3), dict(dt=-1), dict(fmt=2), dict(fmt=5), dict(fmt=0), dict(blocks=2), dict(blocks=-1)):
            assert call(matrix(**bad)) == -8, bad
        assert call(matrix(ld_c=72)) == -3  # no multiple of 16
        assert call(matrix(), x=None) == -1 and call(matrix(), codes=None) == -1 and call(matrix(), scales=None) == -1
        assert call(matrix(), codes=2 * A + 8) == -3 and call(matrix(), scales=3 * A + 2) == -3
        assert call(matrix(), x=A + 1) == -3 and call(matrix(dt=2), x=A + 2) == -3
        assert call(matrix(), codes=A) == -6 and call(matrix(), scales=A + 4) == -6
        assert call(matrix(R=0), x=None, codes=None, scales=None) == 0
        assert call(matrix(K=0), x=None, codes=None, scales=None) == 0
    # codes that would lie over the scales
    assert pack(matrix(), scales=2 * A + 64) == -6


def test_transposed_pack_rejections():
    turned = dict(codes_t=4 * A, scales_t=5 * A)
    assert pack(matrix(), **turned) == -2  # blocks of 1 x 128
    assert pack(matrix(R=200, blocks=1, parts=2), **turned) == -2  # a part of 100 rows
    assert pack(matrix(blocks=1), codes_t=4 * A) == -1 and pack(matrix(blocks=1), scales_t=4 * A) == -1
    assert pack(matrix(blocks=1, ld_t=255), **turned) == -2
    assert pack(matrix(blocks=1, ld_t=264), **turned) == -3
    assert pack(matrix(blocks=1), codes_t=4 * A + 4, scales_t=5 * A) == -3
    assert pack(matrix(blocks=1), codes_t=4 * A, scales_t=5 * A + 2) == -3
    assert pack(matrix(blocks=1), codes_t=2 * A + 16, scales_t=5 * A) == -6
    assert pack(matrix(blocks=1), codes_t=4 * A, scales_t=3 * A) == -6


def desc(m=32, n=64, k=128, ld_x=0, ld_w=0, ld_out=0, ld_r=0, ld_p=0, dt=0, act=0, gated=0, fmt=3):
    return B.EchoLinear8DescC(m, n, k, ld_x, ld_w, ld_out, ld_r, ld_p, dt, act, gated, fmt)


def fwd(d, x=A, sx=2 * A, w=3 * A, sw=4 * A, bias=None, res=None, out=5 * A, p=None, ws=7 * A, ws_bytes=1 << 40):
    return B.lib.echo_linear8(C.byref(d) if d else None, x, sx, w, sw, bias, res, out, p, ws, ws_bytes, None)


def bwd(d, dout=A, x=2 * A, sx=3 * A, w=4 * A, p=5 * A, sp=6 * A, dx=7 * A, dw=8 * A, db=9 * A, ws=10 * A,
        ws_bytes=1 << 30):
    return B.lib.echo_linear_backward8(C.byref(d) if d else None, dout, x, sx, w, p, sp, dx, dw, db, ws, ws_bytes, None)


SHAPES = (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=(1 << 31) + 1), dict(k=(1 << 21) + 1), dict(n=(1 << 21) + 1),
          dict(n=(1 << 20) + 1, gated=1), dict(m=1 << 31, n=1 << 12, k=1), dict(m=1 << 31, n=1, k=1 << 12),
          dict(ld_x=112), dict(ld_x=1 << 22), dict(ld_out=63), dict(ld_out=1 << 22))
TYPES = (dict(dt=2), dict(dt=-1), dict(act=5), dict(act=-1), dict(gated=2), dict(fmt=2), dict(fmt=0), dict(fmt=5))


def test_linear8_rejections():
    assert fwd(None) == -1
    for bad in SHAPES + (dict(ld_w=112), dict(ld_w=1 << 22), dict(ld_r=63), dict(ld_r=1 << 22)):
        assert fwd(desc(**bad)) == -2, bad
    for bad in TYPES:
        assert fwd(desc(**bad)) == -8 and B.lib.echo_linear8_workspace(C.byref(desc(**bad))) == -8, bad
    for bad in (dict(ld_x=136), dict(ld_w=129), dict(ld_x=200)):
        assert fwd(desc(**bad)) == -3, bad
    for name in ("x", "sx", "w", "sw", "out"):
        assert fwd(desc(), **{name: None}) == -1, name
    for name, off in (("x", 8), ("w", 4), ("sx", 2), ("sw", 1), ("out", 1), ("bias", 1), ("res", 1), ("p", 1), ("ws", 8)):
        if name == "ws":
            continue
        assert fwd(desc(), **{name: 20 * A + off}) == -3, name
    for name, at in (("out", A), ("out", 2 * A), ("out", 3 * A + 16), ("out", 4 * A), ("p", 5 * A), ("p", A)):
        assert fwd(desc(), **{name: at}) == -6, (name, at)
    assert fwd(desc(), bias=5 * A) == -6 and fwd(desc(), res=5 * A + 2) == -6
    assert fwd(desc(ld_r=72), res=5 * A) == -6  # in place with another pitch
    assert fwd(desc(m=0), x=None, w=None, out=None) == 0 and fwd(desc(n=0), out=None) == 0


def test_linear8_workspace_is_checked():
    d = desc(m=512, n=256, k=16384)
    need = B.lib.echo_linear8_workspace(C.byref(d))
    assert need > 0  # a long contraction over few tiles is split
    assert fwd(d, ws=None) == -1 and fwd(d, ws_bytes=need - 1) == -9 and fwd(d, ws=7 * A + 8) == -3
    assert fwd(d, ws=5 * A) == -6 and fwd(d, ws=A) == -6
    # a decode step takes none
    assert B.echo_linear8_workspace(16, 4096, 16384) == 0


def test_linear_backward8_rejections():
    assert bwd(None) == -1
    for bad in SHAPES + (dict(ld_w=100), dict(ld_w=1 << 22), dict(ld_p=48, act=1), dict(ld_p=64, gated=1)):
        assert bwd(desc(**bad)) == -2, bad
    for bad in TYPES:
        assert bwd(desc(**bad)) == -8 and B.lib.echo_linear_backward8_workspace(C.byref(desc(**bad))) == -8, bad
    assert bwd(desc(ld_x=136)) == -3 and bwd(desc(ld_p=72, act=1)) == -3
    d = desc(act=4)
    need = B.lib.echo_linear_backward8_workspace(C.byref(d))
    assert need > 0
    for name in ("dout", "x", "sx", "w", "p", "sp", "ws"):
        assert bwd(d, **{name: None}) == -1, name
    assert bwd(d, ws_bytes=need - 1) == -9
    for name, off in (("x", 8), ("p", 8), ("ws", 8), ("sx", 2), ("sp", 2), ("w", 1), ("dout", 1), ("dx", 1), ("dw", 1), ("db", 1)):
        assert bwd(d, **{name: 20 * A + off}) == -3, name
    for name, at in (("dx", A), ("dx", 2 * A), ("dw", 4 * A), ("dw", 7 * A), ("db", 8 * A), ("ws", 5 * A), ("ws", 7 * A),
                     ("dx", 6 * A), ("db", 3 * A)):
        assert bwd(d, **{name: at}) == -6, (name, at)


def test_binding_refuses_what_the_library_cannot_see():
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 32).to(e4), torch.zeros(4, 1)
    for call in (lambda: B.echo_pack8(x, codes, scales, stream=0), lambda: B.echo_unpack8(codes, scales, x, stream=0),
                 lambda: B.echo_linear8(codes, scales, codes, scales, x, stream=0),
                 lambda: B.echo_linear_backward8(x, codes, scales, x, None, None, x, x, stream=0)):
        with pytest.raises(ValueError):
            call()  # tensors of the host
    with pytest.raises(ValueError, match="act"):
        B.echo_linear8_workspace(4, 4, 4, act="tanh")
    assert B.scales8_shape(300, 130) == (300, 2) and B.scales8_shape(300, 260, parts=2) == (300, 4)
    assert B.scales8_shape(300, 130, blocks=True) == (3, 2) and B.scales8_shape(516, 130, blocks=True, parts=2) == (6, 2)
    c = B.codes8_empty(3, 33, e5, device="cpu")
    assert c.shape == (3, 33) and c.stride() == (48, 1) and c.dtype is e5


def test_largest_allowed_shapes_have_an_answer():
    for m, n, k in ((1 << 31, 1, 1), (1 << 31, 8, 64), (1 << 21, 1 << 21, 1 << 21), (1 << 31, 1 << 11, 1 << 11), (0, 0, 0)):
        for gated in (False, True):
            if m * n * 2 <= 1 << 42 and n <= 1 << 20 or not gated:
                assert B.echo_linear8_workspace(m, n, k, gated=gated) >= 0, (m, n, k, gated)
                assert B.echo_linear_backward8_workspace(m, n, k, gated=gated) >= 0, (m, n, k, gated)


def test_grids_and_splits_within_limits(tmp_path):
    """the plan of every allowed size (host arithmetic, g++)"""
    src = tmp_path / "plan.cc"
    src.write_text(r"""
#include <stdio.h>
#include <initializer_list>
#include "linear8_plan.h"
using namespace echo;
int main() {
  for (int64_t m = 1; m <= ECHO_MAX_ROWS; m *= 2)
    for (const int64_t rows : {m - 1, m, m + 1, m + m / 2})
      for (int64_t n = 1; n <= ECHO_MAX_PITCH; n *= 2)
        for (const int64_t k : {INT64_C(1), INT64_C(127), INT64_C(128), INT64_C(4104), n}) {
          if (rows < 1 || rows > ECHO_MAX_ROWS || rows * n > ECHO_MAX_PRODUCT || rows * k > ECHO_MAX_PRODUCT) continue;
          const Plan p = plan_tiles8(rows, n, k);
          const TileCost& c = kCost8[p.tile];
          const int64_t tiles = ((rows + c.bi - 1) / c.bi) * ((n + c.bj - 1) / c.bj) * p.splits;
          if (tiles > 0xFFFFFFFFll || p.splits < 1 || p.chunk % kC8 || p.splits * p.chunk < k ||
              (p.splits - 1) * p.chunk >= k || p.part_bytes < 0 || (p.splits > 1 && p.part_bytes < 4 * rows * n * p.splits)) {
            printf("%lld %lld %lld: tile %d splits %lld\n", (long long)rows, (long long)n, (long long)k, p.tile, (long long)p.splits);
            return 1;
          }
          const TileGrid g = grid_of((uint32_t)tiles, 512);
          if (g.y < 1 || g.y > 65535 || (uint64_t)g.x * 512 > 0xFFFFFFFFull || (uint64_t)g.x * g.y < (uint64_t)tiles) return 2;
        }
  puts("ok");
}
""")
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "error_compensated_bit_echo_amd", "csrc"), str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
