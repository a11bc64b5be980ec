"""The layer operators' ABI without a GPU: include/echo_layer.h and the library
agree, and every bad argument is refused before anything is launched."""
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
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "echo_layer.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(echo_\w+)\s*\(", src, re.M))
    raw = C.CDLL(B.LIB_PATH)
    assert names == set(B.EXPORTED_LAYER)
    for name in names:
        assert hasattr(raw, name), name


def test_new_status_strings():
    for code in (-8, -9):
        assert B.status_string(code) != "unknown status"


C_CONSUMER = r"""
#include <stdio.h>
#include "echo_layer.h"
int main(void) {
  echo_norm_desc n = {0};
  echo_linear_desc l = {0};
  if (echo_norm_backward_workspace(&n) != ECHO_ERR_SHAPE) return 1; /* hidden 0 */
  n.tokens = 4; n.hidden = 8; n.gate_rows = 3;
  if (echo_norm_backward_workspace(&n) != ECHO_ERR_SHAPE) return 2;
  l.m = 4; l.n = 4; l.k = 4; l.dtype = ECHO_F32;
  if (echo_linear_workspace(&l) != ECHO_ERR_TYPE) return 3;
  l.dtype = ECHO_BF16; l.act = ECHO_ACT_SILU; l.gated = 1;
  if (echo_linear_workspace(&l) < 0 || echo_linear_backward_workspace(&l) <= 0) return 4;
  if (echo_linear(&l, 0, 0, 0, 0, 0, 0, 0, 0, 0) != ECHO_ERR_INVALID_ARGUMENT) return 5;
  l.m = 0;
  if (echo_linear(&l, 0, 0, 0, 0, 0, 0, 0, 0, 0) != ECHO_SUCCESS) return 6;
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


def desc(T=8, H=64, ld_y=0, ld_h=0, G=0, dt=0, sdt=0, post=0, pre=1, scale=1.0, eps=1e-6):
    return B.EchoNormDescC(T, H, ld_y, ld_h, G, dt, sdt, post, pre, scale, eps)


def fwd(d, h=A, y=2 * A, gate=None, w1=None, b1=None, w2=3 * A, b2=None, h_out=4 * A, z=5 * A, stats=None):
    return B.lib.echo_norm(C.byref(d) if d else None, h, y, gate, w1, b1, w2, b2, h_out, z, stats, None)


def test_norm_rejections():
    assert fwd(None) == -1
    for bad in (dict(T=-1), dict(H=0), dict(H=16385), dict(T=(1 << 31) + 1), dict(ld_y=63), dict(ld_h=10),
                dict(G=3), dict(G=-1), dict(eps=-1.0), dict(eps=float("nan"))):
        assert fwd(desc(**bad), gate=6 * A if bad.get("G") else None) == -2, bad
    for bad in (dict(dt=3), dict(sdt=1), dict(dt=2, sdt=0), dict(post=3), dict(pre=-1)):
        assert fwd(desc(**bad)) == -8, bad
    assert fwd(desc(), h=None) == -1
    assert fwd(desc(), z=None) == -1                       # pre norm without its output
    assert fwd(desc(pre=0), w2=None) == -1                 # output without a pre norm
    assert fwd(desc(pre=0), z=None) == -1                  # weight without a pre norm
    assert fwd(desc(), w1=6 * A) == -1                     # weight without a post norm
    assert fwd(desc(G=2)) == -1 and fwd(desc(), gate=6 * A) == -1
    assert fwd(desc(), y=None) == -1                       # h_out without y
    assert fwd(desc(post=1), y=None, h_out=None) == -1
    assert fwd(desc(pre=0), w2=None, z=None, h_out=None) == -1
    for bad in (dict(h=A + 1), dict(y=2 * A + 1), dict(w2=3 * A + 1), dict(z=5 * A + 1), dict(stats=6 * A + 2),
                dict(h_out=4 * A + 1)):
        assert fwd(desc(), **bad) == -3, bad
    assert fwd(desc(sdt=2), h=A + 2) == -3                 # a binary32 stream needs 4 bytes
    assert fwd(desc(), z=A + 64) == -6                     # z over h
    assert fwd(desc(), h_out=A + 2) == -6                  # h_out over h but not equal to it
    assert fwd(desc(), z=4 * A) == -6                      # z over h_out
    assert fwd(desc(), stats=2 * A) == -6
    assert fwd(desc(ld_y=100), z=2 * A + 1500) == -6       # within y's last rows, by its pitch
    assert fwd(desc(T=0), h=None, y=None, h_out=None, z=None) == 0


def bwd(d, dz=A, dh_out=2 * A, h_out=3 * A, y=4 * A, stats=5 * A, gate=None, w1=None, b1=None, w2=6 * A, dh=7 * A,
        dy=8 * A, dgate=None, dw1=None, db1=None, dw2=9 * A, db2=None, ws=10 * A, n=1 << 30):
    return B.lib.echo_norm_backward(C.byref(d) if d else None, dz, dh_out, h_out, y, stats, gate, w1, b1, w2, dh, dy,
                                    dgate, dw1, db1, dw2, db2, ws, n, None)


def test_norm_backward_rejections():
    assert bwd(None) == -1
    assert bwd(desc(H=0)) == -2 and bwd(desc(dt=7)) == -8
    assert bwd(desc(), dh=None) == -1 and bwd(desc(), dz=None) == -1 and bwd(desc(), h_out=None) == -1
    assert bwd(desc(), stats=None) == -1
    assert bwd(desc(post=1), y=None) == -1
    assert bwd(desc(), dw1=11 * A) == -1 and bwd(desc(pre=0), dz=None, w2=None) == -1  # gradients of no norm
    assert bwd(desc(), dgate=11 * A) == -1 and bwd(desc(G=2)) == -1
    assert bwd(desc(G=2), gate=11 * A, dgate=12 * A, y=None) == -1
    assert bwd(desc(), ws=None) == -1
    need = B.echo_norm_backward_workspace(8, 64)
    assert need > 0 and bwd(desc(), n=need - 1) == -9
    assert bwd(desc(), dy=8 * A + 1) == -3 and bwd(desc(), ws=10 * A + 8) == -3
    assert bwd(desc(), dh=A) == -6 and bwd(desc(), dw2=10 * A + 32) == -6 and bwd(desc(), dy=7 * A + 16) == -6
    assert bwd(desc(), dh=2 * A + 2) == -6                 # over dh_out but not equal to it
    assert B.echo_norm_backward_workspace(0, 64) == 0
    with pytest.raises(B.EchoError):
        B.echo_norm_backward_workspace(4, 20000)


def ldesc(m=8, n=16, k=32, ld_x=0, ld_w=0, ld_out=0, ld_r=0, dt=0, act=0, gated=0):
    return B.EchoLinearDescC(m, n, k, ld_x, ld_w, ld_out, ld_r, dt, act, gated, 0)


def lin(d, x=A, w=2 * A, bias=None, residual=None, out=3 * A, p=None, ws=None, n=0):
    return B.lib.echo_linear(C.byref(d) if d else None, x, w, bias, residual, out, p, ws, n, None)


BAD_SHAPES = (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=(1 << 31) + 1), dict(k=(1 << 21) + 1), dict(n=(1 << 21) + 1),
              dict(n=(1 << 20) + 1, gated=1), dict(ld_x=31), dict(ld_w=5), dict(ld_out=15), dict(ld_r=15),
              dict(ld_x=(1 << 21) + 8))
BAD_TYPES = (dict(dt=2), dict(dt=-1), dict(act=5), dict(act=-1), dict(gated=2))


def test_linear_rejections():
    assert lin(None) == -1
    for bad in BAD_SHAPES:
        assert lin(ldesc(**bad)) == -2, bad
        assert B.lib.echo_linear_workspace(C.byref(ldesc(**bad))) == -2
        assert B.lib.echo_linear_backward_workspace(C.byref(ldesc(**bad))) == -2
    for bad in BAD_TYPES:
        assert lin(ldesc(**bad)) == -8, bad
    for name in ("x", "w", "out"):
        assert lin(ldesc(), **{name: None}) == -1, name
    for name in ("x", "w", "bias", "residual", "out", "p"):
        assert lin(ldesc(), **{name: 4 * A + 1}) == -3, name
    assert lin(ldesc(), out=A + 64) == -6 and lin(ldesc(), out=2 * A) == -6 and lin(ldesc(), p=3 * A + 16) == -6
    assert lin(ldesc(), residual=3 * A + 2) == -6          # over out but not equal to it
    assert lin(ldesc(ld_x=100), out=A + 1400) == -6        # within x's last rows, by its pitch
    assert lin(ldesc(m=0), x=None, w=None, out=None) == 0
    assert lin(ldesc(n=0), x=None, w=None, out=None) == 0


def linb(d, dout=A, x=2 * A, w=3 * A, p=None, dx=4 * A, dw=5 * A, db=None, ws=6 * A, n=1 << 30):
    return B.lib.echo_linear_backward(C.byref(d) if d else None, dout, x, w, p, dx, dw, db, ws, n, None)


def test_linear_backward_rejections():
    assert linb(None) == -1
    for bad in BAD_SHAPES:
        assert linb(ldesc(**bad)) == -2, bad
    for bad in BAD_TYPES:
        assert linb(ldesc(**bad)) == -8, bad
    for name in ("dout", "x", "w"):
        assert linb(ldesc(), **{name: None}) == -1, name
    assert linb(ldesc(act=4)) == -1 and linb(ldesc(gated=1)) == -1    # p missing
    need = B.echo_linear_backward_workspace(8, 16, 32, act="silu")
    assert need > 0 and linb(ldesc(act=4), p=7 * A, n=need - 1) == -9 and linb(ldesc(act=4), p=7 * A, ws=None) == -1
    for name in ("dout", "x", "w", "p", "dx", "dw", "db"):
        assert linb(ldesc(act=4), **{"p": 7 * A, name: 8 * A + 1}) == -3, name
    assert linb(ldesc(), ws=6 * A + 8) == -3
    assert linb(ldesc(), dx=A) == -6 and linb(ldesc(), dw=4 * A + 2) == -6 and linb(ldesc(), db=3 * A) == -6
    assert linb(ldesc(act=4), p=7 * A, dx=6 * A) == -6                 # over the workspace


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_workspace_queries_take_empty_and_odd_shapes(act, gated):
    for m in (0, 1, 16, 17, 1000, 1 << 20):
        for n in (0, 1, 7, 8, 384, 1793):
            for k in (0, 1, 7, 64, 1001):
                f = B.echo_linear_workspace(m, n, k, act=act, gated=gated)
                b = B.echo_linear_backward_workspace(m, n, k, act=act, gated=gated)
                assert f >= 0 and b >= 0 and f % 16 == 0 and b % 16 == 0, (m, n, k)


def test_binding_refuses_before_the_library():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.echo_norm(t, t, t, t, stream=0)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        B.echo_norm(t.to(torch.int16), t, t, t, stream=0)
    with pytest.raises(ValueError, match="is not one of"):
        B._code(B.NORMS, "batch", "pre")
    with pytest.raises(ValueError, match="GPU tensor"):
        B.echo_linear(t, t, torch.zeros(4, 4, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        B.echo_linear(t.float(), t.float(), t, stream=0)
    with pytest.raises(ValueError, match="even number of rows"):
        B.echo_linear(t, torch.zeros(5, 64, dtype=torch.bfloat16), t, gated=True, stream=0)
    with pytest.raises(ValueError, match="is not one of"):
        B.echo_linear_workspace(4, 4, 4, act="swish")
