"""The rule that chooses a product's tile, splits and grid (host arithmetic only,
compiled with g++; no GPU and no launch): every shape the header allows has a grid
that can be launched, and shapes past it are refused by the queries and the calls."""
import ctypes as C
import os
import subprocess

import pytest

from error_compensated_bit_echo_amd import binding as B
from linear_tile_cases import CASES, TILES, product_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "error_compensated_bit_echo_amd", "csrc"),
                    os.path.join(ROOT, "tests", "linear_plan_check.cc"), "-o", exe], check=True)
    return exe


def test_grids_within_limits_at_every_allowed_size(plan):
    r = subprocess.run([plan, "limits"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "linear plans ok" in r.stdout


def test_products_past_the_limit_are_refused_everywhere():
    A = 1 << 32  # fake addresses: every call below is rejected
    for m, n, k, gated in ((1 << 31, 1 << 12, 8, 0), (1 << 31, 8, 1 << 12, 0), ((1 << 31), 1 << 10, 8, 1), ((1 << 22), (1 << 20) + 1, 1, 0)):
        d = B.EchoLinearDescC(m, n, k, 0, 0, 0, 0, 0, 0, gated, 0)
        over = m * (2 * n if gated else n) > 1 << 42 or m * k > 1 << 42
        assert (B.lib.echo_linear_workspace(C.byref(d)) == -2) == over, (m, n, k)
        assert (B.lib.echo_linear_backward_workspace(C.byref(d)) == -2) == over, (m, n, k)
        if over:
            assert B.lib.echo_linear(C.byref(d), A, 2 * A, None, None, 3 * A, None, 4 * A, 1 << 30, None) == -2
            assert B.lib.echo_linear_backward(C.byref(d), A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, None, 7 * A, 1 << 60, None) == -2


def test_long_products_have_a_workspace_answer():
    """m to the header's limit, over the shapes whose small tiles pass one grid dimension"""
    for m in ((1 << 29) - 1, 1 << 29, 600_000_000, 1 << 30, 1 << 31):
        for n, k in ((1, 1), (8, 8), (8, 64), (64, 7), (128, 8)):
            assert B.echo_linear_workspace(m, n, k) >= 0 and B.echo_linear_backward_workspace(m, n, k) >= 0


@pytest.mark.parametrize("name", list(CASES))
def test_shapes_of_the_tile_tests_take_their_tiles(plan, name):
    """tests/test_gpu_linear_tiles.py runs the large tiles as long as this holds"""
    case = CASES[name]
    r = subprocess.run([plan, "choose", *map(str, product_of(case)), "1"], capture_output=True, text=True, check=True)
    tile, splits = map(int, r.stdout.split())
    assert tile == TILES[case[6]] and (splits > 1) == case[7], (tile, splits)


def test_odd_rows_of_the_tile_tests_are_copied():
    """the forward case of odd rows reaches its tile through copies with whole rows"""
    m, n, k, act, gated = CASES["out 256 copied rows"][:5]
    assert B.echo_linear_workspace(m, n, k, act=act, gated=gated) >= 2 * (m + n) * ((k + 7) // 8 * 8)
