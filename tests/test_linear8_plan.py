"""The shapes of the tile tests take the tiles that they are meant for (host arithmetic,
g++): tests/test_gpu_linear8_tiles.py runs every tile as long as this holds."""
import os
import subprocess

import pytest

from linear8_tile_cases import CASES, TILES, product_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan8") / "linear8_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "error_compensated_bit_echo_amd", "csrc"),
                    os.path.join(ROOT, "tests", "linear8_plan_check.cc"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("name", list(CASES))
def test_shapes_of_the_tile_tests_take_their_tiles(plan, name):
    case = CASES[name]
    r = subprocess.run([plan, *map(str, product_of(case))], capture_output=True, text=True, check=True)
    tile, splits, alone = map(int, r.stdout.split())
    assert (tile, splits > 1, bool(alone)) == (TILES[case[6]], case[7], case[8]), (tile, splits, alone)
