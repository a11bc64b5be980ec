"""The shapes of the ring tests take the tiles and steps that they are meant for (host
arithmetic, g++): tests/test_gpu_linear8_rings.py goes around every ring as long as this
holds."""
import os
import subprocess

import pytest

from linear8_ring_cases import CASES
from linear8_tile_cases import TILES, product_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("steps8") / "linear8_steps_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "error_compensated_bit_echo_amd", "csrc"),
                    os.path.join(ROOT, "tests", "linear8_steps_check.cc"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("name", list(CASES))
def test_shapes_of_the_ring_tests_go_around(plan, name):
    case = CASES[name]
    r = subprocess.run([plan, *map(str, product_of(case))], capture_output=True, text=True, check=True)
    tile, split, steps, fours, alone = map(int, r.stdout.split())
    assert (tile, bool(split), steps, bool(fours), bool(alone)) == (TILES[case[6]], *case[7:]), r.stdout
    assert steps > 8 and case[2] % 16


def test_every_ring_is_gone_around():
    """of one set of wavefronts: 256, and the others where they are not alone"""
    seen = {(c[6], c[4], c[9], c[5] != "pow2") for c in CASES.values() if c[6] == "256" or not c[10]}
    for gated in (False, True):
        assert {("256", gated, f, o) for f, o in ((True, False), (True, True), (False, True))} <= seen
        assert ("128", gated, True, True) in seen and ("64", gated, True, True) in seen
