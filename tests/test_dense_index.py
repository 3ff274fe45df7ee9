"""The tiled products' addresses (CPU): each lane's loads, replayed on the host from the kernels' own arithmetic."""
import ctypes
import os
import shutil
import subprocess

import pytest

from combine_expert_histogram_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
WRONG = {1: "reads outside the rows", 2: "is cut short", 3: "brings another piece", 4: "misses a piece", 5: "reads past its part"}


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    out = str(tmp_path_factory.mktemp("index") / "index.so")
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{build.CSRC}", os.path.join(HERE, "dense_index_check.cpp"),
                    "-o", out], check=True)
    return ctypes.CDLL(out)


# rows of the operand, its K (with K across, the rows of memory): whole tiles, ragged ones, less than a tile, less than a load
SIZES = [(256, 64), (512, 200), (264, 65), (2056, 2049), (392, 777), (8, 65), (680, 3), (8, 1), (72, 127), (136, 66), (1000, 131)]


@pytest.mark.parametrize("gap", [0, 8, 40])
@pytest.mark.parametrize("width", [64, 128, 256])
@pytest.mark.parametrize("rows,K", SIZES)
def test_no_load_leaves_its_rows(index, rows, K, width, gap):
    """Elements between the rows and behind the last one are not read; every element of the operand is, to its place."""
    for kper in (64, 128, 4096):
        bad = index.check_loads(width, 1, rows, K, rows + gap, kper)
        assert not bad, f"K across, parts of {kper}: a load {WRONG[bad]}"
        # K along the rows: whole chunks of it, any number of rows
        bad = index.check_loads(width, 0, K, rows, rows + gap, kper)
        assert not bad, f"K along, parts of {kper}: a load {WRONG[bad]}"


def taken(index, total, dw, grid, ahead):
    counts = (ctypes.c_int * total)()
    index.count_tiles(total, dw, grid, ahead, counts)
    return set(counts)


def test_every_tile_is_taken_once(index):
    """By launches of as many workgroups as the host chooses, one and two to a CU."""
    for total in [*range(1, 300), 448, 511, 512, 513, 1000, 2047, 4097]:
        for most in (256, 512):
            grid = min((total + 7) // 8 * 8, most)
            assert taken(index, total, 0, grid, 0) == {1}, (total, grid)


def test_every_tile_of_a_joint_launch_is_taken_once(index):
    """The second product's, behind any number of the first's: whole rounds, short runs on the last XCDs, few tiles."""
    for dw in [1, 7, 8, 9, 100, 145, 255, 256, 257, 297, 448, 493, 512, 561, 1000]:
        assert taken(index, dw, 0, 256, 0) == {1}
        for dx in [1, 5, 63, 64, 65, 145, 255, 256, 391, 493, 495, 1023, 2145]:
            for ahead in (1, 2, 3, 4, 11, 100):
                assert taken(index, dx, dw, 256, ahead) == {1}, (dw, dx, ahead)
