"""Which tile a block works on (csrc/grid_map.h), walked on the host over whole grids:
every tile is taken once and no block takes one that does not exist, also the blocks
that a grid of more than 2^20 is rounded up by."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_block_quantized_group_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
GRID = 1 << 20                             # blocks of a row of the grid


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("grid") / "walk")
    subprocess.run(["g++", "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-I",
                    os.path.join(ROCM, "include"),
                    os.path.join(HERE, "host", "grid_map_walk.cpp"), "-o", exe], check=True)

    def run(*args, want="ok\n"):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0 and r.stdout == want, (args, r.stdout, r.stderr)
    return run


@pytest.mark.parametrize("per,E", [
    (1, 1), (7, 3), (8, 5), (9, 1024), (33, 60), (1024, 1023), (1023, 1024), (1024, 1024),
    (1025, 1024), (1032, 1016), (GRID, 1), (GRID - 8, 1), (GRID + 1, 1),
    (3 * 342, 1024),                       # fp32, 2 x 21825 by 257, 128 x 128 tiles
    (32 * 33, 1000),                       # fp32, 4096 by 4224
    (2500, 1024)])
def test_tiles_of_every_expert(walk, per, E):
    walk("experts", per, E)


@pytest.mark.parametrize("launched,live", [
    (1, 1), (1, 0), (9, 3), (64, 64), (1000, 999), (GRID - 1, GRID - 1), (GRID, GRID),
    (GRID, GRID - 9), (GRID + 1, GRID + 1), (GRID + 1, 77), (GRID + 1, 0),
    (2 * GRID + 5, 2 * GRID - 3), (3 * GRID, 3 * GRID)])
def test_tiles_of_sorted_rows(walk, launched, live):
    """live of them on the device, where the host launched for the most there can be."""
    walk("tiles", launched, live)


@pytest.mark.parametrize("tile", [16, 64, 256])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 256, 257, (1 << 31) - 256, (1 << 31) - 255,
                                  (1 << 31) - 1])
def test_tiles_of_rows(walk, rows, tile):
    one = -(-rows // tile)
    walk("rows", rows, tile, want=f"{one} {one} {rows // tile + min(rows, 1024)}\n")
