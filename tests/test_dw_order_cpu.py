"""The order of dw's tiles (csrc/dw_order.h, compiled for the host): every tile of every group and split once, and none of the
device's eight XCDs, which take every eighth workgroup, without work while others have some to spare."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_vector_quantised_amd", "csrc")
SOURCE = r"""
#include "dw_order.h"
extern "C" long order(int tiles, int groups, int splits, int side, int *tiles_of_xcd, int *seen) {
  const int shift = mvq::dw_parts_shift(tiles, (long)groups * splits, side);
  const long n = mvq::dw_workgroups(tiles, (long)groups * splits, shift);
  for (long b = 0; b < n; ++b) {
    const mvq::DwPlace p = mvq::dw_place((int)b, tiles, groups, shift);
    if (p.split >= splits || p.tile >= tiles) continue;
    if (p.split < 0 || p.group < 0 || p.group >= groups || p.tile < 0) return -1;
    ++tiles_of_xcd[b & 7];
    ++seen[((long)p.split * groups + p.group) * tiles + p.tile];
  }
  return n;
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    folder = tmp_path_factory.mktemp("order")
    (folder / "order.cpp").write_text(SOURCE)
    lib = str(folder / "liborder.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(folder / "order.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).order
    f.restype = ctypes.c_long

    def run(tiles, groups, splits, side):
        xcd, seen = (ctypes.c_int * 8)(), (ctypes.c_int * (tiles * groups * splits))()
        n = f(tiles, groups, splits, side, xcd, seen)
        assert list(seen) == [1] * len(seen), (tiles, groups, splits, side)
        return n, list(xcd)

    return run


@pytest.mark.parametrize("side", [64, 128, 256])
def test_every_tile_once(order, side):
    for tiles in (1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 36, 63, 64, 65, 100, 127, 128, 129, 448, 1000):
        for groups in (1, 2, 3, 5, 8, 16, 33):
            for splits in (1, 2, 4, 8, 16, 32):
                if tiles * groups * splits > 40000:
                    continue
                n, _ = order(tiles, groups, splits, side)
                # sets in at most 8 parts p, rounded up to 8 parts in all, of tiles / p rounded up:
                # (p sets + 7) (tiles / p + 1) workgroups
                sets = groups * splits
                assert n % 8 == 0 and n <= tiles * sets + 8 * sets + 7 * tiles + 7


@pytest.mark.parametrize("tiles,groups,splits,side", [
    (1, 1, 32, 64),    # 65536 rows of 64 -> 64
    (2, 1, 32, 64),    # 32768 rows of 128 -> 64
    (9, 1, 16, 64),    # 16384 rows of 192 -> 192
    (9, 1, 32, 64), (4, 1, 16, 128), (16, 1, 8, 128), (36, 1, 4, 64), (25, 1, 4, 64), (1, 8, 8, 64), (4, 4, 16, 64), (64, 1, 1, 64)])
def test_all_xcds_work_on_split_contractions(order, tiles, groups, splits, side):
    """A few tiles in parts: every XCD has its share of them, up to one set's part."""
    _, xcd = order(tiles, groups, splits, side)
    share = tiles * groups * splits / 8
    assert min(xcd) > 0 and max(xcd) <= share + max(1, tiles / 8), xcd
