"""How long the product kernel's tail warp waits: it waits in tiles whose segment
ends inside a block of 64 rows only, and such a wait spans all tiles before it (no
GPU needed: the arithmetic is compiled for the host)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_ep_layout_02_gb300", "csrc")

SHIM = r"""
#include "ep_product_wait.h"
extern "C" unsigned long long tile_limit(unsigned long long blocks) { return ep::tile_limit(blocks); }
// the tail warp's walk over a pair's tiles: limits[i] is 0 where it does not wait
extern "C" void walk(const int* rows, int n, unsigned long long* limits) {
    ep::TileWait since;
    for (int i = 0; i < n; ++i) {
        since.enter((rows[i] + 63) / 64);
        limits[i] = 0;
        if (rows[i] % 64 == 0) continue;
        limits[i] = since.limit();
        since.waited();
    }
}
"""
SECOND = 10 ** 9


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    src, lib = str(d / "wait.cpp"), str(d / "wait.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, src, "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.tile_limit.restype, so.tile_limit.argtypes = ctypes.c_ulonglong, [ctypes.c_ulonglong]

    def walk(rows):
        out = (ctypes.c_ulonglong * len(rows))()
        so.walk((ctypes.c_int * len(rows))(*rows), len(rows), out)
        return list(out)
    so.limits = walk
    return so


def test_a_tile_has_a_second_and_two_microseconds_a_block(wait):
    assert wait.tile_limit(0) == SECOND and wait.tile_limit(1 << 25) == SECOND + 2000 * (1 << 25)


@pytest.mark.parametrize("rows", [[64 * 4000] * 1000 + [65], [0] * 20000 + [1], [64] * 5 + [3] + [128] * 7 + [1, 1],
                                  [2 ** 31 - 320] * 13 + [63]])
def test_a_wait_covers_the_tiles_since_the_last_one(wait, rows):
    limits = wait.limits(rows)
    since = 0
    for r, limit in zip(rows, limits):
        # a block of the summed index takes at most 0.4 us, a tile's output at most 20
        since += -(-r // 64) * 400 + 20000
        if limit:
            assert SECOND + since <= limit <= SECOND + 6 * since
            since = 0
        else:
            assert r % 64 == 0
