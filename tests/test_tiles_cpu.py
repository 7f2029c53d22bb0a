"""The row ranges and tile counts of the grouped product (csrc/qsw_tiles.h), on the
CPU: whatever an offset table holds, the tiles that the kernel counts from it
fit in the records that the host reserved from the sizes alone."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_swiglu_mlp_gb300", "csrc")

# The group table as the kernel builds it, from the same functions.
SOURCE = r"""
#include "qsw_tiles.h"
using namespace qsw;

// table[groups + 1]; returns the number of tiles
extern "C" int64_t count_tiles(const int *offsets, int groups, int rows, int max_group, int bt, int n_tiles, int *table) {
  int top = 0;
  int64_t total = 0;
  for (int e = 0; e < groups; ++e) {
    const int lo = raised_offset(offsets[e], top, rows), hi = raised_offset(offsets[e + 1], lo, rows);
    table[e] = lo;
    table[e + 1] = hi;
    total += static_cast<int64_t>(token_tiles(hi - lo < max_group ? hi - lo : max_group, bt)) * n_tiles;
    top = lo;
  }
  return total;
}
extern "C" int64_t most(int rows, int groups, int bt, int n_tiles) { return most_tiles(rows, groups, bt, n_tiles); }
extern "C" void plan(int64_t most, int sms, int unit, int64_t *slots, int64_t *recs) {
  const TilePlan t = plan_tiles(most, sms, unit);
  *slots = t.slots;
  *recs = t.recs;
}
extern "C" int mine(int total, int slot, int slots) { return tiles_of(total, slot, slots); }
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text(SOURCE)
    lib = str(d / "tiles.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I", CSRC,
                    str(d / "tiles.cpp"), "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.count_tiles.restype = so.most.restype = ctypes.c_int64
    so.plan.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64),
                        ctypes.POINTER(ctypes.c_int64)]
    return so


def raised(offsets, rows):
    """The table as documented: within [0, rows], no less than any entry before."""
    out, top = [], 0
    for v in offsets:
        top = max(top, min(max(v, 0), rows))
        out.append(top)
    return out


def check(so, offsets, rows, n_tiles, unit=1, sms=152, max_group=None):
    groups = len(offsets) - 1
    max_group = min(rows, max_group or rows)
    for bt in ([192] if max_group >= 192 else sorted({(max_group + 15) // 16 * 16, (max_group + 31) // 32 * 32})):
        table = (ctypes.c_int * (groups + 1))()
        total = so.count_tiles((ctypes.c_int * (groups + 1))(*offsets), groups, rows, max_group, bt, n_tiles, table)
        table = list(table)
        assert table == raised(offsets, rows)
        most = so.most(rows, groups, bt, n_tiles)
        assert total <= most, (offsets, rows, bt)
        slots, recs = ctypes.c_int64(), ctypes.c_int64()
        so.plan(most, sms, unit, slots, recs)
        slots, recs = slots.value, recs.value
        assert 1 <= recs <= 256 and slots >= 1
        counts = [so.mine(total, s, slots) for s in sorted({0, 1, slots // 2, slots - 1}) if 0 <= s < slots]
        assert max(counts) <= recs
        # a tile split over a cluster is the cluster's only one (its partial sums take the stages' space)
        if most * unit <= sms:
            assert recs == 1


@pytest.mark.parametrize("offsets,rows,n_tiles", [
    ([0, 2] * 32 + [0], 2, 1), ([0, 8192] * 32 + [0], 8192, 16), ([0, 8192] * 16 + [0], 8192, 8),
    ([8192] + [0] * 40, 8192, 16), (list(range(50, -1, -1)), 50, 3), ([-5, 900, 7, -1, 30], 50, 1), ([0] * 65, 10, 1),
    ([2 ** 31 - 1, -2 ** 31] * 3, 1 << 30, 1), ([0, 1 << 30], 1 << 30, 2),
])
def test_backward_tables(tiles, offsets, rows, n_tiles):
    for unit in (1, 2, 4):
        check(tiles, offsets, rows, n_tiles, unit)


def test_random_tables(tiles):
    rng = random.Random(7)
    for _ in range(4000):
        groups, rows = rng.choice([1, 2, 3, 8, 31, 32, 33, 64, 200, 1024]), rng.choice([1, 2, 15, 16, 191, 192, 193, 1000, 8192])
        kind = rng.randrange(4)
        if kind == 0:       # ascending
            off = sorted(rng.randint(0, rows) for _ in range(groups + 1))
        elif kind == 1:     # anything
            off = [rng.randint(-rows, 2 * rows) for _ in range(groups + 1)]
        elif kind == 2:     # alternating
            off = [(e & 1) * rng.randint(rows // 2, rows) for e in range(groups + 1)]
        else:               # descending
            off = sorted((rng.randint(0, rows) for _ in range(groups + 1)), reverse=True)
        check(tiles, off, rows, rng.choice([1, 2, 16, 57]), rng.choice([1, 2, 4]),
              max_group=rng.choice([None, 1, 12, 100, 230]))
