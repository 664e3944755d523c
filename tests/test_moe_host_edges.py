"""The arithmetic of the grouped products' tiles (csrc/moe_tiles.h, which the kernels use) on the host: whatever a
plan's offsets hold, an item's tile is a cell of the workspace."""
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_q4_q8_gb300", "csrc")

# The kernels' prefix sums, 32 experts at a time, then every item.  Prints the tiles of the workspace, those of the plan, the
# largest cell, whether a sum left 32 bits, the cells that a (tile of outputs) met other than once, and rows outside an expert's.
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "moe_tiles.h"
int main(int argc, char **argv)
{
    const int columns = atoi(argv[1]), n_pairs = atoi(argv[2]), row_tiles = atoi(argv[3]), experts = argc - 5;
    std::vector<int> off, cum(experts + 1);
    for (int i = 4; i < argc; ++i) off.push_back(atoi(argv[i]));
    const int64_t most = rz::moe_most_tiles(n_pairs, experts, columns);
    int base = 0;
    bool wrapped = false;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        int v = 0;
        for (int e = e0; e < e0 + 32 && e < experts; ++e) {
            const int own = rz::moe_expert_tiles(off[e], off[e + 1], n_pairs, columns);
            int sum;
            wrapped |= __builtin_add_overflow(v, own, &v) || __builtin_add_overflow(base, v, &sum);
            cum[e] = rz::moe_cut(base + v - own, static_cast<int>(most));
        }
        base = rz::moe_cut(base + v, static_cast<int>(most));
    }
    cum[experts] = base;
    std::vector<int> met(most, 0);
    int64_t top = -1, odd = 0, outside = 0;
    for (int64_t it = 0; it < static_cast<int64_t>(base) * row_tiles; ++it) {
        const rz::MoeItem m = rz::moe_item(it, row_tiles, cum.data(), experts);
        const int64_t cell = static_cast<int64_t>(cum[m.expert]) + m.tile;
        if (cell > top) top = cell;
        if (cell >= 0 && cell < most) ++met[cell];
        outside += m.tile < 0 || m.row_tile < 0 || m.row_tile >= row_tiles || off[m.expert] < 0 ||
                   off[m.expert] + static_cast<int64_t>(m.tile) * columns >= off[m.expert + 1] || off[m.expert + 1] > n_pairs;
    }
    for (int64_t i = 0; i < base; ++i) odd += met[i] != row_tiles;
    printf("%lld %d %lld %d %lld %lld\n", (long long)most, base, (long long)top, (int)wrapped, (long long)odd, (long long)outside);
}
"""


@pytest.fixture(scope="module")
def items(tmp_path_factory):
    gxx = shutil.which("g++") or pytest.skip("no g++")
    at = tmp_path_factory.mktemp("tiles")
    (at / "items.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "items.cpp"), "-o", str(at / "items")], check=True)

    def run(columns, n_pairs, row_tiles, offsets):
        r = subprocess.run([str(at / "items"), *map(str, [columns, n_pairs, row_tiles, *offsets])], check=True, capture_output=True, text=True, timeout=120)
        return dict(zip(("most", "tiles", "top", "wrapped", "odd", "outside"), map(int, r.stdout.split())))

    return run


def bad_offsets(kind, n, E):
    rng = np.random.default_rng(E + n)
    return {
        "overlapping": [0, n] * (E // 2) + [0] * (1 + E % 2),
        "all in the last": [0] * E + [n],
        "decreasing": list(range(E, -1, -1)),
        "outside": [-5, n + 1] * (E // 2) + [2 ** 31 - 1] * (1 + E % 2),
        "far outside": [-2 ** 31, 2 ** 31 - 1] * (E // 2) + [-2 ** 31] * (1 + E % 2),
        "random": rng.integers(-n // 4, n + n // 4 + 2, E + 1).tolist(),
    }[kind]


@pytest.mark.parametrize("kind", ["overlapping", "all in the last", "decreasing", "outside", "far outside", "random"])
@pytest.mark.parametrize("columns,n,E,row_tiles", [(128, 8192, 8, 112), (128, 8192, 8, 1), (128, 1536, 8, 3), (32, 400, 8, 18), (32, 399, 33, 2),
                                                   (16, 65, 64, 5), (16, 1, 1, 1), (16, 500, 512, 7)])
def test_items_of_bad_offsets_stay_in_the_workspace(items, kind, columns, n, E, row_tiles):
    got = items(columns, n, row_tiles, bad_offsets(kind, n, E))
    assert not got["wrapped"] and not got["outside"] and not got["odd"], got
    assert got["tiles"] <= got["most"] and got["top"] == got["tiles"] - 1, got


def test_sums_of_tiles_do_not_wrap(items):
    n = 1 << 27
    for E in (512, 33):  # 2^23 tiles of 16 rows for every other expert
        got = items(16, n, 2, bad_offsets("overlapping", n, E))
        assert not got["wrapped"] and not got["outside"] and got["tiles"] == got["most"] and got["top"] == got["most"] - 1, got


@pytest.mark.parametrize("columns", [16, 32, 128])
@pytest.mark.parametrize("n,E", [(1, 1), (7, 8), (500, 8), (4097, 64), (1000, 512)])
def test_items_of_a_plan_are_its_tiles(items, columns, n, E):
    rng = np.random.default_rng(n + E)
    for live in (n, n // 2, 0):
        rows = rng.multinomial(live, rng.dirichlet(np.full(E, 0.3)))
        got = items(columns, n, 3, np.concatenate([[0], np.cumsum(rows)]).tolist())
        assert got["tiles"] == int((-(-rows // columns)).sum()) and got["top"] == got["tiles"] - 1
        assert not got["odd"] and not got["outside"] and not got["wrapped"]
