"""CPU test of the cache's page lookup (csrc/kda_latent_pages.h, compiled here by the host's compiler): lengths beyond the
table, pages that do not exist, pages that end inside a tile, slots outside the cache."""
import os
import subprocess

import numpy as np
import pytest

from gated_delta_rule_52_amd import _lib

CSRC = os.path.join(os.path.dirname(_lib.__file__), "csrc")

PROGRAM = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include "kda_latent_pages.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace kda;
int main(int argc, char **argv) {
    std::vector<int32_t> table;
    for (int i = 6; i < argc; ++i) table.push_back(atoi(argv[i]));
    const int n = atoi(argv[1]);
    CachePages p{table.data(), atoi(argv[2]), atoi(argv[3]), atoi(argv[4]), static_cast<int>(atoi(argv[2]))};
    const int rows = p.rows(atoi(argv[5]));
    for (int i = 0; i < rows; ++i) printf("%lld ", (long long)p.row(p.block(n, i), i));
    printf("| %lld %lld %lld %lld\n", (long long)slot_row(-1, 7), (long long)slot_row(7, 7), (long long)slot_row(6, 7),
           (long long)slot_row(2147483647, 2147483647));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("pages")
    (where / "pages.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", CSRC, str(where / "pages.cpp"), "-o", str(where / "pages")])
    return str(where / "pages")


@pytest.mark.parametrize("page", [1, 3, 7, 64])
@pytest.mark.parametrize("length", [-5, 0, 1, 6, 7, 8, 27, 28, 29, 10 ** 6, 2 ** 31 - 1])
def test_rows(program, page, length):
    table = np.array([[0, 1, 2, 3], [5, -1, 2 ** 31 - 1, 4], [9, 10, -2 ** 31, 0]])
    blocks = 10
    for n in range(3):
        out = subprocess.check_output([program, str(n), "4", str(page), str(blocks), str(length), *map(str, table.ravel())], text=True)
        got = [int(w) for w in out.split("|")[0].split()]
        want = []
        for pos in range(max(0, min(length, 4 * page))):
            b = int(table[n, pos // page])
            want.append(b * page + pos % page if 0 <= b < blocks else -1)
        assert got == want
        assert out.split("|")[1].split() == ["-1", "-1", "6", "-1"]


def test_large_caches(program):
    """Rows past 2^31 bytes and blocks near the largest number."""
    out = subprocess.check_output([program, "0", "1", "64", "33554431", "3", "33554430"], text=True)
    assert [int(w) for w in out.split("|")[0].split()] == [33554430 * 64 + i for i in range(3)]
