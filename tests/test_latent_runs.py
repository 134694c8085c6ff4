"""CPU test of how the tiles of all sequences are shared out over workgroups (csrc/kda_latent_pages.h, compiled here by the
host's compiler, which ends the program where an int passes its range): up to the most tiles that a call may have."""
import os
import subprocess

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
using namespace kda;
int main(int argc, char **argv) {
    const int total = atoi(argv[1]), splits = atoi(argv[2]);
    for (int w = 0; w < splits; ++w) {
        const TileRun r(total, splits, w);
        printf("%d %d %d\n", r.run, r.begin, r.left);
    }
    printf("%d %d\n", pieces(total, 16), pieces(total, 2147483647));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("runs")
    (where / "runs.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", CSRC, str(where / "runs.cpp"), "-o", str(where / "runs")])
    return str(where / "runs")


# 2,147,483,646: 1,386 sequences of 24,790,576 rows in tiles of 16
@pytest.mark.parametrize("total", [0, 1, 5, 511, 512, 513, 1000, 10 ** 6 + 3, 2147483646, 2147483647])
@pytest.mark.parametrize("splits", [1, 2, 3, 128, 512])
def test_runs_cover_every_tile_once(program, total, splits):
    lines = subprocess.check_output([program, str(total), str(splits)], text=True).split("\n")
    at, want = 0, max(1, -(-total // splits))
    for line in lines[:splits]:
        run, begin, left = map(int, line.split())
        assert run == want and begin == at and left == min(run, total - at)
        at += left
    assert at == total
    assert lines[splits] == f"{-(-total // 16)} {min(total, 1)}"
