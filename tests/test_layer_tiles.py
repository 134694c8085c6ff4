"""CPU tests of the map from launch slots to sequence tiles (csrc/kda_seq_tiles.h, compiled here by the host's compiler)
and of the sizes that the entry points derive from it, up to the longest sequence that 32-bit sizes hold."""
import os
import subprocess

import pytest

from gated_delta_rule_52_amd import _lib

CSRC = os.path.join(os.path.dirname(_lib.__file__), "csrc")
LONGEST = 2 ** 31 - 1
F = 1 << 32

PROGRAM = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include "kda_seq_tiles.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace kda;
// reads: packed? L, T, N, and the offsets or nothing; walks every slot and checks that the tiles found are the
// sequences' rows in order, each once, and that a sequence without rows has one slot of no rows
int main(int argc, char **argv) {
    const bool packed = atoi(argv[1]);
    SeqTiles s{nullptr, atoi(argv[4]), atoi(argv[3]), atoi(argv[2])};
    std::vector<int32_t> cu;
    for (int i = 5; i < argc; ++i) cu.push_back(atoi(argv[i]));
    if (packed) s.cu = cu.data();
    int64_t taken = 0, n = -1, k = 0, next = 0, end = 0;
    for (int64_t slot = 0; slot < s.slots(); ++slot) {
        const Tile t = tile_at(s, slot);
        if (!t.valid) continue;
        ++taken;
        if (t.n != n || k == 0) {
            if (next != end) return printf("sequence %lld ends at %lld, not %lld\n", (long long)n, (long long)next, (long long)end), 1;
            if (t.n != n + 1 || t.k != 0) return printf("slot %lld: sequence %d tile %d\n", (long long)slot, t.n, t.k), 1;
            int len;
            s.sequence(t.n, next, len);
            n = t.n, k = 0, end = next + len;
        }
        if (t.k != k || t.begin != next) return printf("slot %lld: tile %d at %lld\n", (long long)slot, t.k, (long long)t.begin), 1;
        if (t.len < 0 || t.len > s.L || (t.len == 0 && end > next)) return printf("slot %lld: %d rows\n", (long long)slot, t.len), 1;
        next += t.len;
        ++k;
        if (t.last() != (next == end) || t.last() != (k >= t.count)) return printf("slot %lld: last\n", (long long)slot), 1;
        if (t.last()) k = 0;
    }
    if (n + 1 != s.N || next != end) return printf("%lld sequences\n", (long long)n + 1), 1;
    printf("%lld %lld\n", (long long)s.slots(), (long long)taken);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    where = tmp_path_factory.mktemp("tiles")
    (where / "walk.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-ftrapv", "-I", CSRC, str(where / "walk.cpp"), "-o", str(where / "walk")])

    def run(L, T, N, offsets=None):
        r = subprocess.run([str(where / "walk"), str(int(offsets is not None)), str(L), str(T), str(N), *map(str, offsets or [])],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stdout
        return [int(v) for v in r.stdout.split()]

    return run


@pytest.mark.parametrize("L", [64, 144, 256])
@pytest.mark.parametrize("offsets", [[0, 0], [0, 1], [0, 5, 5, 5, 200, 201, 201], [7, 300, 300, 301, 557, 700],
                                     [0, 64, 128, 192], [0, 63, 128, 128, 1000, 1000], [3, 259, 515, 516]])
def test_packed_tiles(walk, L, offsets):
    T, N = offsets[-1] + 11, len(offsets) - 1
    slots, taken = walk(L, T, N, offsets)
    assert slots == T // L + N
    assert taken == sum(max(1, -(-(b - a) // L)) for a, b in zip(offsets, offsets[1:]))


@pytest.mark.parametrize("L,T,N", [(1, 0, 3), (64, 64, 5), (64, 65, 4), (144, 1000, 7), (256, 1, 2), (300, 300, 2)])
def test_fixed_tiles(walk, L, T, N):
    assert walk(L, T, N) == [N * max(1, -(-T // L))] * 2


@pytest.mark.parametrize("L", [240, 256])
@pytest.mark.parametrize("T", [LONGEST, 2 ** 31 - 200, 2 ** 31 - 257])
def test_the_longest_sequences(walk, L, T):
    """Lengths at which a length plus a tile passes 32 bits: one sequence, and one behind a short one."""
    tiles = -(-T // L)
    assert walk(L, T, 1) == [tiles, tiles]
    assert walk(L, T, 1, [0, T]) == [T // L + 1, tiles]
    assert walk(L, T, 2, [0, 100, T]) == [T // L + 2, -(-100 // L) + -(-(T - 100) // L)]


def layer(struct, **kw):
    a = struct()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("T", [LONGEST, 2 ** 31 - 256, 2 ** 31 - 257])
@pytest.mark.parametrize("packed", [False, True])
def test_workspaces_of_the_longest_sequences(T, packed):
    """One channel of one state: tiles of 256 tokens, of which each keeps a state and a sum."""
    a = layer(_lib.SelectiveScanArgs, batch=1, num_seqs=1, T=T, dim=1, ds=1, cu_seqlens=F if packed else None)
    slots = T // 256 + 1 if packed else -(-T // 256)
    assert _lib.layer_raw("kda_selective_scan_fwd_workspace_bytes", a) == slots * 2 * 4
    # the gradients at least their stored states of 16 per 8 tokens and each token's share of dB and dC
    if T < LONGEST:
        b = layer(_lib.SelectiveScanBwdArgs, batch=1, num_seqs=1, T=T, dim=1, ds=1, cu_seqlens=F if packed else None)
        need = _lib.layer_raw("kda_selective_scan_bwd_workspace_bytes", b)
        assert (T // 8 * 16 + 2 * T) * 4 < need < 1 << 36


def test_too_many_tiles_are_refused():
    """Two groups of channels take twice the workgroups, more than one launch holds."""
    for struct, name in ((_lib.SelectiveScanArgs, "kda_selective_scan_fwd"), (_lib.SelectiveScanBwdArgs, "kda_selective_scan_bwd")):
        a = layer(struct, batch=1, num_seqs=1, T=LONGEST, dim=65, ds=1)
        assert _lib.layer_raw(name + "_workspace_bytes", a) == 2 ** 64 - 1
        assert _lib.layer_raw(name, a) == _lib.STATUS_CODE["KDA_ERR_UNSUPPORTED"]
        assert b"one launch" in _lib.load().kda_last_error()
