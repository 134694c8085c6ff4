// kda_seq_tiles.h - how sequences are cut into tiles and how a launch slot finds its tile: plain arithmetic that the
// host's checks, the kernels and a program on the CPU share.
#pragma once

#include <cstdint>

namespace kda {

// Sequences cut into tiles of L tokens.  A launch has one slot per possible tile: sequence n's tiles take
// the slots from (start_n / L + n) on.  As ceil(len / L) <= (start + len) / L - start / L + 1 these ranges
// are disjoint, so a slot finds its tile by a binary search over the offsets alone, without a table made
// beforehand; slots that no tile takes end at once.  Offsets are clamped to the rows that exist, so wrong
// ones cannot lead out of the tensors.
struct SeqTiles {
    const int32_t *cu;  // N + 1 offsets, or nullptr: N sequences of T tokens
    int N, T;           // T: per sequence, or all rows with cu
    int L;              // tokens per tile
    __host__ __device__ int64_t rows() const { return cu ? T : static_cast<int64_t>(N) * T; }
    // tiles of a sequence; lengths go up to 2^31 - 1, where len + L - 1 would pass 32 bits
    __host__ __device__ int tiles(int len) const { return len > 0 ? (len - 1) / L + 1 : 0; }
    __host__ __device__ int per_seq() const { return T > L ? tiles(T) : 1; }  // without cu
    __host__ __device__ int64_t slots() const {
        return cu ? static_cast<int64_t>(T) / L + N : static_cast<int64_t>(N) * per_seq();
    }
    __host__ __device__ __forceinline__ int offset(int n) const {
        const int c = cu[n];
        return c < 0 ? 0 : c > T ? T : c;
    }
    __host__ __device__ __forceinline__ void sequence(int n, int64_t &start, int &len) const {
        if (cu) {
            const int s = offset(n), e = offset(n + 1);
            start = s;
            len = e > s ? e - s : 0;
        } else {
            start = static_cast<int64_t>(n) * T;
            len = T;
        }
    }
    __host__ __device__ __forceinline__ int64_t first_slot(int n, int64_t start) const {
        return cu ? start / L + n : static_cast<int64_t>(n) * per_seq();
    }
};

// Tiles of 256 tokens where the rows allow about 1,024 workgroups of `groups` to a tile, down to 64: longer ones
// leave the chip idle, shorter ones spend on the chain what they gain.  Forward, bf16: 16,384 x 4,096 465 us at 256,
// 471 at 128, 495 at 64, 476 at 512; 8,192 x 1,024 82 at 128, 87 at 64 and 256.  At the lower end, in us with tiles of
// 64, 48 and 32 tokens: 8,192 x 512 57, 65, 71 (gradients 133, 148, 158), 4,096 x 512 37, 41, 44 (82, 89, 93), 3,001 x
// 777 fp32 40, 40, 40 (87, 90, 89).  Below about 500 workgroups shorter ones win, which the rule does not follow:
// 2,500 x 515 fp32 32, 29, 30 (70, 62, 63), 2,048 x 256 26, 24, 24 (59, 53, 49), 1,000 x 128 25, 21, 20 (54, 47, 42).
inline void tile_for(SeqTiles &s, int64_t groups) {
    int64_t L = (s.rows() * groups / 1024 + 15) / 16 * 16;
    L = L < 64 ? 64 : L > 256 ? 256 : L;
    if (L < s.T) s.L = static_cast<int>(L);
}

struct Tile {
    int n, k, count;      // sequence, tile within it, tiles of it (0: an empty sequence's only slot)
    int64_t begin;        // first row
    int len;              // rows in the tile
    bool valid;           // false: no tile takes this slot
    __host__ __device__ __forceinline__ bool last() const { return k + 1 >= count; }
};

__host__ __device__ __forceinline__ Tile tile_at(const SeqTiles &s, int64_t slot) {
    Tile t;
    if (s.cu) {
        int lo = 0, hi = s.N - 1;
        while (lo < hi) {  // the last sequence whose first slot is not behind this one
            const int mid = (lo + hi + 1) >> 1;
            if (s.offset(mid) / s.L + static_cast<int64_t>(mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        t.n = lo;
    } else {
        t.n = static_cast<int>(slot / s.per_seq());
    }
    int64_t start;
    int len;
    s.sequence(t.n, start, len);
    t.count = s.tiles(len);
    const int64_t k = slot - s.first_slot(t.n, start);
    t.valid = k >= 0 && k < (t.count > 0 ? t.count : 1);
    t.k = t.valid ? static_cast<int>(k) : 0;
    t.begin = start + static_cast<int64_t>(t.k) * s.L;
    const int left = len - t.k * s.L;
    t.len = left < s.L ? left : s.L;
    return t;
}

}  // namespace kda
