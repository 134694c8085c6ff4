// kda_latent_pages.h - where a sequence's rows lie in the paged cache, and how tiles of rows are shared out over workgroups:
// plain arithmetic that the kernels and a program on the CPU share.
#pragma once

#include <cstdint>

namespace kda {

struct CachePages {
    const int32_t *table;  // [sequences, max_blocks], stride apart
    int64_t stride;
    int page, num_blocks, max_blocks;
    // a sequence's length as far as its table reaches
    __host__ __device__ __forceinline__ int rows(int length) const {
        const int64_t room = static_cast<int64_t>(max_blocks) * page;
        return length <= 0 ? 0 : length < room ? length : static_cast<int>(room);
    }
    // the block of a sequence's row `pos` < rows(length)
    __host__ __device__ __forceinline__ int block(int64_t sequence, int pos) const {
        return table[sequence * stride + static_cast<unsigned>(pos) / static_cast<unsigned>(page)];
    }
    // the cache row of row `pos` of a sequence on that block, -1 where there is no such block
    __host__ __device__ __forceinline__ int64_t row(int block, int pos) const {
        if (block < 0 || block >= num_blocks) return -1;
        return static_cast<int64_t>(block) * page + static_cast<unsigned>(pos) % static_cast<unsigned>(page);
    }
};

// The cache row that a slot names, -1 for none.
__host__ __device__ __forceinline__ int64_t slot_row(int32_t slot, int64_t cache_rows) {
    return slot >= 0 && slot < cache_rows ? slot : -1;
}

// n in pieces of d, the last one smaller: n goes up to 2^31 - 1, where n + d - 1 would pass 32 bits.
__host__ __device__ __forceinline__ int pieces(int n, int d) { return n > 0 ? (n - 1) / d + 1 : 0; }

// Workgroup w's part of `total` tiles that `splits` workgroups share out evenly: the first `begin` lie in front of it.
struct TileRun {
    int run;          // tiles in a whole part
    int begin, left;  // left: tiles in this one
    __host__ __device__ __forceinline__ TileRun(int total, int splits, int w) : run(total > 0 ? pieces(total, splits) : 1) {
        const int64_t at = static_cast<int64_t>(w) * run;
        begin = at < total ? static_cast<int>(at) : total;
        left = total - begin < run ? total - begin : run;
    }
};

}  // namespace kda
