// kda_latent_pages.h - where a sequence's rows lie in the paged cache: plain arithmetic that the kernels and a program on
// the CPU share.
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

}  // namespace kda
