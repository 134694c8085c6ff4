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
    // the cache row of a sequence's row `pos` < rows(length), -1 on a block that does not exist
    __host__ __device__ __forceinline__ int64_t at(int64_t sequence, int pos) const {
        const unsigned p = static_cast<unsigned>(pos), block = p / static_cast<unsigned>(page);
        const int b = table[sequence * stride + block];
        if (b < 0 || b >= num_blocks) return -1;
        return static_cast<int64_t>(b) * page + (p - block * static_cast<unsigned>(page));
    }
};

// The cache row that a slot names, -1 for none.
__host__ __device__ __forceinline__ int64_t slot_row(int32_t slot, int64_t cache_rows) {
    return slot >= 0 && slot < cache_rows ? slot : -1;
}

}  // namespace kda
