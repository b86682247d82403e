// Trees of drafts and the paged cache: launch arguments and entry points of
// their kernels, and what the kernels share.
#pragma once

#include "topk_cols.h"

#include "topk_round.hpp"

namespace topk {

struct TreeArgs {
    uint32_t lanes;
    Parts cols;
    const int32_t *parents, *lens;  // lens NULL: 0
    uint32_t* mask;
    int64_t mask_ld;
    int32_t* positions;
};
hipError_t launch_tree(const TreeArgs& a, hipStream_t stream);

struct VerifyTreeArgs {
    topk_verify_tree_args v;
    Parts cols;
};
hipError_t launch_verify_tree(const VerifyTreeArgs& a, hipStream_t stream);

// x / d for x < 2^31 and 1 <= d < 2^31 by a product: with s = ceil(log2 d),
// m = floor(2^32 (2^s - d) / d) + 1 and h the upper half of m x,
// x / d = (h + x) >> s (Granlund and Montgomery, 1994); h + x < 2^32.
struct Divisor {
    uint32_t d, m, s;
    static Divisor of(uint32_t d) {
        Divisor v = {d, 1u, 0u};
        while (((uint64_t)1 << v.s) < d) ++v.s;
        v.m = (uint32_t)(((uint64_t)1 << 32) * (((uint64_t)1 << v.s) - d) / d + 1);
        return v;
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return (__umulhi(m, x) + x) >> s; }
};

// The cache, with what its addresses need.
struct Cache {
    topk_cache c;
    Divisor block;
    // Strides in 16 bytes, and of the scales in bytes: no offset of a row's parts passes 32 bits then (the last slot's row
    // ends within 64 GiB of the layer's start, its scale within 4).
    uint32_t block16, slot16, scale_block, scale_slot;
    // Offset of slot r of block b (its first head), in 16 bytes; and of its scale.
    __device__ __forceinline__ uint32_t row16(uint32_t b, uint32_t r) const { return b * block16 + r * slot16; }
    __device__ __forceinline__ uint32_t scale_row(uint32_t b, uint32_t r) const { return b * scale_block + r * scale_slot; }
};

template <class T>
__device__ __forceinline__ T* past16(T* base, uint32_t offset16) {
    return reinterpret_cast<T*>(const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(base)) + ((uint64_t)offset16 << 4));
}

struct CacheWriteArgs {
    Cache cache;  // of the layer
    topk_cache_write_args w;
};
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t stream);

struct CacheMoveArgs {
    Cache cache;
    uint32_t lanes, width;
    const int32_t *lens, *table, *columns;
    int64_t table_ld;
};
hipError_t launch_cache_move(const CacheMoveArgs& a, hipStream_t stream);

struct AttendArgs {
    Cache cache;  // of the layer
    topk_attend_args a;
    Parts cols;
    uint32_t places;  // of a table's row, at most 2^31 - 1
};
hipError_t launch_attend(const AttendArgs& a, hipStream_t stream);
int64_t attend_workspace(const AttendArgs& a);

}  // namespace topk
