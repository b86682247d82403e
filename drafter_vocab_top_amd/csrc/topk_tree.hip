// The tree of a round's drafts, for gfx950: each column's ancestors as a mask,
// and its position.
//
// One wave per lane, 64 columns at a time.  Within the 64, ancestors are found
// by pointer doubling: after r steps a column knows its 2^r nearest and the one
// 2^r above, so a chain of 64 takes 6 steps instead of 63.  A column whose
// line leaves the 64 goes on with the row of the ancestor where it does, which
// is complete by then (parents come before their children).  A chain of latencies:
// one lane of 8 columns 1.6 us, 512 lanes of up to 64 columns 2.8.
#include "topk_cache.hpp"

namespace topk {

namespace {

__device__ __forceinline__ int32_t from_lane(int32_t x, int32_t lane) { return __builtin_amdgcn_ds_bpermute(lane << 2, x); }

__global__ __launch_bounds__(64) void tree_kernel(TreeArgs a) {
    const uint32_t l = blockIdx.x;
    const int32_t lane = (int32_t)threadIdx.x;
    uint32_t cb, ce;
    a.cols.range(l, cb, ce);
    const uint32_t n = ce - cb;
    if (n == 0) return;
    const int32_t len = a.lens ? max_i32(a.lens[l], 0) : 0;
    for (uint32_t base = 0; base < n; base += 64) {
        const uint32_t j = base + (uint32_t)lane;
        const int32_t parent = a.parents[cb + min_u32(j, n - 1u)];
        const bool child = j < n && parent >= 0 && (uint32_t)parent < j;
        int32_t up = child && (uint32_t)parent >= base ? parent - (int32_t)base : -1;  // among the 64
        int32_t out = child && (uint32_t)parent < base ? parent : -1;                  // before them
        uint32_t lo = lane < 32 ? 1u << lane : 0u, hi = lane < 32 ? 0u : 1u << (lane - 32);
        while (__ballot(up >= 0)) {
            const int32_t from = up >= 0 ? up : lane;
            lo |= (uint32_t)from_lane((int32_t)lo, from);
            hi |= (uint32_t)from_lane((int32_t)hi, from);
            const int32_t above_out = from_lane(out, from), above = from_lane(up, from);
            if (up >= 0) {
                out = above_out;
                up = above;
            }
        }
        if (j < n) {
            uint32_t* row = a.mask + (int64_t)(cb + j) * a.mask_ld;
            const uint32_t* before = a.mask + (int64_t)(cb + (uint32_t)max_i32(out, 0)) * a.mask_ld;
            const int64_t w0 = base >> 5;
            for (int64_t w = 0; w < w0 && w < a.mask_ld; ++w) row[w] = out >= 0 ? before[w] : 0u;
            if (w0 < a.mask_ld) row[w0] = lo;
            if (w0 + 1 < a.mask_ld) row[w0 + 1] = hi;
            for (int64_t w = w0 + 2; w < a.mask_ld; ++w) row[w] = 0u;
            const int32_t inside = (int32_t)(__builtin_popcount(lo) + __builtin_popcount(hi));  // with itself
            const int32_t first = out >= 0 ? a.positions[cb + (uint32_t)out] + 1 : len;
            a.positions[cb + j] = first + inside - 1;
        }
        __syncthreads();  // the next 64 read these rows
    }
}

}  // namespace

hipError_t launch_tree(const TreeArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(tree_kernel, dim3(a.lanes), dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
