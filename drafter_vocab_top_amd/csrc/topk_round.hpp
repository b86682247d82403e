// The steps around the top-k in a round: launch arguments and entry points
// of their kernels, and what the kernels share.
#pragma once

#include "topk_cols.h"

#include "topk_device.hpp"

namespace topk {

// An address that can be read in place of an absent array's, so that a read
// needs no branch (a branch around it would make the next ones wait).
template <class T>
__device__ __forceinline__ const T* safe() {
    return (const T*)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
}

// Parts of [0, total): the one of lane l is [start[l], start[l+1]) cut to
// [0, total), or total / lanes entries each without a start array.
struct Parts {
    const int32_t* start;
    uint32_t total;
    uint32_t each;  // total / lanes (start == NULL)
    // from start[l] and start[l + 1] (any values without a start array)
    __device__ __forceinline__ void cut(uint32_t l, int32_t b, int32_t e, uint32_t& begin, uint32_t& end) const {
        begin = start ? (b < 0 ? 0u : min_u32((uint32_t)b, total)) : l * each;
        end = start ? (e < 0 ? 0u : min_u32((uint32_t)e, total)) : begin + each;
        if (end < begin) end = begin;
    }
    // where start[l] and start[l + 1] can be read
    __device__ __forceinline__ const int32_t* at(uint32_t l) const { return start ? start + l : safe<int32_t>(); }
    __device__ __forceinline__ void range(uint32_t l, uint32_t& begin, uint32_t& end) const {
        int32_t b = 0, e = 0;
        if (start) {  // (a uniform branch: the reads stay scalar)
            b = start[l];
            e = start[l + 1];
        }
        cut(l, b, e, begin, end);
    }
};

// topk_cols_adjust (see the header): sizes narrowed to 32 bits where the
// entry point has checked them.
struct AdjustArgs {
    const void* x;
    void* out;
    int64_t ld, out_ld;
    uint32_t V, C, lanes;
    Parts cols;               // the lanes' columns
    const int32_t* counts;    // NULL: no history
    int64_t counts_ld;
    const uint32_t* seen;
    int64_t seen_ld;
    const float *repetition, *presence, *frequency;
    const int32_t* drafts;    // NULL: none
    Parts draft_parts;
    const int32_t* bias_ids;  // NULL: none
    const float* bias_values;
    Parts bias_parts;
    const uint32_t* mask;     // NULL: none
    int64_t mask_ld;
    int32_t mask_count;
    const int32_t* mask_index;
};
hipError_t launch_adjust(int dtype, int layout, const AdjustArgs& a, hipStream_t stream);

struct CountArgs {
    uint32_t V, lanes;
    const int32_t* ids;
    Parts parts;
    const int32_t *prompt_len, *fresh;
    uint32_t* counts;
    int64_t counts_ld;
    uint32_t* seen;
    int64_t seen_ld;
};
hipError_t launch_count(const CountArgs& a, hipStream_t stream);

struct VerifyArgs {
    topk_verify_args v;
    Parts cols, draft_parts;
};
hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream);

hipError_t launch_plan_round(const topk_plan_args& a, hipStream_t stream);

// The grid's y size is at most 65,535.
constexpr int64_t kGridY = 65535;

}  // namespace topk
