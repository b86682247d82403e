// Top-k lists as distributions, a wave for each list and a lane for each entry:
// what the verification kernels share.  Every step is IEEE double in a fixed
// order with no contraction (it is part of the library's contract).
#pragma once

#include "topk_draw.hpp"

namespace topk {

// x of lane - N of the same 16 lanes (0.0 where there is none).
template <int kCtrl, int kRowMask>
__device__ __forceinline__ double dpp_or_zero(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, kRowMask, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, kRowMask, 0xF, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Lane m gets x_0 + ... + x_m: within each 16 lanes in steps of 1, 2, 4 and
// 8, then the sum of the first 16 onto the second and of the third onto the
// fourth, then the sum of the first 32 onto the others.  (A sum in list order
// would be 64 dependent additions instead of 6.)
__device__ __forceinline__ double running_sum(double x) {
#pragma clang fp contract(off)
    x = x + dpp_or_zero<0x111, 0xF>(x);  // row_shr:1
    x = x + dpp_or_zero<0x112, 0xF>(x);
    x = x + dpp_or_zero<0x114, 0xF>(x);
    x = x + dpp_or_zero<0x118, 0xF>(x);
    x = x + dpp_or_zero<0x142, 0xA>(x);  // row_bcast:15
    x = x + dpp_or_zero<0x143, 0xC>(x);  // row_bcast:31
    return x;
}

// This lane's entry of a list: its value, and the list's first.
template <class DT>
__device__ __forceinline__ void load_entry(const void* values, int64_t row, int32_t k, double& v, double& v0) {
    const typename DT::storage* p = static_cast<const typename DT::storage*>(values) + row * k;
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    v = stored_value<DT>(p, lane < k ? lane : 0);
    v0 = lane_value(v, 0);
}

// The probability of this lane's entry (0 past the nucleus of n entries).
__device__ __forceinline__ double probability(double v, double v0, int32_t k, double temperature, double top_p, int32_t& n) {
#pragma clang fp contract(off)
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    n = 1;
    if (temperature == 0.0 || !__builtin_isfinite(v0)) return lane == 0 ? 1.0 : 0.0;
    const bool in = lane < k;
    const double w = in ? fixed_exp((v - v0) / temperature) : 0.0;
    const double sums = running_sum(w);
    const unsigned long long reach = __ballot(in && sums >= top_p * lane_value(sums, k - 1));
    n = reach ? (int32_t)first_lane(reach) + 1 : k;
    return lane < n ? w / lane_value(sums, n - 1) : 0.0;
}

// The probability of token d: that of the first entry with its id.
__device__ __forceinline__ double probability_of(int32_t d, int32_t id, double p, int32_t k) {
    const unsigned long long m = __ballot((int32_t)(threadIdx.x & 63u) < k && id == d);
    return m ? lane_value(p, (int)first_lane(m)) : 0.0;
}

}  // namespace topk
