// Steps shared by the kernels that draw tokens: the generator, exp in fixed
// steps and the reading of a list's values.  What they compute is part of the
// library's contract (a draw is reproducible bit for bit), so it is written
// once.
//
// Philox4x32-10 is the counter-based generator of Salmon, Moraes, Dror and
// Shaw ("Parallel random numbers: as easy as 1, 2, 3", SC 2011).  exp is
// evaluated by a fixed method: reduction x = n ln 2 + r (n = rint(x / ln 2),
// ln 2 in two parts, Cody and Waite's scheme with fused multiply-adds), the
// degree-13 Taylor polynomial of e^r by Horner's rule with fused
// multiply-adds, then ldexp by n; 0 below -745.
#pragma once

#include "topk_device.hpp"

namespace topk {

__device__ __forceinline__ void philox4x32_10(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        if (round > 0) {
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        const uint32_t lo0 = 0xD2511F53u * c[0], hi0 = __umulhi(0xD2511F53u, c[0]);
        const uint32_t lo1 = 0xCD9E8D57u * c[2], hi1 = __umulhi(0xCD9E8D57u, c[2]);
        const uint32_t n0 = hi1 ^ c[1] ^ k0, n2 = hi0 ^ c[3] ^ k1;
        c[0] = n0;
        c[1] = lo1;
        c[2] = n2;
        c[3] = lo0;
    }
}

__device__ __forceinline__ double fixed_exp(double x) {
#pragma clang fp contract(off)
    if (!(x >= -745.0)) return 0.0;
    const double inv_ln2 = 1.4426950408889634;
    const double ln2_hi = 6.93147180369123816490e-01;
    const double ln2_lo = 1.90821492927058770002e-10;
    const double n = __builtin_rint(x * inv_ln2);
    double r = __builtin_fma(-n, ln2_hi, x);
    r = __builtin_fma(-n, ln2_lo, r);
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, r, 1.0 / 479001600.0);
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// The uniform in [0, 1) of counter (offset, column, stream) and key seed.
__device__ __forceinline__ double philox_uniform(uint64_t seed, uint64_t offset, uint32_t column, uint32_t stream) {
    uint32_t ctr[4] = {(uint32_t)offset, (uint32_t)(offset >> 32), column, stream};
    philox4x32_10(ctr, (uint32_t)seed, (uint32_t)(seed >> 32));
    return (double)((((uint64_t)ctr[0] << 32) | ctr[1]) >> 11) * 0x1.0p-53;
}

template <class DT>
__device__ __forceinline__ double stored_value(const typename DT::storage* v, int64_t i) {
    uint32_t b = (uint32_t)v[i];
    if constexpr (DT::kPerVec == 8) b <<= 16;  // bf16: the upper half of a binary32
    return (double)__builtin_bit_cast(float, b);
}

__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ uint32_t first_lane(unsigned long long mask) {
    return (uint32_t)__builtin_ctzll(mask);
}

}  // namespace topk
