// Sampling one draft per column from its top-k list, for gfx950.
//
// The ignis "DFlash2" page measures sampled drafting at temperature 1.0,
// top_p 0.95 and top_k 20 ("Greedy coding is the best case"; last row of
// "The numbers") without spelling out the sampler.  This kernel implements
// the standard reading.  For a column whose top-k values are
// v_0 >= ... >= v_{k-1} (largest first, as the top-k kernels emit them):
//   w_j = exp((v_j - v_0) / T),  S_m = w_0 + ... + w_{m-1} (in that order),
//   n = the smallest m with S_m >= top_p * S_k,
//   u = a uniform in [0, 1) from Philox4x32-10,
//   j* = the smallest j < n with S_{j+1} > u * S_n,
// and the output is ids[j*] (and j*).  A column whose top value is not
// finite takes j* = 0.
//
// The draw is an integer decided by floating point, so every step is IEEE
// double in a fixed order, with no contraction of separate operations into
// fused ones, and exp is evaluated by a fixed method instead of the device
// library's: reduction x = n ln 2 + r (n = rint(x / ln 2), ln 2 in two
// parts, Cody and Waite's scheme with fused multiply-adds), the degree-13
// Taylor polynomial of e^r by Horner's rule with fused multiply-adds, then
// ldexp by n; 0 below -745.  Philox4x32-10 is the counter-based generator of
// Salmon, Moraes, Dror and Shaw ("Parallel random numbers: as easy as 1, 2,
// 3", SC 2011): counter (offset low, offset high, column, 0), key (seed low,
// seed high), ten rounds; u = ((out0 << 32 | out1) >> 11) * 2^-53.
//
// One wave per column.  Lane j computes w_j (one exp per lane, in
// parallel); the sums must keep the sequential order, so every lane then
// walks j = 0 .. k-1 with w_j broadcast from lane j and adds it when j <= its
// own index: lane m ends with S_{m+1}, summed in exactly the order above.
// Ballots find n and j*.
#include "topk_draw.hpp"
#include "topk_internal.hpp"

namespace topk {

namespace {

constexpr int kSampleThreads = 256;
constexpr int kSampleWaves = kSampleThreads / 64;  // one column per wave

template <class DT>
__global__ __launch_bounds__(kSampleThreads) void topk_sample_kernel(SampleArgs a) {
#pragma clang fp contract(off)
    using storage = typename DT::storage;
    const uint32_t lane = threadIdx.x & 63u;
    const int64_t c = (int64_t)blockIdx.x * kSampleWaves + (threadIdx.x >> 6);
    if (c >= a.C) return;  // wave-uniform
    const int32_t k = a.k;
    const storage* v = static_cast<const storage*>(a.values) + c * k;
    uint32_t pick = 0;
    const double v0 = stored_value<DT>(v, 0);
    if (__builtin_isfinite(v0)) {
        const bool in = (int32_t)lane < k;
        const double w = in ? fixed_exp((stored_value<DT>(v, lane) - v0) / a.temperature) : 0.0;
        double acc = 0.0;  // S_{lane+1} (S_k for lanes >= k)
        for (int32_t j = 0; j < k; ++j) {
            const double wj = lane_value(w, j);
            if (j <= (int32_t)lane) acc = acc + wj;
        }
        const double total = lane_value(acc, k - 1);
        const double need = a.top_p * total;
        const unsigned long long reach = __ballot(in && acc >= need);
        const uint32_t n = reach ? first_lane(reach) + 1u : (uint32_t)k;  // lane k-1 always reaches
        const double sn = lane_value(acc, (int)n - 1);
        const double u = philox_uniform(a.seed, a.offset, (uint32_t)c, 0u);
        const double target = u * sn;
        const unsigned long long above = __ballot(lane < n && acc > target);
        pick = above ? first_lane(above) : n - 1u;  // u < 1 makes lane n-1 pass
    }
    if (lane == 0) {
        a.out_ids[c] = a.ids[c * k + pick];
        if (a.out_pos) a.out_pos[c] = (int32_t)pick;
    }
}

}  // namespace

hipError_t launch_sample(int dtype, const SampleArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.C + kSampleWaves - 1) / kSampleWaves)), block(kSampleThreads);
    if (dtype == 0)
        hipLaunchKernelGGL(topk_sample_kernel<Bf16>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(topk_sample_kernel<F32>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
