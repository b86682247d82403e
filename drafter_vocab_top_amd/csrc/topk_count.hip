// Token histories of the lanes, for gfx950: counts[l][r] holds bit 31 if
// token r occurs in lane l's prompt and below it how often it occurs in the
// lane's output; seen[l] has a bit per token whose word is not zero.
//
// Integer atomics: the result does not depend on their order.
#include "topk_round.hpp"

namespace topk {

namespace {

__global__ __launch_bounds__(kBlock) void count_clear(CountArgs a, uint32_t l0) {
    const uint32_t l = l0 + blockIdx.y;
    if (a.fresh[l] == 0) return;
    const uint32_t first = blockIdx.x * kBlock + threadIdx.x, stride = gridDim.x * kBlock;
    for (uint32_t r = first; r < a.V; r += stride) a.counts[(int64_t)l * a.counts_ld + r] = 0u;
    for (uint32_t w = first; w < (a.V + 31u) / 32u; w += stride) a.seen[(int64_t)l * a.seen_ld + w] = 0u;
}

__global__ __launch_bounds__(kBlock) void count_add(CountArgs a) {
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= a.parts.total) return;
    uint32_t l = 0;
    if (a.parts.start) {
        // the last lane that starts at or before token i
        uint32_t lo = 0, hi = a.lanes;
        while (hi - lo > 1u) {
            const uint32_t mid = lo + (hi - lo) / 2u;
            if (a.parts.start[mid] <= (int32_t)i) lo = mid;
            else hi = mid;
        }
        l = lo;
    } else {
        l = i / a.parts.each;
    }
    uint32_t b, e;
    a.parts.range(l, b, e);
    const uint32_t r = (uint32_t)a.ids[i];
    if (i < b || i >= e || r >= a.V) return;
    uint32_t* word = a.counts + (int64_t)l * a.counts_ld + r;
    if (a.prompt_len && (int64_t)(i - b) < (int64_t)a.prompt_len[l]) atomicOr(word, 0x80000000u);
    else atomicAdd(word, 1u);
    atomicOr(a.seen + (int64_t)l * a.seen_ld + (r >> 5), 1u << (r & 31u));
}

}  // namespace

hipError_t launch_count(const CountArgs& a, hipStream_t stream) {
    if (a.fresh) {
        for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
            const uint32_t n = (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY);
            const uint32_t blocks = min((a.V + 16u * kBlock - 1u) / (16u * kBlock), 64u);
            hipLaunchKernelGGL(count_clear, dim3(blocks, n), dim3(kBlock), 0, stream, a, (uint32_t)l0);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        }
    }
    if (a.parts.total == 0) return hipSuccess;
    hipLaunchKernelGGL(count_add, dim3((a.parts.total + kBlock - 1) / kBlock), dim3(kBlock), 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
