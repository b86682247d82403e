// Token histories of the lanes, for gfx950: counts[l][r] holds bit 31 if
// token r occurs in lane l's prompt and below it how often it occurs in the
// lane's output; seen[l] has a bit per token whose word is not zero.
//
// Whole numbers, added and or-ed: no order of the tokens changes the result.
//
// Few tokens (a round's commits): one thread per token, two atomics in
// memory.  Long lists, and lanes that start anew: a workgroup owns a share of
// a lane's rows in LDS, reads all of the lane's tokens, counts its own and
// writes its rows, so that nothing is cleared first and the many occurrences
// of frequent tokens meet in LDS instead of in one cache line.
//
// One MI355X, replayed from a graph: 64 lanes of up to 8 tokens 2.9 us, a
// launch and one chain of reads and atomics; 8 fresh lanes of 25,000 tokens
// each 10.3 us, about 5 of them the reading of each lane's tokens by all 32
// workgroups of the lane (L2), 2 their LDS atomics and 2 the 8 MB of rows.
#include "topk_round.hpp"

#include "topk_col_common.hpp"

namespace topk {

namespace {

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
    // the prompt's tokens set the flag, the others add one
    if (a.prompt_len && (int64_t)(i - b) < (int64_t)a.prompt_len[l]) atomicOr(word, 0x80000000u);
    else atomicAdd(word, 1u);
    atomicOr(a.seen + (int64_t)l * a.seen_ld + (r >> 5), 1u << (r & 31u));
}

constexpr uint32_t kOwnThreads = 1024;
constexpr uint32_t kOwnRows = 8192;  // rows of a workgroup, at most (32 KB of LDS)

// Workgroup x of gridDim.x = 1 << tiles_log owns the groups of 32 rows whose
// index is x modulo the number of workgroups: frequent tokens (low ids, in a
// vocabulary sorted by use) spread over all of them, and a group is a whole
// word of `seen` and a whole cache line of counts.
__global__ __launch_bounds__(kOwnThreads) void count_own(CountArgs a, uint32_t l0, uint32_t tiles_log) {
    __shared__ alignas(16) uint32_t own[kOwnRows];
    const uint32_t l = l0 + blockIdx.y, tid = threadIdx.x, tile = blockIdx.x, tiles_mask = (1u << tiles_log) - 1u;
    const int32_t* start = a.parts.at(l);
    const int32_t b0 = start[0], e0 = start[1], fresh0 = *(a.fresh ? a.fresh + l : safe<int32_t>()),
                  prompt0 = *(a.prompt_len ? a.prompt_len + l : safe<int32_t>());
    uint32_t b, e;
    a.parts.cut(l, b0, e0, b, e);
    const bool fresh = a.fresh && fresh0 != 0;
    if (!fresh && b == e) return;
    const int64_t prompt = a.prompt_len ? (int64_t)prompt0 : 0;
    const uint32_t groups = (a.V + 31u) / 32u;
    const uint32_t mine = tile < groups ? ((groups - 1u - tile) >> tiles_log) + 1u : 0u;  // groups of this workgroup
    for (uint32_t i = tid; i < mine * 8u; i += kOwnThreads) reinterpret_cast<u32x4*>(own)[i] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    constexpr uint32_t U = 4;  // reads of four tokens in flight
    auto add = [&](uint32_t i, uint32_t r) {
        const uint32_t g = r >> 5;
        if (r < a.V && (g & tiles_mask) == tile) {
            uint32_t* word = &own[(g >> tiles_log) * 32u + (r & 31u)];
            if ((int64_t)(i - b) < prompt) {
                if (!(*word >> 31)) atomicOr(word, 0x80000000u);
            } else {
                atomicAdd(word, 1u);
            }
        }
    };
    const uint32_t n4 = (e - b) / 4u;
    for (uint32_t q0 = tid; q0 < n4; q0 += kOwnThreads * U) {
        u32x4 v[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) __builtin_memcpy(&v[u], a.ids + b + min_u32(q0 + u * kOwnThreads, n4 - 1u) * 4u, 16);
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t q = q0 + u * kOwnThreads;
            if (q >= n4) break;
            const uint32_t i = b + q * 4u;
            const uint32_t vx = v[u].x, vy = v[u].y, vz = v[u].z, vw = v[u].w;
            add(i, vx);
            add(i + 1u, vy);
            add(i + 2u, vz);
            add(i + 3u, vw);
        }
    }
    if (tid < ((e - b) & 3u)) add(b + n4 * 4u + tid, (uint32_t)a.ids[b + n4 * 4u + tid]);
    __syncthreads();
    // half a wave per group of 32 rows
    for (uint32_t g = tid >> 5; g < mine; g += kOwnThreads / 32u) {
        const uint32_t group = (g << tiles_log) + tile, r = group * 32u + (tid & 31u);
        uint32_t w = own[g * 32u + (tid & 31u)];
        uint32_t* count = a.counts + (int64_t)l * a.counts_ld + r;
        const bool any = w != 0;
        if (r < a.V) {
            if (fresh) *count = w;
            else if (any) *count = (*count + (w & 0x7FFFFFFFu)) | (w & 0x80000000u);
        }
        const uint32_t word = (uint32_t)(__ballot(any) >> (tid & 32u));
        if ((tid & 31u) == 0) {
            uint32_t* seen = a.seen + (int64_t)l * a.seen_ld + group;
            if (fresh) *seen = word;
            else if (word) *seen |= word;
        }
    }
}

}  // namespace

hipError_t launch_count(const CountArgs& a, hipStream_t stream) {
    // Atomics cost by the tokens of a lane that meet in one word, owned rows by
    // the lane.  Equal (248,046 rows) near 1,024 tokens a lane for 1 lane (4.6
    // and 5.1 us) and 8 (5.4 and 5.5), near 4,096 for 64 (28.9 and 27.1); 8
    // tokens of 64 lanes 3.0 and 17.0, 26,000 of 8 lanes 158 and 10.
    if (!a.fresh && a.parts.total / a.lanes < 1024u + 48u * (uint64_t)a.lanes) {
        if (a.parts.total == 0) return hipSuccess;
        hipLaunchKernelGGL(count_add, dim3((a.parts.total + kBlock - 1) / kBlock), dim3(kBlock), 0, stream, a);
        return hipGetLastError();
    }
    uint32_t tiles_log = 0;
    while (((uint64_t)kOwnRows << tiles_log) < (uint64_t)(a.V + 31u) / 32u * 32u) ++tiles_log;
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const dim3 grid(1u << tiles_log, (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY));
        hipLaunchKernelGGL(count_own, grid, dim3(kOwnThreads), 0, stream, a, (uint32_t)l0, tiles_log);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace topk
