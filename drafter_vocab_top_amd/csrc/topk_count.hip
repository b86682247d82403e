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
// One MI355X, replayed from a graph: 64 lanes of up to 8 tokens 3.0 us, a
// launch and one chain of reads and atomics; 8 fresh lanes of 25,000 tokens
// each 9.4 us; one lane's 120,000 prompt tokens 18.9.  Every workgroup of a lane
// looks at all of its tokens, some 12 instructions each: that bounds it.
#include "topk_round.hpp"

#include "topk_col_common.hpp"

namespace topk {

namespace {

// One token per thread.  Starts may run backwards (such a lane is empty), so
// the lane of a token is found in one of two ways, by the workgroup's tokens:
// bisection where they lie between the first start and the last, a look at
// all lanes where some do not (padding behind the last lane, mostly: 512
// lanes and 4,000 tokens of nobody 3.2 us, as without them; 65,000 lanes 36,
// without them 20).
__global__ __launch_bounds__(kBlock) void count_add(CountArgs a) {
    __shared__ uint32_t lane_at[kBlock], end_at[kBlock];  // of the lane whose tokens begin here
    __shared__ uint32_t begins[kBlock / 32];
    const uint32_t tid = threadIdx.x, total = a.parts.total, w0 = blockIdx.x * kBlock, i = w0 + tid;
    const uint32_t w1 = min_u32(w0 + kBlock, total);  // the workgroup's tokens: w0 .. w1 - 1
    const uint32_t r = (uint32_t)a.ids[min_u32(i, total - 1u)];
    const int32_t* start = a.parts.start;
    uint32_t l = 0;
    bool owned = i < total;
    if (!start) {
        l = min_u32(i, total - 1u) / a.parts.each;
    } else if (start[0] <= (int32_t)w0 && start[a.lanes] >= (int32_t)w1) {
        // start[l] <= i < start[hi] to the end, in whatever order those between
        // are; lanes do not overlap, so the lane found is the token's only one.
        uint32_t hi = a.lanes;
        while (hi - l > 1u) {
            const uint32_t mid = l + (hi - l) / 2u;
            if (start[mid] <= (int32_t)i) l = mid;
            else hi = mid;
        }
    } else {
        // All lanes are looked at for those that have tokens here; of each the first
        // is marked.  A token's lane is that of the last mark before it.
        if (tid < kBlock / 32) begins[tid] = 0;
        __syncthreads();
        constexpr uint32_t U = 8;  // reads in flight
        for (uint32_t k0 = tid; k0 < a.lanes; k0 += kBlock * U) {
            int32_t s[U], t[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                const uint32_t k = min_u32(k0 + u * kBlock, a.lanes - 1u);
                s[u] = start[k];
                t[u] = start[k + 1];
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                uint32_t b, e;
                const uint32_t k = k0 + u * kBlock;
                a.parts.cut(k, s[u], t[u], b, e);
                if (k >= a.lanes || b >= e || b >= w1 || e <= w0) continue;
                const uint32_t at = b > w0 ? b - w0 : 0u;
                lane_at[at] = k;
                end_at[at] = e;
                atomicOr(&begins[at >> 5], 1u << (at & 31u));
            }
        }
        __syncthreads();
        uint32_t w = tid >> 5, m = begins[w] & (0xFFFFFFFFu >> (31u - (tid & 31u)));
        while (m == 0 && w > 0) m = begins[--w];
        owned = false;
        if (m) {
            const uint32_t at = w * 32u + 31u - (uint32_t)__builtin_clz(m);
            l = lane_at[at];
            owned = i < end_at[at];
        }
    }
    if (!owned || r >= a.V) return;
    uint32_t* word = a.counts + (int64_t)l * a.counts_ld + r;
    // the prompt's tokens set the flag, the others add one
    uint32_t b, e;
    a.parts.range(l, b, e);
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
    const uint32_t prompt = a.prompt_len && prompt0 > 0 ? (uint32_t)prompt0 : 0u;
    const uint32_t groups = (a.V + 31u) / 32u;
    const uint32_t mine = tile < groups ? ((groups - 1u - tile) >> tiles_log) + 1u : 0u;  // groups of this workgroup
    for (uint32_t i = tid; i < mine * 8u; i += kOwnThreads) reinterpret_cast<u32x4*>(own)[i] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    constexpr uint32_t U = 2;  // reads of four tokens in flight (more are no faster: instructions bound it)
    // Token i of the lane.  (Every instruction outside the branch is taken by
    // every workgroup for every token.)
    auto add = [&](uint32_t i, uint32_t r) {
        if (((r >> 5) & tiles_mask) == tile && r < a.V) {
            uint32_t* word = &own[(r >> 5 >> tiles_log) * 32u + (r & 31u)];
            if (i < prompt) {
                // (a frequent token's flag once: 120,000 equal tokens 18.6 us, not 104; tokens as they come 19.4, not 15.3)
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
            add(q * 4u, v[u].x);
            add(q * 4u + 1u, v[u].y);
            add(q * 4u + 2u, v[u].z);
            add(q * 4u + 3u, v[u].w);
        }
    }
    if (tid < ((e - b) & 3u)) add(n4 * 4u + tid, (uint32_t)a.ids[b + n4 * 4u + tid]);
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
    // Atomics cost some 4 ns for each token of a lane and 0.06 more for each
    // lane; owned rows a start, 4 ns a workgroup and 0.6 us per million rows.
    // Measured, atomics and owned rows, in us:
    //   one lane, 1,024 rows        128 tokens 2.8 and 3.1, 512 5.0 and 3.0
    //   8 lanes, 32,768 rows        128 tokens 3.2 and 3.7, 512 4.6 and 3.8
    //   64 lanes, 248,046 rows      8 tokens 3.1 and 18.1, 2,048 19.0 and 23.2
    //   512 lanes, 8,192 rows       128 tokens 6.4 and 7.2, 512 16.9 and 8.2
    //   65,000 lanes, 1,024 rows    8 tokens 32 and 304, 128 466 and 329
    const uint64_t lanes = a.lanes, tiles = ((uint64_t)a.V + kOwnRows - 1) / kOwnRows;
    if (!a.fresh && a.parts.total / lanes * (200u + 3u * lanes) < 35000u + lanes * (200u * tiles + (uint64_t)a.V * 7u / 200u)) {
        if (a.parts.total == 0) return hipSuccess;
        hipLaunchKernelGGL(count_add, dim3((a.parts.total + kBlock - 1) / kBlock), dim3(kBlock), 0, stream, a);
        return hipGetLastError();
    }
    uint32_t tiles_log = 0;
    while (((uint64_t)kOwnRows << tiles_log) < (uint64_t)(a.V + 31u) / 32u * 32u) ++tiles_log;
    // Few lanes: more workgroups, each with fewer rows to rewrite, as long as every
    // one has a CU of its own (5 lanes of 3,400 tokens, 30,281 rows: 20
    // workgroups 7.8 us, 160 4.1, 320 5.0; 248,046 rows, 4,000 tokens: 32
    // workgroups 6.4, 256 3.7).
    while (((uint64_t)a.lanes << tiles_log) <= 128 && a.V >> tiles_log > 512u) ++tiles_log;
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const dim3 grid(1u << tiles_log, (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY));
        hipLaunchKernelGGL(count_own, grid, dim3(kOwnThreads), 0, stream, a, (uint32_t)l0, tiles_log);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace topk
