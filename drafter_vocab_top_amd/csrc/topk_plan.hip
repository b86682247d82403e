// The plan of a round, for gfx950: which columns each lane gets, where the
// keys of their tokens go, and the cache blocks they need.
//
// Everything is whole numbers: over the lanes, in order, the running sum of
// the blocks needed decides who is served, and the running sum of the served
// lanes' columns where theirs begin.  One launch: every workgroup runs both
// sums over all lanes (they are few, and stay in the caches), 256 to
// 1,024 lanes at a time, and then writes its own range of columns, finding each column's
// lane by bisection in LDS.  Workgroup 0 writes what there is per lane; new
// table entries are spread over all workgroups.
//
// Which lanes are served is a prefix of those that need blocks, and of those
// that want columns: a running sum that has passed its limit stays beyond
// it.  So the blocks of the served lanes are the first ones handed out.
//
// One MI355X, replayed from a graph: 64 lanes, 512 columns 3.5 us, a launch and
// the chain lanes, sums, lane of a column, table entry, store; 512 lanes,
// 577,000 columns (9.2 MB written) 7.2 us.
#include "topk_round.hpp"

namespace topk {

namespace {


constexpr int64_t kFewColumns = 262144;

struct alignas(16) PlanLane {
    uint32_t base;       // position - column, of the lane's columns
    uint32_t held;
    uint32_t free_base;  // its table entry e >= held is free_ids[free_base - e]
    uint32_t unused;
};

template <uint32_t kLanes>
struct PlanShared {
    PlanLane lane[kLanes];
    uint32_t end[kLanes];    // columns of the lanes up to and including this one
    uint32_t taken[kLanes];  // blocks of the served lanes up to and including this one
    int64_t wave_sum[2][kWaves];
    uint32_t served, taken_to, refused;
};

// x / block size, for x < 2^31: with s the least exponent for which 2^s is no
// less than the size, m = ceil(2^(31+s) / size) exceeds the quotient by less
// than 1, so x * m / 2^(31+s) exceeds x / size by less than
// x / (2^(31+s)) <= 1 / size.
struct BlockOf {
    uint32_t mul, shift;
    explicit BlockOf(uint32_t size) : shift(31) {
        while ((1ull << (shift - 31)) < size) ++shift;
        mul = (uint32_t)(((1ull << shift) + size - 1u) / size);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (uint32_t)((uint64_t)x * mul >> shift); }
};

template <int kCtrl, int kRowMask>
__device__ __forceinline__ int64_t dpp_or_zero(int64_t x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, kCtrl, kRowMask, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)((uint64_t)x >> 32), kCtrl, kRowMask, 0xF, true);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sum of the values of the threads before this one; total: of all threads.
// sums: kWaves values of LDS that no other call before the next barrier uses.
__device__ __forceinline__ int64_t block_sum_before(int64_t* sums, int64_t v, int64_t& total) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    int64_t upto = v;
    upto += dpp_or_zero<0x111, 0xF>(upto);  // row_shr:1, 2, 4, 8
    upto += dpp_or_zero<0x112, 0xF>(upto);
    upto += dpp_or_zero<0x114, 0xF>(upto);
    upto += dpp_or_zero<0x118, 0xF>(upto);
    upto += dpp_or_zero<0x142, 0xA>(upto);  // row_bcast:15, 31
    upto += dpp_or_zero<0x143, 0xC>(upto);
    if (lane == 63u) sums[wave] = upto;
    __syncthreads();
    int64_t before = upto - v;
    total = 0;
#pragma unroll
    for (uint32_t w = 0; w < (uint32_t)kWaves; ++w) {
        if (w < wave) before += sums[w];
        total += sums[w];
    }
    return before;
}

// The first of the ascending values v[lo .. hi] that is above x (v[hi] is).
__device__ __forceinline__ uint32_t first_above(const uint32_t* v, uint32_t lo, uint32_t hi, uint32_t x) {
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2u;
        if (v[mid] > x) hi = mid;
        else lo = mid + 1u;
    }
    return lo;
}

// kPer: consecutive lanes of a thread; U: columns of a thread.
template <uint32_t kPer, uint32_t U>
__global__ __launch_bounds__(kBlock) void plan_kernel(topk_plan_args a, BlockOf block_of) {
    constexpr uint32_t kPlanLanes = kBlock * kPer;  // lanes per step
    constexpr uint32_t kPlanColumns = kBlock * U;   // columns of a workgroup
    __shared__ PlanShared<kPlanLanes> sh;
    const uint32_t tid = threadIdx.x;
    const bool first_wg = blockIdx.x == 0;
    const uint32_t bs = (uint32_t)a.block_size, capacity = (uint32_t)a.capacity;
    const uint32_t k0 = blockIdx.x * kPlanColumns, k1 = min_u32(capacity, k0 + kPlanColumns);
    const int32_t fc = *a.free_count;
    const uint32_t free_n = fc < 0 ? 0u : min_u32((uint32_t)fc, (uint32_t)a.n_free_ids);
    if (tid == 0) sh.served = sh.taken_to = sh.refused = 0;
    int64_t blocks_before = 0, columns_before = 0;  // running sums over the steps
    uint32_t served = 0, taken_to = 0;              // columns and blocks handed out so far

    for (uint32_t l0 = 0; l0 < (uint32_t)a.lanes; l0 += kPlanLanes) {
        const uint32_t n = min_u32(kPlanLanes, (uint32_t)a.lanes - l0);
        uint32_t add[kPer], need[kPer], len[kPer], held[kPer], total[kPer];
        bool want[kPer];
        int64_t blocks = 0;
        int32_t ln[kPer], ad[kPer], hl[kPer];
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {  // (at the last lane past the end: no branch between the reads)
            const uint32_t l = l0 + min_u32(tid * kPer + q, n - 1u);
            ln[q] = a.lens[l];
            ad[q] = a.add[l];
            hl[q] = a.held[l];
        }
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            len[q] = ln[q] < 0 ? 0u : (uint32_t)ln[q];
            add[q] = ad[q] < 0 || tid * kPer + q >= n ? 0u : (uint32_t)ad[q];
            held[q] = hl[q] < 0 ? 0u : min_u32((uint32_t)hl[q], (uint32_t)a.table_ld);
            const bool some = add[q] != 0 && len[q] + add[q] <= 0x7FFFFFFFu;
            total[q] = some ? block_of(len[q] + add[q] - 1u) + 1u : 0u;
            want[q] = some && total[q] <= (uint32_t)a.table_ld;
            need[q] = want[q] && total[q] > held[q] ? total[q] - held[q] : 0u;
            blocks += need[q];
        }
        int64_t step_total;
        int64_t upto = blocks_before + block_sum_before(sh.wave_sum[0], blocks, step_total);
        blocks_before += step_total;
        int64_t taken[kPer], columns = 0;
        bool ok[kPer];
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            upto += need[q];
            taken[q] = upto;
            ok[q] = want[q] && (need[q] == 0 || upto <= (int64_t)free_n);
            columns += ok[q] ? add[q] : 0u;
        }
        upto = columns_before + block_sum_before(sh.wave_sum[1], columns, step_total);
        columns_before += step_total;
        uint32_t top = 0, top_taken = 0, refused = 0;
        int64_t end[kPer];
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            upto += ok[q] ? add[q] : 0u;
            end[q] = upto;
            ok[q] = ok[q] && upto <= (int64_t)capacity;
            if (upto <= (int64_t)capacity) top = max_u32(top, (uint32_t)upto);
            if (ok[q] && need[q]) top_taken = max_u32(top_taken, (uint32_t)taken[q]);
            refused += (uint32_t)__popcll(__ballot(add[q] != 0 && !ok[q]));
        }
        if (refused && (tid & 63u) == 0) atomicAdd(&sh.refused, refused);
        const uint32_t served_from = served, taken_from = taken_to;
        if (columns_before <= (int64_t)capacity && blocks_before <= (int64_t)free_n) {
            // everyone who wants columns is served (all threads agree)
            served = (uint32_t)columns_before;
            taken_to = (uint32_t)blocks_before;
        } else {
            top = wave_max_u32(top);
            top_taken = wave_max_u32(top_taken);
            if ((tid & 63u) == 0) {
                atomicMax(&sh.served, top);
                atomicMax(&sh.taken_to, top_taken);
            }
            __syncthreads();
            served = max_u32(served, sh.served);
            taken_to = max_u32(taken_to, sh.taken_to);
        }
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            const uint32_t i = tid * kPer + q;
            const uint32_t e = end[q] <= (int64_t)capacity ? (uint32_t)end[q] : served;
            sh.end[i] = e;
            sh.taken[i] = taken[q] < (int64_t)taken_to ? (uint32_t)taken[q] : taken_to;
            // (of a lane that is not served, no column or block looks at these)
            sh.lane[i] = PlanLane{len[q] - (e - add[q]), held[q], free_n - 1u - ((uint32_t)taken[q] - need[q]) + held[q], 0u};
            if (first_wg && i < n) {
                a.out_col_start[l0 + i + 1] = (int32_t)e;
                a.out_held[l0 + i] = (int32_t)(ok[q] ? max_u32(total[q], held[q]) : held[q]);
            }
        }
        __syncthreads();
        // this workgroup's columns of these lanes, all of a thread's at once
        const uint32_t ka = k0 > served_from ? k0 : served_from, kb = min_u32(k1, served);
        if (ka < kb) {
            // the lanes of the first and last column (known where they are the step's)
            const uint32_t lo = ka == served_from ? 0u : first_above(sh.end, 0, n - 1u, ka);
            const uint32_t hi = kb == served ? n - 1u : first_above(sh.end, lo, n - 1u, kb - 1u);
            uint32_t l[U], pos[U], bi[U];
            int32_t id[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                const uint32_t t = min_u32(ka + u * kBlock + tid, kb - 1u);
                const uint32_t i = first_above(sh.end, lo, hi, t);
                const PlanLane p = sh.lane[i];
                l[u] = l0 + i;
                pos[u] = p.base + t;
                bi[u] = block_of(pos[u]);
                id[u] = *(bi[u] < p.held ? a.table + (int64_t)l[u] * a.table_ld + bi[u] : a.free_ids + (p.free_base - bi[u]));
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                const uint32_t t = ka + u * kBlock + tid;
                if (t >= kb) break;
                a.out_col_lane[t] = (int32_t)l[u];
                a.out_col_pos[t] = (int32_t)pos[u];
                a.out_slots[t] = (int64_t)id[u] * bs + (pos[u] - bi[u] * bs);
            }
        }
        // and its share of the new table entries
        for (uint32_t b = taken_from + blockIdx.x * kBlock + tid; b < taken_to; b += gridDim.x * kBlock) {
            const uint32_t i = first_above(sh.taken, 0, n - 1u, b);
            const uint32_t at = b + sh.lane[i].free_base - (free_n - 1u);
            a.table[(int64_t)(l0 + i) * a.table_ld + at] = a.free_ids[free_n - 1u - b];
        }
        __syncthreads();
    }
    for (uint32_t t = (k0 > served ? k0 : served) + tid; t < k1; t += kBlock) {
        a.out_col_lane[t] = -1;
        a.out_col_pos[t] = -1;
        a.out_slots[t] = -1;
    }
    if (first_wg && tid == 0) {
        a.out_col_start[0] = 0;
        *a.out_free_count = (int32_t)(free_n - taken_to);
        *a.out_refused = (int32_t)sh.refused;
    }
}

}  // namespace

namespace {

template <uint32_t U>
hipError_t launch_columns(const topk_plan_args& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.capacity + kBlock * U - 1) / (kBlock * U))), block(kBlock);
    const BlockOf block_of((uint32_t)a.block_size);
    // one step for up to 1,024 lanes, with no more lanes to a thread than it takes
    if (a.lanes <= kBlock) hipLaunchKernelGGL((plan_kernel<1, U>), grid, block, 0, stream, a, block_of);
    else if (a.lanes <= 2 * kBlock) hipLaunchKernelGGL((plan_kernel<2, U>), grid, block, 0, stream, a, block_of);
    else hipLaunchKernelGGL((plan_kernel<4, U>), grid, block, 0, stream, a, block_of);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_plan_round(const topk_plan_args& a, hipStream_t stream) {
    // One column per thread is the shortest chain (512 columns: 3.5 us, in
    // fours 5.0; 262,144: 5.6 and 6.6), until the workgroups that repeat the
    // sums over the lanes outnumber those that run at once (524,288 columns:
    // 12.2 us, in fours 8.2).
    if (a.capacity <= kFewColumns) return launch_columns<1>(a, stream);
    return launch_columns<4>(a, stream);
}

}  // namespace topk
