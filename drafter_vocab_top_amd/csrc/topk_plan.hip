// The plan of a round, for gfx950: which columns each lane gets, where the
// keys of their tokens go, and the cache blocks they need.
//
// Everything is whole numbers: over the lanes, in order, the running sum of
// the blocks needed decides who is served, and the running sum of the served
// lanes' columns where theirs begin.  One launch: every workgroup runs both
// sums over all lanes (they are few, and stay in the caches), 1,024 lanes at
// a time, and then writes its own range of columns, finding each column's
// lane by bisection in LDS.  Workgroup 0 writes what there is per lane; new
// table entries are spread over all workgroups.
//
// Which lanes are served is a prefix of those that need blocks, and of those
// that want columns: a running sum that has passed its limit stays beyond
// it.  So the blocks of the served lanes are the first ones handed out.
#include "topk_round.hpp"

namespace topk {

namespace {

constexpr uint32_t kPlanLanes = 1024;             // lanes per step
constexpr uint32_t kPer = kPlanLanes / kBlock;    // consecutive lanes of a thread
constexpr uint32_t kPlanColumns = 2048;           // columns per workgroup

struct PlanShared {
    uint32_t end[kPlanLanes];    // columns of the lanes up to and including this one
    uint32_t taken[kPlanLanes];  // blocks of the served lanes up to and including this one
    uint32_t need[kPlanLanes];
    uint32_t len[kPlanLanes];
    uint32_t held[kPlanLanes];
    int64_t wave_sum[kWaves];
    uint32_t served, taken_to, refused;
};

// Sum of the values of the threads before this one; total: of all threads.
__device__ __forceinline__ int64_t block_sum_before(PlanShared& sh, int64_t v, int64_t& total) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    int64_t upto = v;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63u) sh.wave_sum[wave] = upto;
    __syncthreads();
    int64_t before = upto - v;
    total = 0;
#pragma unroll
    for (uint32_t w = 0; w < (uint32_t)kWaves; ++w) {
        if (w < wave) before += sh.wave_sum[w];
        total += sh.wave_sum[w];
    }
    __syncthreads();
    return before;
}

// The first of n ascending values that is above x (one is).
__device__ __forceinline__ uint32_t first_above(const uint32_t* v, uint32_t n, uint32_t x) {
    uint32_t lo = 0, hi = n - 1u;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2u;
        if (v[mid] > x) hi = mid;
        else lo = mid + 1u;
    }
    return lo;
}

__global__ __launch_bounds__(kBlock) void plan_kernel(topk_plan_args a) {
    __shared__ PlanShared sh;
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
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            const uint32_t i = tid * kPer + q, l = l0 + i;
            add[q] = need[q] = len[q] = held[q] = total[q] = 0;
            want[q] = false;
            if (i < n) {
                const int32_t ln = a.lens[l], ad = a.add[l], h = a.held[l];
                len[q] = ln < 0 ? 0u : (uint32_t)ln;
                add[q] = ad < 0 ? 0u : (uint32_t)ad;
                held[q] = h < 0 ? 0u : min_u32((uint32_t)h, (uint32_t)a.table_ld);
                if (add[q] != 0) {
                    total[q] = (len[q] + add[q] - 1u) / bs + 1u;
                    want[q] = total[q] <= (uint32_t)a.table_ld && len[q] + add[q] <= 0x7FFFFFFFu;
                    if (want[q] && total[q] > held[q]) need[q] = total[q] - held[q];
                }
            }
            blocks += need[q];
        }
        int64_t step_total;
        int64_t upto = blocks_before + block_sum_before(sh, blocks, step_total);
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
        upto = columns_before + block_sum_before(sh, columns, step_total);
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
            refused += add[q] != 0 && !ok[q] ? 1u : 0u;
        }
        if (top) atomicMax(&sh.served, top);
        if (top_taken) atomicMax(&sh.taken_to, top_taken);
        if (refused) atomicAdd(&sh.refused, refused);
        __syncthreads();
        const uint32_t served_from = served, taken_from = taken_to;
        served = sh.served;
        taken_to = sh.taken_to;
#pragma unroll
        for (uint32_t q = 0; q < kPer; ++q) {
            const uint32_t i = tid * kPer + q;
            const uint32_t e = end[q] <= (int64_t)capacity ? (uint32_t)end[q] : served;
            sh.end[i] = e;
            sh.taken[i] = taken[q] < (int64_t)taken_to ? (uint32_t)taken[q] : taken_to;
            sh.need[i] = need[q];
            sh.len[i] = len[q];
            sh.held[i] = held[q];
            if (first_wg && i < n) {
                a.out_col_start[l0 + i + 1] = (int32_t)e;
                a.out_held[l0 + i] = (int32_t)(ok[q] ? max_u32(total[q], held[q]) : held[q]);
            }
        }
        __syncthreads();
        // this workgroup's columns of these lanes
        const uint32_t ka = k0 > served_from ? k0 : served_from, kb = min_u32(k1, served);
        for (uint32_t t = ka + tid; t < kb; t += kBlock) {
            const uint32_t i = first_above(sh.end, n, t), l = l0 + i;
            const uint32_t pos = sh.len[i] + (t - (i ? sh.end[i - 1] : served_from));
            const uint32_t bi = pos / bs, h = sh.held[i];
            const int32_t id = bi < h ? a.table[(int64_t)l * a.table_ld + bi]
                                      : a.free_ids[free_n - 1u - (sh.taken[i] - sh.need[i] + (bi - h))];
            a.out_col_lane[t] = (int32_t)l;
            a.out_col_pos[t] = (int32_t)pos;
            a.out_slots[t] = (int64_t)id * bs + (pos - bi * bs);
        }
        // and its share of the new table entries
        for (uint32_t b = taken_from + blockIdx.x * kBlock + tid; b < taken_to; b += gridDim.x * kBlock) {
            const uint32_t i = first_above(sh.taken, n, b);
            const uint32_t at = sh.held[i] + (b - (sh.taken[i] - sh.need[i]));
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

hipError_t launch_plan_round(const topk_plan_args& a, hipStream_t stream) {
    const uint32_t blocks = (uint32_t)((a.capacity + kPlanColumns - 1) / kPlanColumns);
    hipLaunchKernelGGL(plan_kernel, dim3(blocks), dim3(kBlock), 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
