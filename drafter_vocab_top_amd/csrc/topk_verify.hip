// Verification of drafts against the target's top-k lists, for gfx950.
//
// For lane l, with p_j the distribution of its column j, d_j its j-th draft
// and q_j the distribution the draft was sampled from (both as
// topk_cols_sample draws: temperature, nucleus, sums in list order):
//   draft j is accepted if u * q_j(d_j) < p_j(d_j);
//   the first refused column t gives a token from max(p_t - q_t, 0), or, with
//   every draft accepted, the column behind them gives one from p.
// Accepting with probability min(1, p/q) and drawing from the positive part
// of p - q otherwise leaves each token distributed as p.
//
// One workgroup per lane, one wave per column: a column's test and the token
// it would give do not depend on the other columns, so the waves compute
// both at once and only then agree on the first refusal.  List entry i lies
// in lane i (k <= 64).
//
// The decisions are integers made by floating point, so every step is IEEE
// double in a fixed order with no contraction; sums run in list order.
#include "topk_draw.hpp"
#include "topk_round.hpp"

namespace topk {

namespace {

constexpr uint32_t kVerifyWaves = 8;  // columns judged at once
constexpr uint32_t kVerifyThreads = kVerifyWaves * 64;

// Lane m gets x_0 + ... + x_m (x_0 .. x_{n-1}, added in this order; lanes
// past the end hold the total).
__device__ __forceinline__ double ordered_sums(double x, int32_t n) {
#pragma clang fp contract(off)
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    double acc = 0.0;
    for (int32_t j = 0; j < n; ++j) {
        const double xj = lane_value(x, j);
        if (j <= lane) acc = acc + xj;
    }
    return acc;
}

// The probability of this lane's entry of a list (0 past the nucleus).
template <class DT>
__device__ __forceinline__ double probability(const typename DT::storage* v, int32_t k, double temperature,
                                              double top_p) {
#pragma clang fp contract(off)
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const double v0 = stored_value<DT>(v, 0);
    if (temperature == 0.0 || !__builtin_isfinite(v0)) return lane == 0 ? 1.0 : 0.0;
    const bool in = lane < k;
    const double w = in ? fixed_exp((stored_value<DT>(v, lane) - v0) / temperature) : 0.0;
    const double sums = ordered_sums(w, k);
    const double need = top_p * lane_value(sums, k - 1);
    const unsigned long long reach = __ballot(in && sums >= need);
    const int32_t n = reach ? (int32_t)first_lane(reach) + 1 : k;
    return lane < n ? w / lane_value(sums, n - 1) : 0.0;
}

// The probability of token d: that of the first entry with its id.
__device__ __forceinline__ double probability_of(int32_t d, int32_t id, double p, int32_t k) {
    const unsigned long long m = __ballot((int32_t)(threadIdx.x & 63u) < k && id == d);
    return m ? lane_value(p, (int)first_lane(m)) : 0.0;
}

template <class DT>
__global__ __launch_bounds__(kVerifyThreads) void verify_kernel(VerifyArgs args) {
#pragma clang fp contract(off)
    using storage = typename DT::storage;
    __shared__ int32_t token[kVerifyWaves];
    __shared__ uint32_t refused[kVerifyWaves];
    const topk_verify_args& a = args.v;
    const uint32_t l = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
    const int32_t lane = (int32_t)(tid & 63u);
    int32_t* out = a.out_tokens + (int64_t)l * a.max_tokens;
    uint32_t cb, ce, db, de;
    args.cols.range(l, cb, ce);
    args.draft_parts.range(l, db, de);
    uint32_t count = 0;  // tokens of the lane
    if (ce > cb) {
        const uint32_t m = min_u32(min_u32(de - db, ce - cb - 1u), (uint32_t)a.max_tokens - 1u);
        for (uint32_t j0 = 0;; j0 += kVerifyWaves) {
            const uint32_t j = j0 + wave;
            if (j <= m) {  // wave-uniform
                const int64_t c = (int64_t)cb + j;
                const int32_t id = lane < a.k ? a.target_ids[c * a.k + lane] : 0;
                const double p = probability<DT>(static_cast<const storage*>(a.target_values) + c * a.k, a.k,
                                                 a.temperature, a.top_p);
                bool accept = false;
                double rest = p;
                if (j < m) {
                    const int64_t row = (int64_t)db + j;
                    const int32_t d = a.drafts[row];
                    double q_d = 1.0, q_at = lane < a.k && id == d ? 1.0 : 0.0;
                    if (a.draft_values) {
                        const int32_t qid = lane < a.kq ? a.draft_ids[row * a.kq + lane] : 0;
                        const double q = probability<DT>(static_cast<const storage*>(a.draft_values) + row * a.kq, a.kq,
                                                         a.temperature, a.top_p);
                        q_d = probability_of(d, qid, q, a.kq);
                        bool found = false;
                        q_at = 0.0;
                        for (int32_t t = 0; t < a.kq; ++t) {
                            const double qt = lane_value(q, t);
                            if (!found && __builtin_amdgcn_readlane(qid, t) == id) {
                                found = true;
                                q_at = qt;
                            }
                        }
                    }
                    const double u = philox_uniform(a.seed, a.offset, (uint32_t)c, 1u);
                    accept = u * q_d < probability_of(d, id, p, a.k);
                    const double diff = p - q_at;
                    rest = diff > 0.0 ? diff : 0.0;
                    if (__ballot(rest > 0.0) == 0ull) rest = p;
                }
                const double sums = ordered_sums(rest, a.k);
                const double target = philox_uniform(a.seed, a.offset, (uint32_t)c, 2u) * lane_value(sums, a.k - 1);
                const unsigned long long above = __ballot(lane < a.k && sums > target);
                const unsigned long long some = __ballot(lane < a.k && rest > 0.0);
                // (a product rounded up to the total leaves none above it: the last entry that can be drawn)
                const uint32_t pick = above ? first_lane(above) : some ? 63u - (uint32_t)__builtin_clzll(some) : 0u;
                const int32_t next = __builtin_amdgcn_readlane(id, (int)pick);
                if (lane == 0) {
                    token[wave] = next;
                    refused[wave] = accept ? 0u : 1u;
                }
            }
            __syncthreads();
            const uint32_t n = min_u32(kVerifyWaves, m + 1u - j0);  // columns of this step
            uint32_t t = 0;
            while (t < n && !refused[t]) ++t;  // column m is never accepted
            if (tid < t) out[j0 + tid] = a.drafts[(int64_t)db + j0 + tid];
            if (t < n) {
                if (tid == 0) out[j0 + t] = token[t];
                count = j0 + t + 1u;
                break;
            }
            __syncthreads();  // the next step writes token and refused again
        }
    }
    for (uint32_t i = count + tid; i < (uint32_t)a.max_tokens; i += kVerifyThreads) out[i] = -1;
    if (tid == 0) a.out_count[l] = (int32_t)count;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.v.lanes), block(kVerifyThreads);
    if (a.v.dtype == TOPK_BF16) hipLaunchKernelGGL(verify_kernel<Bf16>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(verify_kernel<F32>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
