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
// One workgroup per lane, one wave per column: a column's test does not depend
// on the other columns, so the waves make them at once, agree on the first
// refusal, and that column's wave draws the token.  List entry i lies in lane i
// (k <= 64), and a running sum is a scan over the wave.
//
// The decisions are integers made by floating point, so every step is IEEE
// double in a fixed order with no contraction.
//
// One MI355X, replayed from a graph: one lane of 7 drafts, k = 20, 4.3 us (a
// launch and the chain starts, lists, exp, sums, test, token); 512 lanes of up
// to 15 drafts, k = 64, fp32, 6.8 us for at most 6.2 MB of lists: some 590
// instructions a wave, half of them vector instructions.  With sums in list
// order (64 dependent additions, three times) and a token for every column it
// was 27.7.
#include "topk_draw.hpp"
#include "topk_round.hpp"

namespace topk {

namespace {

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

template <class DT, uint32_t kWavesPerLane>
__global__ __launch_bounds__(kWavesPerLane * 64) void verify_kernel(VerifyArgs args) {
#pragma clang fp contract(off)
    __shared__ uint32_t refused[kWavesPerLane];
    const topk_verify_args& a = args.v;
    const uint32_t l = blockIdx.x, tid = threadIdx.x;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const int32_t lane = (int32_t)(tid & 63u);
    int32_t* out = a.out_tokens + (int64_t)l * a.max_tokens;
    uint32_t cb, ce, db, de;
    args.cols.range(l, cb, ce);
    args.draft_parts.range(l, db, de);
    uint32_t count = 0;  // tokens of the lane
    if (ce > cb) {
        const uint32_t m = min_u32(min_u32(de - db, ce - cb - 1u), (uint32_t)a.max_tokens - 1u);
        for (uint32_t j0 = 0;; j0 += kWavesPerLane) {
            const uint32_t j = j0 + wave;
            const int64_t c = (int64_t)cb + min_u32(j, m), row = (int64_t)db + j;
            const bool judged = j < m, listed = judged && a.draft_values;
            int32_t id = 0, d = 0, qid = 0, n, nq = 1;
            double p = 0.0, q = 0.0;
            bool accept = false;
            if (j <= m) {  // wave-uniform
                // everything the column reads
                id = a.target_ids[c * a.k + (lane < a.k ? lane : 0)];
                double v, v0, qv = 0.0, qv0 = 0.0;
                load_entry<DT>(a.target_values, c, a.k, v, v0);
                if (judged) d = a.drafts[row];
                if (listed) {
                    qid = a.draft_ids[row * a.kq + (lane < a.kq ? lane : 0)];
                    load_entry<DT>(a.draft_values, row, a.kq, qv, qv0);
                }
                p = probability(v, v0, a.k, a.temperature, a.top_p, n);
                if (judged) {
                    double q_d = 1.0;
                    if (listed) {
                        q = probability(qv, qv0, a.kq, a.temperature, a.top_p, nq);
                        q_d = probability_of(d, qid, q, a.kq);
                    }
                    accept = philox_uniform(a.seed, a.offset, (uint32_t)c, 1u) * q_d < probability_of(d, id, p, a.k);
                }
                if (lane == 0) refused[wave] = accept ? 0u : 1u;
            }
            __syncthreads();
            const uint32_t columns = min_u32(kWavesPerLane, m + 1u - j0);  // of this step
            uint32_t t = 0;
            while (t < columns && !refused[t]) ++t;  // column m is never accepted
            if (tid < t) out[j0 + tid] = a.drafts[(int64_t)db + j0 + tid];
            if (t < columns) {
                if (wave == t) {
                    double rest = p;
                    if (judged) {
                        double q_at = lane < a.k && id == d ? 1.0 : 0.0;
                        if (listed) {
                            q_at = 0.0;
                            // from the last, so that the first entry of an id stays
                            for (int32_t i = nq - 1; i >= 0; --i) {
                                const double qi = lane_value(q, i);
                                if (__builtin_amdgcn_readlane(qid, i) == id) q_at = qi;
                            }
                        }
                        const double diff = p - q_at;
                        rest = diff > 0.0 ? diff : 0.0;
                        if (__ballot(rest > 0.0) == 0ull) rest = p;
                    }
                    const double sums = running_sum(rest);
                    const double target = philox_uniform(a.seed, a.offset, (uint32_t)c, 2u) * lane_value(sums, a.k - 1);
                    const unsigned long long some = __ballot(rest > 0.0);
                    const unsigned long long above = __ballot(rest > 0.0 && sums > target);
                    // (a product rounded up to the total leaves none above it: the last entry that can be drawn)
                    const uint32_t pick = above ? first_lane(above) : some ? 63u - (uint32_t)__builtin_clzll(some) : 0u;
                    const int32_t next = __builtin_amdgcn_readlane(id, (int)pick);
                    if (lane == 0) out[j0 + t] = next;
                }
                count = j0 + t + 1u;
                break;
            }
            __syncthreads();  // the next step writes refused again
        }
    }
    for (uint32_t i = count + tid; i < (uint32_t)a.max_tokens; i += kWavesPerLane * 64u) out[i] = -1;
    if (tid == 0) a.out_count[l] = (int32_t)count;
}

template <class DT>
hipError_t launch_dt(const VerifyArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.v.lanes);
    // Four waves for up to four columns a lane (2,048 lanes of 4: 9.5 us, with
    // eight waves 12.4), eight for more (512 lanes of 8: 7.2, with four 7.6).
    // Sixteen would judge columns that an earlier refusal makes useless (512
    // lanes of 16: 11.1 against 7.4; both steps are needed only where the first
    // eight are accepted).
    if ((a.v.C + a.v.lanes - 1) / a.v.lanes <= 4) hipLaunchKernelGGL((verify_kernel<DT, 4>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((verify_kernel<DT, 8>), grid, dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
    return a.v.dtype == TOPK_BF16 ? launch_dt<Bf16>(a, stream) : launch_dt<F32>(a, stream);
}

}  // namespace topk
