// Verification of a tree of drafts against the target's top-k lists, for
// gfx950, from given random numbers.
//
// At column c, with weights w = p_c and their sum W, each child x in turn is
// accepted if u_x q(x) < w(x) / W; a refused one leaves w = max(w - W q, 0), the
// part of the normalised weights above q, scaled by W (a scale changes nothing:
// only quotients by the new sum are used).  Where no child is accepted the
// token is drawn from what is left.
//
// One workgroup per lane, one wave per column: what a column's children meet does
// not depend on the other columns, so the waves judge the current column, its
// children and columns behind them at once, and the path through them is then a
// walk in LDS.
//
// A chain of latencies bounds it: one lane of up to 16 columns and lists of 20 takes
// 4.5 us, 512 lanes of up to 64 columns and lists of 64 take 12 (880 instructions
// a wave, in binary64 and one after the other).
//
// The decisions are integers made by floating point, so every step is IEEE
// double in a fixed order with no contraction.
#include "topk_cache.hpp"
#include "topk_lists.hpp"

namespace topk {

namespace {

// The probabilities in a draft list of this lane's target token (0 where it has
// none, and past the target list): that of the first entry with its id.
__device__ __forceinline__ double probability_at(int32_t id, double q, int32_t qid, int32_t nq) {
    int32_t at = -1;
    for (int32_t i = nq - 1; i >= 0; --i)  // from the last, so that the first entry of an id stays
        at = __builtin_amdgcn_readlane(qid, i) == id ? i : at;
    const uint64_t b = __builtin_bit_cast(uint64_t, q);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(at << 2, (int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(at << 2, (int)(uint32_t)(b >> 32));
    return at < 0 ? 0.0 : __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// 64 columns of a lane, one for each thread of a wave: those from 64 q on.
struct Columns {
    int32_t parent, token;
    float u;
    __device__ __forceinline__ void load(const topk_verify_tree_args& a, uint32_t cb, uint32_t n, uint32_t q) {
        const uint32_t x = q * 64u + (threadIdx.x & 63u);
        const int64_t c = (int64_t)cb + min_u32(x, n - 1u);
        parent = x < n ? a.parents[c] : -1;
        token = a.tokens[c];
        u = a.uniforms[2 * c];
    }
};

// The column that a wave judges when the path stands at column `now`: that for
// wave 0, its children for the next ones (one of them comes next), the columns
// behind it for the rest, all among the 64 that `now` is one of.  Where the
// waves can judge all columns they take them in order.  n: none.
template <uint32_t kWaves>
__device__ __forceinline__ uint32_t column_of_wave(const Columns& c, uint32_t n, uint32_t now, uint32_t wave) {
    if (n - now <= kWaves || wave == 0) return now + wave;
    const uint32_t x = (now & ~63u) + (threadIdx.x & 63u);
    const bool behind = x > now && x < n;
    unsigned long long kids = __ballot(behind && c.parent == (int32_t)now);
    const unsigned long long rest = __ballot(behind && c.parent != (int32_t)now);
    uint32_t skip = wave - 1u;
    const uint32_t many = (uint32_t)__builtin_popcountll(kids);
    if (skip >= many) {
        skip -= many;
        kids = rest;
    }
    for (uint32_t i = 0; i < skip; ++i) kids &= kids - 1ull;
    return kids ? (now & ~63u) + first_lane(kids) : n;
}

template <class DT, uint32_t kWaves>
__global__ __launch_bounds__(kWaves * 64) void verify_tree_kernel(VerifyTreeArgs args) {
#pragma clang fp contract(off)
    __shared__ int32_t chosen[kWaves];   // the accepted child of each column, or -1
    __shared__ uint32_t judged[kWaves];  // the columns
    const topk_verify_tree_args& a = args.v;
    const uint32_t l = blockIdx.x, tid = threadIdx.x;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const int32_t lane = (int32_t)(tid & 63u);
    int32_t* tokens = a.out_tokens + (int64_t)l * a.max_tokens;
    int32_t* columns = a.out_columns + (int64_t)l * a.max_tokens;
    const uint32_t most = (uint32_t)a.max_tokens;
    uint32_t cb, ce;
    args.cols.range(l, cb, ce);
    const uint32_t n = ce - cb;
    uint32_t t = 0;  // accepted drafts
    bool some = n > 0;
    uint32_t now = 0;  // the column where the path stands
    Columns first64;  // (most trees have no more)
    if (some) first64.load(a, cb, n, 0);
    while (some) {
        Columns near = first64;
        if (now >= 64u && n - now > kWaves) near.load(a, cb, n, now >> 6);
        const uint32_t j = column_of_wave<kWaves>(near, n, now, wave);
        double w = 0.0, p = 0.0;
        int32_t id = 0;
        if (j < n) {  // wave-uniform
            const int64_t c = (int64_t)cb + j;
            double v, v0, qv = 0.0, qv0 = 0.0;
            int32_t qid = 0;
            id = a.target_ids[c * a.k + (lane < a.k ? lane : 0)];
            load_entry<DT>(a.target_values, c, a.k, v, v0);
            if (a.draft_values) {
                qid = a.draft_ids[c * a.kq + (lane < a.kq ? lane : 0)];
                load_entry<DT>(a.draft_values, c, a.kq, qv, qv0);
            }
            int32_t np, nq = 0;
            p = probability(v, v0, a.k, a.temperature, a.top_p, np);
            w = p;
            double W = 1.0, q = 0.0, q_at = 0.0;
            bool have_q = false, have_at = false;
            int32_t accepted = -1;
            for (uint32_t x0 = (j + 1u) & ~63u; x0 < n && accepted < 0; x0 += 64u) {
                Columns columns_of = first64;
                if (x0) columns_of.load(a, cb, n, x0 >> 6);
                const int32_t token = columns_of.token;
                const float u = columns_of.u;
                unsigned long long kids = __ballot(x0 + (uint32_t)lane > j && columns_of.parent == (int32_t)j);
                while (kids) {
                    const uint32_t i = first_lane(kids);
                    kids &= kids - 1ull;
                    const int32_t d = __builtin_amdgcn_readlane(token, (int)i);
                    const double u_x = (double)__builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, u), (int)i));
                    double q_x = 1.0;
                    if (a.draft_values) {
                        if (!have_q) q = probability(qv, qv0, a.kq, a.temperature, a.top_p, nq);
                        have_q = true;
                        q_x = probability_of(d, qid, q, a.kq);
                    }
                    const double w_x = probability_of(d, id, w, a.k);
                    if (u_x * q_x * W < w_x) {
                        accepted = (int32_t)(x0 + i);
                        break;
                    }
                    if (!a.draft_values) {
                        q_at = lane < a.k && id == d ? 1.0 : 0.0;
                    } else if (!have_at) {
                        q_at = probability_at(id, q, qid, nq);
                        have_at = true;
                    }
                    const double left = w - W * q_at;
                    const double rest = left > 0.0 ? left : 0.0;
                    const double total = lane_value(running_sum(rest), a.k - 1);
                    w = total > 0.0 ? rest : p;
                    W = total > 0.0 ? total : 1.0;
                }
            }
            if (lane == 0) chosen[wave] = accepted;
        }
        if (lane == 0) judged[wave] = j;
        __syncthreads();
        bool last = false;
        uint32_t slot = 0;  // of the column where the path stands (the first is judged)
        while (slot < kWaves) {
            const int32_t down = chosen[slot];
            if (tid == 0) columns[t] = (int32_t)now;
            last = down < 0 || t + 1u == most;
            if (last) break;
            if (tid == 0) tokens[t] = a.tokens[(int64_t)cb + (uint32_t)down];
            ++t;
            now = (uint32_t)down;
            slot = 0;
            while (slot < kWaves && judged[slot] != now) ++slot;
        }
        if (last) {
            if (wave == slot) {
                if (t + 1u == most) w = p;  // no child was judged
                const double sums = running_sum(w);
                const double target = (double)a.uniforms[2 * ((int64_t)cb + now) + 1] * lane_value(sums, a.k - 1);
                const unsigned long long positive = __ballot(w > 0.0);
                const unsigned long long above = __ballot(w > 0.0 && sums > target);
                // (a product rounded up to the total leaves none above it: the last entry that can be drawn)
                const uint32_t pick = above ? first_lane(above) : positive ? 63u - (uint32_t)__builtin_clzll(positive) : 0u;
                const int32_t next = __builtin_amdgcn_readlane(id, (int)pick);
                if (lane == 0) tokens[t] = next;
            }
            break;
        }
        __syncthreads();  // the next step writes chosen again
    }
    const uint32_t count = some ? t + 1u : 0u;
    for (uint32_t i = count + tid; i < most; i += kWaves * 64u) {
        tokens[i] = -1;
        columns[i] = -1;
    }
    if (tid == 0) a.out_count[l] = (int32_t)count;
}

template <class DT>
hipError_t launch_dt(const VerifyTreeArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.v.lanes);
    // Eight waves while the card has room for them (256 lanes of 8 columns with two levels 4.2 us, with four waves
    // 5.3; a chain of 8 accepted drafts 6.0 and 6.9), four where more lanes than that share it (1,024 lanes: 7.2 and
    // 9.2 us, with eight waves 7.4 and 11.2).
    if (a.v.lanes <= 256) hipLaunchKernelGGL((verify_tree_kernel<DT, 8>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((verify_tree_kernel<DT, 4>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_tree(const VerifyTreeArgs& a, hipStream_t stream) {
    return a.v.dtype == TOPK_BF16 ? launch_dt<Bf16>(a, stream) : launch_dt<F32>(a, stream);
}

}  // namespace topk
