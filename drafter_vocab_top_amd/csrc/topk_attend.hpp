// What the kernels of topk_cols_attend share: how the work of all lanes is cut
// into parts, which places a row sees, and the weights of a softmax.
#pragma once

#include "topk_cache.hpp"

namespace topk {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNone = -__builtin_inff();
// x, and no reason to compute what depends on it ahead of the loop that asks (the registers
// would be missed in the loop).
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// What the second kernel needs to know of an item that a part ends in.
struct Cut {
    uint32_t more;  // further parts that hold pieces of it; 0: nothing to join
    uint32_t first_row, rows, first_col, head;
    uint32_t pad[3];
};

// Sizes of a launch that do not depend on what the device holds.
struct Shape {
    uint32_t workers;  // workgroups, a power of two
    uint32_t shift;    // its logarithm
    uint32_t rows;     // of an item
    Divisor group;     // query heads of a key head
    Cut* cuts;
    float* sums;       // [2 workers][rows][2]: maximum and sum
    float* parts;      // [2 workers][rows][DP]
};

struct LaneWork {
    uint32_t cb, n, len, end;  // first column, columns, places before them, places
    uint32_t first, steps;     // its first step, and how many
    uint32_t tiles;            // items of a key head

    // Some row may not see places from here on: the lane's columns, and what lies past the table's row (where the
    // lane's tokens do not fit in it, this is before len).
    __device__ __forceinline__ uint32_t open() const { return min_u32(len, end); }
};

template <uint32_t kStep>
__device__ __forceinline__ LaneWork lane_work(const AttendArgs& args, const Shape& sh, uint32_t l, int32_t b, int32_t e, int32_t len) {
    LaneWork w;
    uint32_t ce;
    args.cols.cut(l, b, e, w.cb, ce);
    w.n = ce - w.cb;
    w.len = (uint32_t)max_i32(len, 0);
    w.end = (uint32_t)min((uint64_t)w.len + w.n, (uint64_t)args.places);
    const uint32_t all = (w.end + kStep - 1u) / kStep;
    const uint32_t window = (uint32_t)args.a.window;
    w.first = 0;
    if (window && w.len + 1u > window) w.first = min_u32((w.len + 1u - window) / kStep, all - 1u);
    w.steps = all - w.first;
    w.tiles = (w.n * sh.group.d + sh.rows - 1u) / sh.rows;
    if (w.n == 0) w.steps = w.tiles = 0;
    return w;
}

__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t x, uint32_t by) {
    return ((uint64_t)(uint32_t)__shfl_up((int)(uint32_t)(x >> 32), by) << 32) | (uint32_t)__shfl_up((int)(uint32_t)x, by);
}

__device__ __forceinline__ uint32_t bcast(uint32_t x, uint32_t lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, (int)lane);
}

__device__ __forceinline__ uint64_t bcast(uint64_t x, uint32_t lane) {
    return ((uint64_t)bcast((uint32_t)(x >> 32), lane) << 32) | bcast((uint32_t)x, lane);
}

// The steps of all lanes (the sum), or with `find` the lane that step `at` of
// them belongs to; `before` gets the steps of the lanes before it.  It is looked
// for from `lane` on, `before` being the steps of those before that one: a
// workgroup's steps only grow, so it passes each lane once.  All of a wave's
// threads take part, 64 lanes at a time.
template <uint32_t kStep>
__device__ __forceinline__ uint64_t all_steps(const AttendArgs& args, const Shape& sh, bool find, uint64_t at, uint64_t& before,
                                              uint32_t& lane, LaneWork& work) {
    const uint32_t lanes = (uint32_t)args.a.lanes, id = threadIdx.x & 63u;
    uint64_t sum = find ? before : 0;
    for (uint32_t l0 = find ? lane : 0; l0 < lanes; l0 += 64u) {
        const uint32_t l = min_u32(l0 + id, lanes - 1u);
        const int32_t* s = args.cols.at(l);
        const int32_t b = s[0], e = s[args.cols.start ? 1 : 0], len = args.a.lens[l];
        LaneWork w = lane_work<kStep>(args, sh, l, b, e, len);
        if (l0 + id >= lanes) w.steps = 0;
        const uint64_t own = (uint64_t)w.steps * w.tiles * (uint32_t)args.cache.c.heads;
        uint64_t run = own;
#pragma unroll
        for (uint32_t d = 1; d < 64u; d <<= 1) {
            const uint64_t up = shfl_up_u64(run, d);
            if (id >= d) run += up;
        }
        if (find) {
            const unsigned long long m = __ballot(sum + run > at);
            if (m) {
                const uint32_t k = (uint32_t)__builtin_ctzll(m);
                before = sum + bcast(run, k) - bcast(own, k);
                lane = l0 + k;
                work.cb = bcast(w.cb, k);
                work.n = bcast(w.n, k);
                work.len = bcast(w.len, k);
                work.end = bcast(w.end, k);
                work.first = bcast(w.first, k);
                work.steps = bcast(w.steps, k);
                work.tiles = bcast(w.tiles, k);
                return sum;
            }
        }
        sum += bcast(run, 63u);
    }
    return sum;
}

// x of lane - N of the same 16 lanes, or of the end of an earlier 16 (0 where there is none).
template <int kCtrl, int kRowMask>
__device__ __forceinline__ uint32_t dpp_add(uint32_t x) {
    return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRowMask, 0xF, true);
}

// The lanes' steps, read once where a wave's threads can keep them: up to 64 lanes with less than 2^26 each.
template <uint32_t kStep>
struct Steps {
    LaneWork own;  // of the lane of this thread
    uint32_t run;  // steps up to its end
    bool kept;
    uint64_t total;

    __device__ __forceinline__ Steps(const AttendArgs& args, const Shape& sh) {
        kept = false;
        uint64_t before;
        uint32_t lane;
        const uint32_t lanes = (uint32_t)args.a.lanes, id = threadIdx.x & 63u;
        if (lanes <= 64u) {
            const uint32_t l = min_u32(id, lanes - 1u);
            const int32_t* s = args.cols.at(l);
            own = lane_work<kStep>(args, sh, l, s[0], s[args.cols.start ? 1 : 0], args.a.lens[l]);
            const uint64_t all = id < lanes ? (uint64_t)own.steps * own.tiles * (uint32_t)args.cache.c.heads : 0u;
            if (!__ballot(all >> 26)) {
                run = (uint32_t)all;
                run = dpp_add<0x111, 0xF>(run);  // row_shr:1
                run = dpp_add<0x112, 0xF>(run);
                run = dpp_add<0x114, 0xF>(run);
                run = dpp_add<0x118, 0xF>(run);
                run = dpp_add<0x142, 0xA>(run);  // row_bcast:15
                run = dpp_add<0x143, 0xC>(run);  // row_bcast:31
                kept = true;
                total = bcast(run, 63u);
            }
        }
        if (!kept) total = all_steps<kStep>(args, sh, false, 0, before, lane, own);
    }

    // The lane that step `at` belongs to, and the steps of those before it (at first those of a lane that is not behind it).
    __device__ __forceinline__ void find(const AttendArgs& args, const Shape& sh, uint64_t at, uint64_t& before, uint32_t& lane, LaneWork& w) const {
        if (!kept) {
            all_steps<kStep>(args, sh, true, at, before, lane, w);
            return;
        }
        lane = (uint32_t)__builtin_ctzll(__ballot(run > (uint32_t)at));
        w.cb = bcast(own.cb, lane);
        w.n = bcast(own.n, lane);
        w.len = bcast(own.len, lane);
        w.end = bcast(own.end, lane);
        w.first = bcast(own.first, lane);
        w.steps = bcast(own.steps, lane);
        w.tiles = bcast(own.tiles, lane);
        before = bcast(run, lane) - w.steps * w.tiles * (uint32_t)args.cache.c.heads;
    }
};

// A condition that is the same in all lanes, as the compiler has to know: a matrix
// instruction takes no notice of lanes that are switched off, so none may
// stand in a branch that is taken by switching them off.
__device__ __forceinline__ bool uniform(bool x) { return __builtin_amdgcn_readfirstlane(x ? 1 : 0) != 0; }

__device__ __forceinline__ uint32_t divide(uint64_t a, uint32_t b) {
    return (a >> 32) == 0 ? (uint32_t)a / b : (uint32_t)(a / b);
}

// Bits of places [a, b) among the 32 from `base` on.
__device__ __forceinline__ uint32_t range_bits(uint32_t a, uint32_t b, uint32_t base) {
    const uint32_t lo = a > base ? min_u32(a - base, 32u) : 0u, hi = b > base ? min_u32(b - base, 32u) : 0u;
    return lo < hi ? (~0u >> (32u - hi)) & (~0u << lo) : 0u;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ int32_t from_lane(int32_t x, uint32_t lane) { return __builtin_amdgcn_ds_bpermute((int)(lane << 2), x); }

__device__ __forceinline__ float max_over_groups(float x) {
    x = __builtin_fmaxf(x, __shfl_xor(x, 16));
    return __builtin_fmaxf(x, __shfl_xor(x, 32));
}

// Two e4m3 elements times a power of two, as bfloat16.
template <bool kHigh>
__device__ __forceinline__ uint32_t widen(uint32_t x, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, kHigh));
}

// The places that a row sees among the 32 from `base` on, as bits: `column` is
// the row's, `low` the first place that it sees of those before the columns.
__device__ __forceinline__ uint32_t seen_bits(const AttendArgs& args, const LaneWork& w, uint32_t column, uint32_t low, uint32_t base) {
    const topk_attend_args& a = args.a;
    asm volatile("" : "+s"(base));  // (nothing of this is computed where no row asks for it)
    uint32_t bits = range_bits(low, w.open(), base);
    if (base + 32u > w.len) {
        uint32_t own;
        if (a.mask) {
            const uint32_t* row = a.mask + (int64_t)(w.cb + column) * a.mask_ld;
            const uint32_t i0 = base > w.len ? base - w.len : 0u, word = i0 >> 5, words = (uint32_t)a.mask_ld;
            uint32_t x0 = word < words ? row[word] : 0u;
            uint32_t x1 = word + 1u < words ? row[word + 1u] : 0u;
            // (both are waited for here: a wait behind the branch would be one for keys and values too, in every step)
            asm volatile("" : "+v"(x0), "+v"(x1));
            own = base >= w.len ? (uint32_t)((((uint64_t)x1 << 32) | x0) >> (i0 & 31u)) : x0 << (w.len - base);
        } else {
            const uint32_t window = (uint32_t)a.window;
            own = range_bits(window && column + 1u > window ? w.len + (column + 1u - window) : w.len, w.len + column + 1u, base);
        }
        bits |= own & range_bits(w.len, w.end, base);
    }
    return bits;
}

// The first place that column j of the lane sees of those before the columns.
__device__ __forceinline__ uint32_t first_seen(const AttendArgs& args, const LaneWork& w, uint32_t j) {
    const topk_attend_args& a = args.a;
    if (!a.window) return 0;
    const uint32_t position = a.positions ? (uint32_t)max_i32(a.positions[w.cb + j], (int32_t)w.len) : w.len + j;
    return position + 1u > (uint32_t)a.window ? position + 1u - (uint32_t)a.window : 0u;
}

// The largest of a wave's values, of which each 16 lanes have all.
__device__ __forceinline__ uint32_t max_of_16(uint32_t x) {
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) x = max_u32(x, (uint32_t)__shfl_xor((int)x, s));
    return bcast(x, 0u);
}

// Scores of 16 kQueries queries against 32 kTiles places become weights: lane 16 g + r has query r of each 16 and
// places 4 g + i and 16 + 4 g + i of each 32.  m, sum and o (16 x 16 tiles, a query in each column) are the running
// maximum, sum and output, all in binary32.  The weights are rounded to bfloat16, which the products with values take:
// each is off by at most 2^-8 of itself, whatever its size (binary16 would be nearer, but neither it nor its products
// reach as far as bfloat16 values do; two bfloat16 halves would be half as many products again).  The sum is a product
// with ones, of the weights as they are rounded, so that a common part of their errors cancels.  Over 131,072 places
// outputs are off by 0.0023 of their size on the whole, of which 0.0017 are their own rounding.  `seen`: with `masked`,
// the places that each query sees.  (m, sum and o may be of more queries: the first ones are these.)
template <int kTiles, int kQueries, int kOut, int kAll>
__device__ __forceinline__ void weigh(f32x4 (&s)[kTiles][kQueries][2], bool masked, const uint32_t (&seen)[kTiles][kQueries], float factor,
                                      uint32_t g, float (&m)[kAll], f32x4 (&sum)[kAll], f32x4 (&o)[kAll][kOut],
                                      bf16x8 (&weights)[kTiles][kQueries]) {
    if (masked) {
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
            for (int n = 0; n < kQueries; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][n][t][e] = (seen[u][n] >> (t * 16 + (int)g * 4 + e)) & 1u ? s[u][n][t][e] : kNone;
    }
    float top[kQueries];
    bool grown = false;
#pragma unroll
    for (int n = 0; n < kQueries; ++n) {
        top[n] = kNone;
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                top[n] = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(top[n], s[u][n][t][0]), s[u][n][t][1]), s[u][n][t][2]), s[u][n][t][3]);
        top[n] *= factor;
        grown |= top[n] > m[n] + 8.0f;
    }
    if (__ballot(grown)) {
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            const float now = __builtin_fmaxf(m[n], max_over_groups(top[n]));
            const float old = __builtin_amdgcn_exp2f(m[n] - (now == kNone ? 0.0f : now));
            m[n] = now;
            sum[n][0] *= old;  // (the product's rows are alike, and the first is the one that is read)
#pragma unroll
            for (int i = 0; i < kOut; ++i) o[n][i] *= old;
        }
    }
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int u = 0; u < kTiles; ++u)
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            const float zero = m[n] == kNone ? 0.0f : m[n];
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][n][e >> 2][e & 3], factor, -zero));
            u32x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
            weights[u][n] = __builtin_bit_cast(bf16x8, y);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, ones), weights[u][n], sum[n], 0, 0, 0);
        }
}

// 2^(byte - 127); of 255 an infinity, whose exponent the widening takes as NaN.
__device__ __forceinline__ float power_of(uint32_t byte) { return __builtin_bit_cast(float, byte ? byte << 23 : 0x400000u); }

// Clears what is not finite of two bfloat16 values; `odd` gets a bit where there is any.
__device__ __forceinline__ uint32_t only_finite(uint32_t x, uint32_t& odd) {
    // an exponent of ones and one more carry into the sign's place
    const uint32_t b = ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    odd |= b;
    return x & ~((b << 1) - (b >> 15));
}

// 0 times two bfloat16 values: 0, or NaN where one is not finite.
__device__ __forceinline__ uint32_t times_zero(uint32_t x) {
    const uint32_t b = ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;  // (as above)
    return ((b << 1) - (b >> 15)) & 0x7FFF7FFFu;
}

// Queries as the products take them: such that the scores grow with the products, by a factor that is positive.  (One
// branch, which positive scales skip: a choice for each element made one lane's columns over 2,048 places 2 % slower.)
template <int kQueries, int kKeySteps>
__device__ __forceinline__ void sign_queries(bf16x8 (&q)[kQueries][kKeySteps], float scale) {
    if (scale > 0.0f) return;
#pragma unroll
    for (int n = 0; n < kQueries; ++n)
#pragma unroll
        for (int s = 0; s < kKeySteps; ++s) {
            u32x4 x = __builtin_bit_cast(u32x4, q[n][s]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = scale < 0.0f ? x[i] ^ 0x80008000u : times_zero(x[i]);
            q[n][s] = __builtin_bit_cast(bf16x8, x);
        }
}

// The weight of place `key` of 32 for this lane's query.
__device__ __forceinline__ float weight_of(const bf16x8& weights, uint32_t key, uint32_t r) {
    const u32x4 y = __builtin_bit_cast(u32x4, weights);
    const uint32_t word = (key >> 4) * 2u + ((key >> 1) & 1u);  // places 16 t + 4 g + i: word 2 t + i / 2 of group g
    const uint32_t both = word == 0 ? y[0] : word == 1 ? y[1] : word == 2 ? y[2] : y[3];
    const uint32_t x = (uint32_t)from_lane((int32_t)both, r + 16u * ((key >> 2) & 3u));
    return __builtin_bit_cast(float, key & 1u ? x & 0xFFFF0000u : x << 16);
}

// DP of the kernels: dim rounded up.
inline int padded_dim(const AttendArgs& a) { return a.cache.c.dim <= 64 ? 64 : a.cache.c.dim <= 128 ? 128 : 256; }

constexpr uint32_t kRowsStep = 64;  // places of a step where a workgroup's waves share the rows
void launch_attend_rows(const AttendArgs& a, const Shape& s, hipStream_t stream);

}  // namespace topk
