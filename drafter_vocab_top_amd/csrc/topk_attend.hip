// Attention of a round's columns over the paged cache, for gfx950.
//
//   out = sum_p w_p v_p / sum_p w_p,  w_p = exp(s_p - m),  s_p = scale (q . k_p)
//
// The columns of a lane and the query heads of a key head share that key head's
// keys and values: together they are the rows of one matrix, cut into items of
// R = 16 kQueries rows.  An item's places are cut into steps of 128, 32 for
// each of a workgroup's four waves.
//
// Products are 16 x 16 x 32 matrix instructions on transposed operands.
// S^T = K Q^T has a query in each lane's column and keys in its registers, so
// the running maximum and sum of a softmax need no other lane, and the weights
// come out of it as the right operand of O^T = V^T W^T needs them: with lane
// 16 g + r holding keys 4 g + i and 16 + 4 g + i, i < 4, the contraction just
// runs over the 32 keys in that order.  Keys go from memory to the registers
// where the instruction wants them (a lane has 16 bytes of one key), values
// likewise: lane 16 g + r reads elements 8 r .. 8 r + 7 of its eight keys (rows
// of 256 contiguous bytes), and byte permutations pair the keys of each element.
// So nothing passes through LDS until the end.  The next keys are on their way
// while weights are made and values multiplied, the next values while keys are.
//
// The maximum is only raised when a score passes it by more than 2^8 (weights
// then stay below 2^8, which costs nothing in floating point), so most steps
// neither exchange maxima nor rescale.
//
// The work, items times steps over all lanes, is cut into equal parts for the
// workgroups of one wave of launches, whatever the lanes' lengths (read on the
// device).  A part that ends inside an item leaves its partial maximum, sums
// and output in the workspace, and a second kernel joins them.
//
// Memory bounds it: 2 lanes of 6 columns over 98,304 bfloat16 places of 8 key
// heads of 128 are 806 MB in 152 us, 5.3 TB/s where a large copy makes 5.4 (140
// us of it in this kernel, 10 in the join).  An e4m3 cache, whose rows are 128
// bytes, is read at 4.1 TB/s (64 lanes of 6 columns over 6,144 places: 826 MB in
// 200 us; the same with every block in cache 111 us); twice as many places in
// flight did not change that.  One lane over 2,048 places is a chain of
// latencies: 15 us, 12 of them here (lengths, table, keys, and the sums of four
// waves).
#include <algorithm>

#include "topk_attend.hpp"

namespace topk {

namespace {

constexpr uint32_t kStep = 128;       // places of a step
constexpr uint32_t kTile = 32;        // of one wave
// Workgroups that share the parts to join, for each two rows (DP = 128) of an item.  With 16, 64 and 256 of them one
// lane's columns over 2,048 places take 15.9, 16.1 and 17.2 us, 64 lanes of 64 rows 217, 208 and 216.
constexpr uint32_t kJoinGroups = 64;

// DP: dim rounded up to 64, 128 or 256; kWhole: dim is DP.
template <int DP, bool kWhole, bool kFp8, int kQueries>
struct Item {
    static constexpr int kSize = kFp8 ? 1 : 2;
    static constexpr int kKeySteps = DP / 32;                 // products of a score
    static constexpr int kKeyLoads = kFp8 ? DP / 64 : DP / 32;
    static constexpr int kHalf = DP < 128 ? DP : 128;         // elements of a value that 16 lanes read at once
    static constexpr int kHalves = DP / kHalf;
    static constexpr int kOwn = kHalf / 16;                   // of them one lane's
    static constexpr int kValueWords = kOwn * kSize / 4;
    static constexpr int kOut = DP / 16;                      // 16 x 16 tiles of O^T for 16 queries
    static constexpr uint32_t kRows = 16 * kQueries;

    bf16x8 q[kQueries][kKeySteps];
    u32x4 k[2][kKeyLoads];
    uint32_t v[8][kHalves][kValueWords];
    f32x4 o[kQueries][kOut];
    float m[kQueries];
    f32x4 sum[kQueries];
    uint32_t scales, next_scales;  // of key lane & 31: lanes 0 - 31 the keys', 32 - 63 the values'
    // One lane's share of a tile's addresses: place base + (lane & 31).
    struct Places {
        uint32_t id, in_block;
    };

    __device__ __forceinline__ Places lookup(const AttendArgs& a, const int32_t* table, uint32_t base, uint32_t end, uint32_t lane) const {
        const uint32_t p = min_u32(base + (lane & 31u), end - 1u), b = a.cache.block.div(p);
        Places s;
        s.id = (uint32_t)min_i32(max_i32(table[b], 0), (int32_t)a.cache.c.blocks - 1);
        s.in_block = p - b * a.cache.block.d;
        return s;
    }

    // Offset in 16 bytes of the row of the place that lane `key` looked up.
    struct Rows {
        uint32_t own;
        __device__ __forceinline__ uint32_t of(uint32_t key) const { return (uint32_t)from_lane((int32_t)own, key); }
    };
    __device__ __forceinline__ Rows rows_of(const AttendArgs& a, const Places& s) const { return Rows{a.cache.row16(s.id, s.in_block)}; }

    __device__ __forceinline__ void load_scales(const AttendArgs& a, const Places& s, uint32_t head, uint32_t lane) {
        if constexpr (kFp8) {
            const topk_cache& c = a.cache.c;
            const uint8_t* from = (lane & 32u) ? c.value_scales : c.key_scales;
            next_scales = (from + (int64_t)head * c.scale_head_stride)[a.cache.scale_row(s.id, s.in_block)];
        }
    }

    __device__ __forceinline__ float scale_from(uint32_t lane) const {
        return power_of((uint32_t)from_lane((int32_t)scales, lane));
    }

    __device__ __forceinline__ void load_keys(const AttendArgs& a, const uint8_t* keys, const Rows& at, uint32_t lane) {
        const uint32_t g = lane >> 4;
        const int32_t dim = a.cache.c.dim;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* row = past16(keys, at.of((uint32_t)t * 16u + (lane & 15u))) + (kWhole ? g * 16u : 0u);
#pragma unroll
            for (int i = 0; i < kKeyLoads; ++i) {
                // (past the row: its start, cleared below)
                const int32_t d = i * (64 / kSize) + (kWhole ? 0 : (int32_t)g * (16 / kSize));
                k[t][i] = *reinterpret_cast<const u32x4*>(row + (kWhole || d < dim ? d * kSize : 0));
            }
        }
    }

    __device__ __forceinline__ void load_values(const AttendArgs& a, const uint8_t* values, const Rows& at, uint32_t lane) {
        const uint32_t r = lane & 15u, g = lane >> 4;
        const int32_t dim = a.cache.c.dim;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint8_t* row = past16(values, at.of((uint32_t)(e >> 2) * 16u + g * 4u + (uint32_t)(e & 3))) + (kWhole ? r * (kOwn * kSize) : 0u);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const int32_t d = h * kHalf + (kWhole ? 0 : (int32_t)r * kOwn);
                const uint8_t* p = row + (kWhole || d < dim ? d * kSize : 0);
                if constexpr (kValueWords == 4) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[e][h][i] = x[i];
                } else if constexpr (kValueWords == 2) {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
                    v[e][h][0] = x[0];
                    v[e][h][1] = x[1];
                } else {
                    v[e][h][0] = *reinterpret_cast<const uint32_t*>(p);
                }
            }
        }
    }

    // The left operand of product `step` of keys 16 t .. 16 t + 15.
    __device__ __forceinline__ bf16x8 key_operand(const AttendArgs& a, int t, int step, float scale, uint32_t lane) const {
        u32x4 x;
        int32_t d;  // this lane's first element
        const int32_t g = (int32_t)(lane >> 4);
        if constexpr (kFp8) {
            const u32x4 raw = k[t][step / 2];
            const uint32_t w0 = raw[2 * (step & 1)], w1 = raw[2 * (step & 1) + 1];
            x[0] = widen<false>(w0, scale);
            x[1] = widen<true>(w0, scale);
            x[2] = widen<false>(w1, scale);
            x[3] = widen<true>(w1, scale);
            d = (step / 2) * 64 + g * 16 + (step & 1) * 8;
        } else {
            x = k[t][step];
            d = step * 32 + g * 8;
        }
        if (!kWhole && d >= a.cache.c.dim) x = u32x4{0u, 0u, 0u, 0u};
        return __builtin_bit_cast(bf16x8, x);
    }

    // The element of a row that this lane's operands of `step` start with.
    __device__ __forceinline__ static int32_t operand_element(int step, uint32_t lane) {
        const int32_t g = (int32_t)(lane >> 4);
        return kFp8 ? (step / 2) * 64 + g * 16 + (step & 1) * 8 : step * 32 + g * 8;
    }

    // Adds the values that are not finite, each to the rows that see it.
    __device__ __forceinline__ void add_odd(const AttendArgs& a, const int32_t* table, const uint8_t* values, uint32_t head, uint32_t base,
                                            uint32_t end, const uint32_t (&seen)[kQueries], const bf16x8 (&weights)[kQueries], uint32_t lane) {
        const uint32_t r = lane & 15u, g = lane >> 4;
        const Places s = lookup(a, table, base, end, lane);
        const Rows at = rows_of(a, s);
        uint32_t scale_byte = 0;
        if constexpr (kFp8) {
            const topk_cache& c = a.cache.c;
            scale_byte = c.value_scales[(int64_t)head * c.scale_head_stride + a.cache.scale_row(s.id, s.in_block)];
        }
        for (uint32_t key = 0; key < kTile && base + key < end; ++key) {
            const uint8_t* row = past16(values, at.of(key));
            const float scale = power_of((uint32_t)from_lane((int32_t)scale_byte, key));
            float weight[kQueries];
            bool sees[kQueries];
#pragma unroll
            for (int n = 0; n < kQueries; ++n) {
                weight[n] = weight_of(weights[n], key, r);
                sees[n] = seen[n] >> key & 1u;
            }
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t d = h * kHalf + ((int32_t)g * 4 + e) * kOwn;
                    const uint8_t* from = row + (kWhole || d < a.cache.c.dim ? d * kSize : 0);
#pragma unroll
                    for (int i = 0; i < kOwn; i += 2) {
                        uint32_t x;
                        if constexpr (kFp8) x = widen<false>(*reinterpret_cast<const uint16_t*>(from + i), scale);
                        else x = *reinterpret_cast<const uint32_t*>(from + 2 * i);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float v1 = __builtin_bit_cast(float, k ? x & 0xFFFF0000u : x << 16);
#pragma unroll
                            for (int n = 0; n < kQueries; ++n)
                                if (sees[n] && !__builtin_isfinite(v1)) o[n][h * kOwn + i + k][e] += weight[n] * v1;
                        }
                    }
                }
        }
    }

    // Rows first_row .. of the lane's matrix; a row past the last is the last
    // again (it is not written).
    __device__ __forceinline__ void load_queries(const AttendArgs& args, const Shape& sh, const LaneWork& w, uint32_t head, uint32_t first_row, uint32_t lane) {
        const topk_attend_args& a = args.a;
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            const uint32_t row = min_u32(first_row + (uint32_t)n * 16u + (lane & 15u), w.n * sh.group.d - 1u);
            const uint32_t j = sh.group.div(row), h = head * sh.group.d + (row - j * sh.group.d);
            const uint16_t* from = static_cast<const uint16_t*>(a.q) + (int64_t)(w.cb + j) * a.q_stride + (int64_t)h * a.q_head_stride;
#pragma unroll
            for (int s = 0; s < kKeySteps; ++s) {
                const int32_t d = operand_element(s, lane);
                u32x4 x = u32x4{0u, 0u, 0u, 0u};
                if (kWhole || d < args.cache.c.dim) x = *reinterpret_cast<const u32x4*>(from + d);
                q[n][s] = __builtin_bit_cast(bf16x8, x);
            }
        }
        sign_queries(q, a.scale);
    }
};

template <int DP, bool kWhole, bool kFp8, int kQueries>
__global__ __launch_bounds__(256, DP < 256 ? 2 : 1) void attend_kernel(AttendArgs args, Shape sh) {
    using I = Item<DP, kWhole, kFp8, kQueries>;
    constexpr uint32_t R = I::kRows;
    constexpr uint32_t kPitch = DP + 4;  // floats of a row in LDS
    __shared__ float lds_o[4][R][kPitch];
    __shared__ float lds_m[4][R], lds_l[4][R];
    const topk_attend_args& a = args.a;
    const topk_cache& c = args.cache.c;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // consecutive parts go to one of the eight dies, whose workgroups share a cache
    const uint32_t worker = sh.workers >= 8u ? (blockIdx.x & 7u) * (sh.workers >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    uint64_t before = 0;
    uint32_t l = 0;
    LaneWork w = {};
    const Steps<kStep> steps(args, sh);
    const uint64_t total = steps.total, per = (total + sh.workers - 1u) >> sh.shift;
    uint64_t at = per * worker;
    const uint64_t stop = min(at + per, total);
    uint32_t more = 0;  // parts behind this one that hold the rest of its last item
    const float factor = a.scale == 0.0f ? 1.0f : __builtin_fabsf(a.scale) * kLog2e;
    bool found = false;
    while (at < stop) {
        if (!found || at >= before + (uint64_t)w.steps * w.tiles * (uint32_t)c.heads) steps.find(args, sh, at, before, l, w);
        found = true;
        const uint64_t in_lane = at - before;
        const uint32_t item = divide(in_lane, w.steps), step = (uint32_t)(in_lane - (uint64_t)item * w.steps);
        const uint32_t head = item / w.tiles, first_row = (item - head * w.tiles) * R;
        const uint32_t last_step = (uint32_t)min((uint64_t)w.steps, step + (stop - at));
        const int32_t* table = a.table + (int64_t)l * a.table_ld;
        const uint32_t rows = w.n * sh.group.d;

        I it;
        const uint32_t lane = opaque(threadIdx.x) & 63u, r = lane & 15u;
        const uint8_t* keys = static_cast<const uint8_t*>(c.keys) + (int64_t)head * c.head_stride * I::kSize;
        const uint8_t* values = static_cast<const uint8_t*>(c.values) + (int64_t)head * c.head_stride * I::kSize;
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            it.m[n] = kNone;
            it.sum[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < I::kOut; ++i) it.o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // (in the order in which they are waited for)
        uint32_t base = (w.first + step) * kStep + wave * kTile;
        const uint32_t stop_at = min_u32((w.first + last_step) * kStep, w.end);
        const typename I::Places now = it.lookup(args, table, base, w.end, lane);
        typename I::Places next = it.lookup(args, table, base + kStep, w.end, lane);
        it.load_queries(args, sh, w, head, first_row, lane);
        if (base < stop_at) {
            const typename I::Rows at = it.rows_of(args, now);
            it.load_scales(args, now, head, lane);
            it.load_keys(args, keys, at, lane);
            it.load_values(args, values, at, lane);
        }
        // each row's column, the first place of those before the lane's columns that it sees
        uint32_t column[kQueries], low[kQueries];
        uint32_t all_see = 0;  // all rows see the places from here up to the lane's columns
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            column[n] = sh.group.div(min_u32(first_row + (uint32_t)n * 16u + r, rows - 1u));
            low[n] = first_seen(args, w, column[n]);
            if (a.window) all_see = max_u32(all_see, max_of_16(low[n]));
        }

        for (; base < stop_at; base += kStep) {
            const bool masked = uniform(base + kTile > w.open() || base < all_see);  // some row may not see all
            const uint32_t lane = opaque(threadIdx.x & 63u), r = lane & 15u, g = lane >> 4;
            it.scales = it.next_scales;
            // scores of 32 places
            f32x4 s[1][kQueries][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float scale = kFp8 ? it.scale_from((uint32_t)t * 16u + r) : 1.0f;
#pragma unroll
                for (int n = 0; n < kQueries; ++n) s[0][n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < I::kKeySteps; ++i) {
                    const bf16x8 x = it.key_operand(args, t, i, scale, lane);
#pragma unroll
                    for (int n = 0; n < kQueries; ++n)
                        s[0][n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, it.q[n][i], s[0][n][t], 0, 0, 0);
                }
            }
            // the next keys (past the end: the last place again)
            __builtin_amdgcn_sched_barrier(0);
            const typename I::Places now = next;
            next = it.lookup(args, table, base + 2 * kStep, w.end, lane);
            const typename I::Rows at = it.rows_of(args, now);
            it.load_scales(args, now, head, lane);
            it.load_keys(args, keys, at, lane);
            __builtin_amdgcn_sched_barrier(0);

            uint32_t seen[1][kQueries] = {};
            bf16x8 weights[1][kQueries];
            if (masked) {
#pragma unroll
                for (int n = 0; n < kQueries; ++n) seen[0][n] = seen_bits(args, w, column[n], low[n], base);
            }
            weigh(s, masked, seen, factor, g, it.m, it.sum, it.o, weights);

            // values, two elements of a key in each word
            uint32_t pairs[8][I::kHalves][I::kOwn / 2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float scale = kFp8 ? it.scale_from(32u + (uint32_t)(e >> 2) * 16u + g * 4u + (uint32_t)(e & 3)) : 1.0f;
#pragma unroll
                for (int h = 0; h < I::kHalves; ++h)
#pragma unroll
                    for (int i = 0; i < I::kValueWords; ++i) {
                        const uint32_t x = it.v[e][h][i];
                        if constexpr (kFp8) {
                            pairs[e][h][2 * i] = widen<false>(x, scale);
                            pairs[e][h][2 * i + 1] = widen<true>(x, scale);
                        } else {
                            pairs[e][h][i] = x;
                        }
                    }
            }
            // A row may not see a value that is not finite, which a weight of 0 does not
            // remove: such values count as 0 here and are added below, one by one.
            uint32_t odd = 0;
            if (masked) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool past = base + (uint32_t)(e >> 2) * 16u + g * 4u + (uint32_t)(e & 3) >= w.end;
#pragma unroll
                    for (int h = 0; h < I::kHalves; ++h)
#pragma unroll
                        for (int i = 0; i < I::kOwn / 2; ++i)
                            pairs[e][h][i] = only_finite(past ? 0u : pairs[e][h][i], odd);
                }
            }
#pragma unroll
            for (int h = 0; h < I::kHalves; ++h)
#pragma unroll
                for (int i = 0; i < I::kOwn; ++i) {
                    u32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = __builtin_amdgcn_perm(pairs[2 * e + 1][h][i / 2], pairs[2 * e][h][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int n = 0; n < kQueries; ++n)
                        it.o[n][h * I::kOwn + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), weights[0][n],
                                                                                          it.o[n][h * I::kOwn + i], 0, 0, 0);
                }
            if (uniform(masked && __ballot(odd != 0u) != 0ull)) it.add_odd(args, table, values, head, base, w.end, seen[0], weights[0], lane);
            __builtin_amdgcn_sched_barrier(0);
            it.load_values(args, values, at, lane);
        }

        // the four waves' sums together
        const uint32_t tid_ = opaque(threadIdx.x), r_ = tid_ & 15u, g_ = (tid_ >> 4) & 3u;
        const bool direct = step == 0 && last_step == w.steps;
        const uint32_t slot = 2u * worker + (step == 0 ? 1u : 0u);
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            if (g_ == 0) {
                lds_m[wave][n * 16 + (int)r_] = it.m[n];
                lds_l[wave][n * 16 + (int)r_] = it.sum[n][0];
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            float top = kNone;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __builtin_fmaxf(top, lds_m[k][n * 16 + (int)r_]);
            const float mine = __builtin_amdgcn_exp2f(it.m[n] - (top == kNone ? 0.0f : top));
#pragma unroll
            for (int h = 0; h < I::kHalves; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < I::kOwn; i += 4) {
                        f32x4 x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = it.o[n][h * I::kOwn + i + k][e] * mine;
                        *reinterpret_cast<f32x4*>(&lds_o[wave][n * 16 + (int)r_][h * I::kHalf + ((int)g_ * 4 + e) * I::kOwn + i]) = x;
                    }
        }
        __syncthreads();
        // 16 threads a row
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            const uint32_t q = tid_ >> 4, part = tid_ & 15u, row = (uint32_t)n * 16u + q;
            float all = kNone, sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) all = __builtin_fmaxf(all, lds_m[k][row]);
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += lds_l[k][row] * __builtin_amdgcn_exp2f(lds_m[k][row] - (all == kNone ? 0.0f : all));
            const uint32_t d0 = part * (DP / 16);
            float y[DP / 16];
#pragma unroll
            for (int i = 0; i < DP / 16; i += 4) {
                f32x4 x = *reinterpret_cast<const f32x4*>(&lds_o[0][row][d0 + i]);
#pragma unroll
                for (int k = 1; k < 4; ++k) x += *reinterpret_cast<const f32x4*>(&lds_o[k][row][d0 + i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[i + k] = x[k];
            }
            if (!direct) {
                float* to = sh.parts + ((int64_t)slot * R + row) * DP + d0;
#pragma unroll
                for (int i = 0; i < DP / 16; i += 4) *reinterpret_cast<f32x4*>(to + i) = f32x4{y[i], y[i + 1], y[i + 2], y[i + 3]};
                if (part == 0) {
                    sh.sums[((int64_t)slot * R + row) * 2] = all;
                    sh.sums[((int64_t)slot * R + row) * 2 + 1] = sum;
                }
            } else if (first_row + row < rows && (int32_t)d0 < c.dim) {
                const uint32_t j = sh.group.div(first_row + row), h = head * sh.group.d + (first_row + row - j * sh.group.d);
                uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (int64_t)(w.cb + j) * a.out_stride +
                                                           (int64_t)h * a.out_head_stride + d0);
                const float inverse = 1.0f / sum;
#pragma unroll
                for (int i = 0; i < DP / 16; i += 2)
                    if ((int32_t)d0 + i < c.dim) to[i / 2] = sum == 0.0f ? 0u : pack_bf16(y[i] * inverse, y[i + 1] * inverse);
            }
        }
        __syncthreads();  // (the next item's maxima come here)
        at += last_step - step;
        if (at == stop && step == 0 && last_step < w.steps) {
            more = (uint32_t)(((uint64_t)(w.steps - last_step) + per - 1u) / per);
            if (tid_ == 0) sh.cuts[worker] = Cut{more, first_row, rows, w.cb, head, {}};
        }
    }
    if (more == 0 && threadIdx.x == 0) sh.cuts[worker].more = 0;
}

// Joins the pieces of the items that a part ends in: a workgroup for two rows (DP =
// 128) of one after another, its waves share the pieces.
template <int DP>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs args, Shape sh) {
    constexpr uint32_t kThreads = DP / 4;           // of a row
    constexpr uint32_t kRowsAtOnce = 64 / kThreads; // of a wave
    constexpr uint32_t kAhead = 4;                  // pieces in flight
    __shared__ float lds_m[4][kRowsAtOnce], lds_l[4][kRowsAtOnce];
    __shared__ f32x4 lds_o[4][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t q = lane / kThreads, d = (lane % kThreads) * 4u, first = blockIdx.y * kRowsAtOnce, row = first + q;
    // every gridDim.x-th part is this workgroup's, at most 64 of them
    const uint32_t candidate = blockIdx.x + gridDim.x * lane;
    const uint32_t parts_of_it = candidate < sh.workers ? sh.cuts[candidate].more : 0u;
    // where no item has more pieces than a wave keeps in flight, each wave joins items of its own
    const bool alone = !__ballot(parts_of_it >= kAhead);
    const uint32_t apart = alone ? 1u : 4u;
    uint32_t count = 0;
    for (unsigned long long todo = __ballot(parts_of_it != 0u); todo; todo &= todo - 1ull, ++count) {
        if (alone && (count & 3u) != wave) continue;
        const uint32_t worker = blockIdx.x + gridDim.x * (uint32_t)__builtin_ctzll(todo);
        const Cut cut = sh.cuts[worker];
        if (cut.first_row + first >= cut.rows) continue;
        float m = kNone, sum = 0.0f;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        for (uint32_t i0 = alone ? 0u : wave; i0 <= cut.more; i0 += apart * kAhead) {
            float m1[kAhead], l1[kAhead];
            f32x4 o1[kAhead];
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u) {
                const uint32_t i = min_u32(i0 + apart * u, cut.more), slot = i == 0 ? 2u * worker + 1u : 2u * (worker + i);
                const int64_t at = (int64_t)slot * sh.rows + row;
                m1[u] = sh.sums[2 * at];
                l1[u] = sh.sums[2 * at + 1];
                o1[u] = *reinterpret_cast<const f32x4*>(sh.parts + at * DP + d);
            }
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u) {
                if (i0 + apart * u > cut.more) break;
                const float top = __builtin_fmaxf(m, m1[u]), zero = top == kNone ? 0.0f : top;
                const float f0 = __builtin_amdgcn_exp2f(m - zero), f1 = __builtin_amdgcn_exp2f(m1[u] - zero);
                sum = sum * f0 + l1[u] * f1;
                o = o * f0 + o1[u] * f1;
                m = top;
            }
        }
        if (!alone) {
            if (lane % kThreads == 0) {
                lds_m[wave][q] = m;
                lds_l[wave][q] = sum;
            }
            lds_o[wave][lane] = o;
            __syncthreads();
            float top = kNone;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __builtin_fmaxf(top, lds_m[k][q]);
            sum = 0.0f;
            o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = __builtin_amdgcn_exp2f(lds_m[k][q] - (top == kNone ? 0.0f : top));
                sum += lds_l[k][q] * f;
                o += lds_o[k][lane] * f;
            }
            __syncthreads();  // the next part's sums come here
        }
        if ((alone || wave == 0) && cut.first_row + row < cut.rows && (int32_t)d < args.cache.c.dim) {
            const uint32_t j = sh.group.div(cut.first_row + row), h = cut.head * sh.group.d + (cut.first_row + row - j * sh.group.d);
            uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.a.out) + (int64_t)(cut.first_col + j) * args.a.out_stride +
                                                       (int64_t)h * args.a.out_head_stride + d);
            const float inverse = 1.0f / sum;
            to[0] = sum == 0.0f ? 0u : pack_bf16(o[0] * inverse, o[1] * inverse);
            to[1] = sum == 0.0f ? 0u : pack_bf16(o[2] * inverse, o[3] * inverse);
        }
    }
}

// Places of a lane that are read, at most.
int64_t span_of(const AttendArgs& a) {
    return a.a.window ? std::min<int64_t>(a.places, (int64_t)a.a.window + a.a.C + 128) : a.places;
}

// Rows of an item: those of an average lane's columns and a key head's queries, rounded up.  Up to 32 the
// waves of a workgroup share the places, beyond that the rows (topk_attend_rows.hip).  Fewer rows than there are mean
// that keys and values are read again: 64 lanes over 6,144 places of 8 key heads of 128, e4m3 and bfloat16, 32 rows
// 216 and 348 us (in items of 16: 362 and 555), 64 rows 231 and 356 (of 32: 354 and 594), 128 rows 305 and 380 (of
// 64: 409 and 631), 256 rows 471 (of 128: 561).  Of dim 256 the registers hold 16 and 64 rows.
// Little work is done sooner in more and smaller items, whose parts take less time each and leave smaller pieces:
// 4 lanes of 256 rows over 300 places 17 us in items of 16, 20 of 32, 27 of 256; 8 lanes of 64 rows over 1,024 places 23,
// 25 and (of 64) 28; one lane of 256 rows over 2,048 places 21, 22 and 27, over 8,192 33, 30 and 36, over 32,768 82, 59
// and 58.  The limits are of the bytes that are then read (from cache, but for the first time).
uint32_t rows_of(const AttendArgs& a) {
    const int64_t rows = (a.a.C + a.a.lanes - 1) / a.a.lanes * (a.a.heads / a.cache.c.heads);
    const double once = 2.0 * (a.cache.c.format == TOPK_CACHE_FP8 ? 1 : 2) * a.cache.c.dim * a.cache.c.heads * (double)a.a.lanes * (double)span_of(a);
    if (rows <= 16 || once * (double)((rows + 15) / 16) <= 150e6) return 16;
    if (padded_dim(a) < 256 && (rows <= 32 || once * (double)((rows + 31) / 32) <= 300e6)) return 32;
    if (rows <= 64 || padded_dim(a) == 256) return 64;
    return rows <= 128 ? 128 : 256;
}

Shape shape_of(const AttendArgs& a, int64_t* bytes) {
    Shape s = {};
    const int dp = padded_dim(a);
    s.rows = rows_of(a);
    s.group = Divisor::of((uint32_t)(a.a.heads / a.cache.c.heads));
    const int64_t step = s.rows <= 32 ? kStep : kRowsStep;
    // at most so many parts as workgroups run at once (two on a compute unit, where 256 registers for each thread allow
    // it: with one, 64 lanes of 64 rows take 260 us instead of 208), and as there are steps
    const int64_t most = dp < 256 && s.rows < 256 ? 512 : 256;
    const int64_t items = a.cache.c.heads * ((a.a.C * s.group.d + a.a.lanes * (s.rows - 1)) / s.rows);
    const int64_t steps = std::min<int64_t>(most, (span_of(a) + step - 1) / step + 1);
    while ((int64_t)1 << s.shift < std::min(most, items * steps)) ++s.shift;
    s.workers = 1u << s.shift;
    const int64_t cuts = (sizeof(Cut) * s.workers + 255) / 256 * 256;
    const int64_t sums = (int64_t)2 * s.workers * s.rows * 2 * sizeof(float);
    const int64_t parts = (int64_t)2 * s.workers * s.rows * dp * sizeof(float);
    *bytes = cuts + sums + parts;
    uint8_t* p = static_cast<uint8_t*>(a.a.workspace);
    s.cuts = reinterpret_cast<Cut*>(p);
    s.sums = reinterpret_cast<float*>(p + cuts);
    s.parts = reinterpret_cast<float*>(p + cuts + sums);
    return s;
}

template <int DP, bool kWhole, bool kFp8, int kQueries>
void launch(const AttendArgs& a, const Shape& s, hipStream_t stream) {
    hipLaunchKernelGGL((attend_kernel<DP, kWhole, kFp8, kQueries>), dim3(s.workers), dim3(256), 0, stream, a, s);
}

template <int DP, bool kWhole, bool kFp8>
hipError_t launch_queries(const AttendArgs& a, hipStream_t stream) {
    int64_t bytes;
    const Shape s = shape_of(a, &bytes);
    if (s.rows == 16) launch<DP, kWhole, kFp8, 1>(a, s, stream);
    else if (s.rows > 32) launch_attend_rows(a, s, stream);
    if constexpr (DP < 256)
        if (s.rows == 32) launch<DP, kWhole, kFp8, 2>(a, s, stream);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL((join_kernel<DP>), dim3(std::min(s.workers, kJoinGroups), s.rows * DP / 256), dim3(256), 0, stream, a, s);
    return hipGetLastError();
}

template <int DP, bool kFp8>
hipError_t launch_whole(const AttendArgs& a, hipStream_t stream) {
    return a.cache.c.dim == DP ? launch_queries<DP, true, kFp8>(a, stream) : launch_queries<DP, false, kFp8>(a, stream);
}

template <bool kFp8>
hipError_t launch_dim(const AttendArgs& a, hipStream_t stream) {
    const int dp = padded_dim(a);
    if (dp == 64) return launch_whole<64, kFp8>(a, stream);
    if (dp == 128) return launch_whole<128, kFp8>(a, stream);
    return launch_whole<256, kFp8>(a, stream);
}

}  // namespace

int64_t attend_workspace(const AttendArgs& a) {
    int64_t bytes;
    shape_of(a, &bytes);
    return bytes;
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    return a.cache.c.format == TOPK_CACHE_FP8 ? launch_dim<true>(a, stream) : launch_dim<false>(a, stream);
}

}  // namespace topk
