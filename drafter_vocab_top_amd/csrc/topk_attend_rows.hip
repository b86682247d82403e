// Attention over the paged cache where a key head has many rows (see
// topk_attend.hip for the mathematics and how the work is cut).
//
// The waves of a workgroup share keys and values through LDS, 64 places at a
// time.  kGroups groups of 16 kQueries rows each have a wave, or two that take
// 32 of the places each and add up at the end (64 rows: four waves of 16 rows
// would read every operand from LDS for half as many products).  The next 64
// places are on their way to registers while these are worked on (an e4m3 cache
// is widened between registers and LDS, once for all rows).
//
// A batch's columns may be fewer than it has room for, which is what an item's size
// goes by.  A wave's rows are every kGroups-th 16 of an item, so that few rows are
// many waves' alike, and a wave leaves out what it has no rows for: 64 lanes of
// 32 rows in items of 256 take 267 us (442 with all products made), 16 lanes of
// 64 rows, bfloat16, 106 (137), full items of 128 rows 2 % longer.
//
// Without a mask all places up to the lane's last column are passed for each of
// its items, those behind an item's own columns among them: 8 prompts of 2,048
// columns with 32 query heads take 880 us, 0.62 PFLOP/s of the products made and
// half of that of the products needed.
//
// 64 lanes of 48 rows over 6,144 e4m3 places of 8 key heads of 128: 826 MB in 208
// us, 4.0 TB/s (a large copy makes 5.4).  16 lanes of 192 rows, bfloat16: 418 MB
// and 78 GFLOP in 139 us.  Neither memory nor the matrix cores (20 and 32 % of
// the time) bound it: a wave's products, weights and staging follow one another,
// and two waves on a SIMD overlap them in part.  Priorities for one of the two,
// and scores of the next places made among the weights of these (which takes
// all registers), did not help (153 and 164 us where it was 150).
//
// LDS holds rows of elements in chunks of 8, swapped so that 16 lanes that read a
// chunk of 16 keys, or four keys' 16 elements of a transposed read, meet 16 (8)
// different parts of the 64 banks, and 8 lanes that write every other chunk of a
// row (a widened vector gives two) 8 different ones of the 8 that 128 bytes are
// (without that 30 % of an e4m3 cache's LDS cycles were conflicts: 64 lanes of 64
// rows over 8192 places 231 and 221 us).  Values are read transposed: lane 16 g + r
// gets element r of places 4 g .. 4 g + 3.
#include <type_traits>

#include "topk_attend.hpp"

namespace topk {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int DP, bool kWhole, bool kFp8, int kQueries, int kGroups>
struct Rows {
    static constexpr int kSize = kFp8 ? 1 : 2;
    static constexpr uint32_t kStep = kRowsStep;
    static constexpr int kChunks = DP / 8;                       // 16-byte chunks of a row in LDS
    static constexpr int kVectors = DP * kSize / 16;             // 16-byte vectors of a row in memory
    static constexpr uint32_t kWaves = kGroups < 4 ? 4 : kGroups, kThreads = 64 * kWaves;
    static constexpr bool kAll = kStep * kVectors >= kThreads;   // (256 rows, dim 64, e4m3: half of the threads bring a step)
    static constexpr int kLoads = kAll ? kStep * kVectors / kThreads : 1;  // of keys (and of values) for each thread
    static constexpr int kKeySteps = DP / 32;
    static constexpr int kOut = DP / 16;
    static constexpr uint32_t kRows = 16 * kQueries * kGroups;
    static constexpr uint32_t kSplits = kWaves / kGroups;

    // Where chunk `c` of place `key` lies, in 16-byte units.
    __device__ __forceinline__ static uint32_t key_chunk(uint32_t key, uint32_t c) {
        return key * kChunks + (c ^ (c >> 3 & 1u) ^ (DP == 64 ? (key >> 1) & 7u : key & 15u));
    }
    __device__ __forceinline__ static uint32_t value_chunk(uint32_t key, uint32_t c) {
        return key * kChunks + (c ^ (c >> 3 & 1u) ^ (2u * (DP == 64 ? (key >> 1) & 3u : key & 7u)));
    }

    u32x4 k[kLoads], v[kLoads];  // on their way
    uint32_t key_scale, value_scale;  // of the lane's place, as binary32

    // Place base + lane of the step: block and slot in it.
    __device__ __forceinline__ static void lookup(const AttendArgs& a, const int32_t* table, uint32_t base, uint32_t end, uint32_t lane, uint32_t& id,
                                                  uint32_t& in_block) {
        const uint32_t p = min_u32(base + lane, end - 1u), b = a.cache.block.div(p);
        id = (uint32_t)table[b];  // (as it stands there: nothing waits for it before it is asked for)
        in_block = p - b * a.cache.block.d;
    }

    __device__ __forceinline__ static uint32_t valid(const AttendArgs& a, uint32_t id) {
        return (uint32_t)min_i32(max_i32((int32_t)id, 0), (int32_t)a.cache.c.blocks - 1);
    }

    __device__ __forceinline__ void load(const AttendArgs& a, const uint8_t* keys, const uint8_t* values, uint32_t head, uint32_t id,
                                         uint32_t in_block, uint32_t tid) {
        const topk_cache& c = a.cache.c;
        id = valid(a, id);
        const uint32_t at = a.cache.row16(id, in_block);
        if constexpr (kFp8) {
            const uint32_t s = a.cache.scale_row(id, in_block);
            const int64_t h = (int64_t)head * c.scale_head_stride;
            key_scale = (c.key_scales + h)[s];
            value_scale = (c.value_scales + h)[s];
        }
        if (!kAll && tid >= kStep * kVectors) return;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t x = (uint32_t)i * kThreads + tid, key = x / kVectors, part = x % kVectors;
            const uint32_t off = (uint32_t)from_lane((int32_t)at, key) + (kWhole || (int32_t)(part * 16u) < c.dim * kSize ? part : 0u);
            k[i] = *reinterpret_cast<const u32x4*>(past16(keys, off));
            v[i] = *reinterpret_cast<const u32x4*>(past16(values, off));
        }
    }

    // What has arrived goes to LDS; values past the end and keys' elements past the row as zeros.  With `masked` (some row
    // may not see some place) values that are not finite go there as zeros too: a weight of 0 would not remove
    // them.  They are added one by one (add_odd), where `odd` says that there are any: it gets `base`.
    __device__ __forceinline__ void store(const AttendArgs& a, u32x4* lds_k, u32x4* lds_v, uint32_t base, uint32_t end, bool masked, uint32_t* odd,
                                          uint32_t tid) const {
        if (masked) store_as<true>(a, lds_k, lds_v, base, end, odd, tid);  // (so is every step with places past the end)
        else store_as<false>(a, lds_k, lds_v, base, end, odd, tid);
    }

    template <bool kMasked>
    __device__ __forceinline__ void store_as(const AttendArgs& a, u32x4* lds_k, u32x4* lds_v, uint32_t base, uint32_t end, uint32_t* odd,
                                             uint32_t tid) const {
        if (!kAll && tid >= kStep * kVectors) return;
        uint32_t found = 0;
        const int32_t ks_bits = __builtin_bit_cast(int32_t, power_of(key_scale)), vs_bits = __builtin_bit_cast(int32_t, power_of(value_scale));
        constexpr uint32_t kApart = kThreads / kVectors;  // of a thread's places
        const uint32_t first = tid / kVectors, part = tid % kVectors;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t key = (uint32_t)i * kApart + first;
            // (places 16 apart have their chunks swapped alike)
            const uint32_t like = (uint32_t)i * kApart % 16u + first, whole = (uint32_t)i * kApart / 16u * 16u * kChunks;
            const bool in_row = kWhole || (int32_t)(part * 16u) < a.cache.c.dim * kSize;
            const u32x4 zero = {0u, 0u, 0u, 0u};
            if constexpr (kFp8) {
                const float ks = __builtin_bit_cast(float, from_lane(ks_bits, key)), vs = __builtin_bit_cast(float, from_lane(vs_bits, key));
                u32x4 y[2], z[2];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    y[h >> 1][2 * (h & 1)] = widen<false>(k[i][h], ks);
                    y[h >> 1][2 * (h & 1) + 1] = widen<true>(k[i][h], ks);
                    z[h >> 1][2 * (h & 1)] = widen<false>(v[i][h], vs);
                    z[h >> 1][2 * (h & 1) + 1] = widen<true>(v[i][h], vs);
                }
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    lds_k[key_chunk(like, 2u * part + h) + whole] = in_row ? y[h] : zero;
                    if constexpr (kMasked) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[h][e] = base + key < end ? only_finite(z[h][e], found) : 0u;
                    }
                    lds_v[value_chunk(like, 2u * part + h) + whole] = z[h];
                }
            } else {
                lds_k[key_chunk(like, part) + whole] = in_row ? k[i] : zero;
                u32x4 z = v[i];
                if constexpr (kMasked) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = base + key < end ? only_finite(z[e], found) : 0u;
                }
                lds_v[value_chunk(like, part) + whole] = z;
            }
        }
        if (found) *odd = base;
    }

    // Adds the values that are not finite of the 32 places from `base` on, each to the rows that see it.
    template <int N>
    __device__ __forceinline__ static void add_odd(const AttendArgs& a, const int32_t* table, const uint8_t* values, uint32_t head, uint32_t base,
                                                   uint32_t end, const uint32_t (&seen)[N], const bf16x8 (&weights)[N],
                                                   f32x4 (&o)[kQueries][kOut], uint32_t lane) {
        const topk_cache& c = a.cache.c;
        const uint32_t r = lane & 15u, g = lane >> 4;
        for (uint32_t key = 0; key < 32u && base + key < end; ++key) {
            uint32_t id, in_block;
            lookup(a, table, base + key, end, 0u, id, in_block);
            id = valid(a, id);
            const uint8_t* row = past16(values, a.cache.row16(id, in_block));
            float scale = 1.0f;
            if constexpr (kFp8)
                scale = power_of(c.value_scales[(int64_t)head * c.scale_head_stride + a.cache.scale_row(id, in_block)]);
            float weight[N];
#pragma unroll
            for (int n = 0; n < N; ++n) weight[n] = weight_of(weights[n], key, r);
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                const int32_t d = i * 16 + (int32_t)g * 4;
                const uint8_t* from = row + (kWhole || d < c.dim ? d * kSize : 0);
                u32x2 x;
                if constexpr (kFp8) {
                    const uint32_t y = *reinterpret_cast<const uint32_t*>(from);
                    x[0] = widen<false>(y, scale);
                    x[1] = widen<true>(y, scale);
                } else {
                    x = *reinterpret_cast<const u32x2*>(from);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v1 = __builtin_bit_cast(float, e & 1 ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16);
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        if ((seen[n] >> key & 1u) && !__builtin_isfinite(v1)) o[n][i][e] += weight[n] * v1;
                }
            }
        }
    }
};

template <int DP, bool kWhole, bool kFp8, int kQueries, int kGroups>
__global__ __launch_bounds__(64 * (kGroups < 4 ? 4 : kGroups), DP < 256 ? 2 : 1) void attend_rows_kernel(AttendArgs args, Shape sh) {
    using I = Rows<DP, kWhole, kFp8, kQueries, kGroups>;
    constexpr uint32_t R = I::kRows, kStep = kRowsStep, kSplits = I::kSplits;
    constexpr uint32_t kAhead = 4;             // operands of values read ahead
    constexpr uint32_t kTiles = 2u / kSplits;  // times 32 places of a wave
    static_assert(kSplits <= 2, "");
    __shared__ u32x4 lds_k[2][kStep * I::kChunks], lds_v[2][kStep * I::kChunks];
    __shared__ uint32_t lds_odd[2];
    __shared__ uint32_t lds_see[I::kWaves];
    if (threadIdx.x < 2u) lds_odd[threadIdx.x] = ~0u;
    __syncthreads();
    const topk_attend_args& a = args.a;
    const topk_cache& c = args.cache.c;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t split = wave % kSplits, group = wave / kSplits;  // its places, its rows: every kGroups-th 16
    // where this lane reads: chunk i of key r, and element 16 i of value 4 g + r / 4 (the other places lie whole rows further)
    uint32_t key_at[I::kKeySteps], value_at[I::kOut];
    {
        const uint32_t r = threadIdx.x & 15u, g = (threadIdx.x >> 4) & 3u;
#pragma unroll
        for (uint32_t i = 0; i < (uint32_t)I::kKeySteps; ++i) key_at[i] = I::key_chunk(r, i * 4u + g) * 16u;
#pragma unroll
        for (uint32_t i = 0; i < (uint32_t)I::kOut; ++i)
            value_at[i] = I::value_chunk(g * 4u + (r >> 2), 2u * i + ((r & 3u) >> 1)) * 16u + (r & 1u) * 8u;
    }
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
        const uint32_t rows = w.n * sh.group.d, wave_row = first_row + group * 16u;
        const uint8_t* keys = static_cast<const uint8_t*>(c.keys) + (int64_t)head * c.head_stride * I::kSize;
        const uint8_t* values = static_cast<const uint8_t*>(c.values) + (int64_t)head * c.head_stride * I::kSize;

        bf16x8 q[kQueries][I::kKeySteps];
        f32x4 o[kQueries][I::kOut];
        f32x4 sum[kQueries];
        float m[kQueries];
        uint32_t column[kQueries], low[kQueries], all_see = 0;
        {
            const uint32_t lane = opaque(threadIdx.x) & 63u, r = lane & 15u, g = lane >> 4;
#pragma unroll
            for (int n = 0; n < kQueries; ++n) {
                m[n] = kNone;
                sum[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < I::kOut; ++i) o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                // (a row past the last is the last again; it is not written)
                const uint32_t row = min_u32(wave_row + (uint32_t)n * 16u * kGroups + r, rows - 1u);
                const uint32_t j = sh.group.div(row), h = head * sh.group.d + (row - j * sh.group.d);
                column[n] = j;
                low[n] = first_seen(args, w, j);
                if (a.window) all_see = max_u32(all_see, max_of_16(low[n]));
                const uint16_t* from = static_cast<const uint16_t*>(a.q) + (int64_t)(w.cb + j) * a.q_stride + (int64_t)h * a.q_head_stride;
#pragma unroll
                for (int s = 0; s < I::kKeySteps; ++s) {
                    const int32_t d = s * 32 + (int32_t)g * 8;
                    u32x4 x = u32x4{0u, 0u, 0u, 0u};
                    if (kWhole || d < c.dim) x = *reinterpret_cast<const u32x4*>(from + d);
                    q[n][s] = __builtin_bit_cast(bf16x8, x);
                }
            }
            sign_queries(q, a.scale);
        }
        if (a.window) {  // all rows of the item see the places from here up to the lane's columns
            if (threadIdx.x % 64u == 0u) lds_see[wave] = all_see;
            __syncthreads();
#pragma unroll
            for (uint32_t i = 0; i < I::kWaves; ++i) all_see = max_u32(all_see, lds_see[i]);
            all_see = bcast(all_see, 0u);
        }
        auto masked_from = [&](uint32_t first, uint32_t places) { return uniform(first + places > w.open() || first < all_see); };

        uint32_t base = (w.first + step) * kStep;
        const uint32_t stop_at = min_u32((w.first + last_step) * kStep, w.end);
        // (which of this wave's 16 rows there are)
        const bool one = uniform(wave_row < rows), two = uniform(wave_row + 16u * kGroups < rows);
        I it;
        uint32_t id, in_block;
        {
            const uint32_t tid = opaque(threadIdx.x);
            I::lookup(args, table, base, w.end, tid & 63u, id, in_block);
            it.load(args, keys, values, head, id, in_block, tid);
            I::lookup(args, table, base + kStep, w.end, tid & 63u, id, in_block);
            it.store(args, lds_k[0], lds_v[0], base, w.end, masked_from(base, kStep), &lds_odd[0], tid);
            it.load(args, keys, values, head, id, in_block, tid);
            I::lookup(args, table, base + 2 * kStep, w.end, tid & 63u, id, in_block);
        }
        __syncthreads();
        for (uint32_t buffer = 0; base < stop_at; base += kStep, buffer ^= 1u) {
            const uint8_t* ks = reinterpret_cast<const uint8_t*>(lds_k[buffer]);
            const uint8_t* vs = reinterpret_cast<const uint8_t*>(lds_v[buffer]);
            const uint32_t lane = opaque(threadIdx.x & 63u), g = lane >> 4;
            const uint32_t b0 = base + split * 32u;                             // this wave's places: kTiles times 32
            // (of the whole step, as its values went to LDS: what was cleared there is added by the wave whose places it is of)
            const bool masked = masked_from(base, kStep);
            const uint32_t own = split * 32u * I::kChunks * 16u;
            auto work = [&](auto count) __attribute__((always_inline)) {
                constexpr int N = decltype(count)::value;  // of the wave's kQueries 16 rows
                // Operands are read ahead of their products (left to itself the compiler waits for each).
                f32x4 s[kTiles][N][2];
                bf16x8 x[2][I::kKeySteps];
                auto read_keys = [&](uint32_t t) __attribute__((always_inline)) {
#pragma unroll
                    for (uint32_t i = 0; i < (uint32_t)I::kKeySteps; ++i)
                        x[t & 1u][i] = *reinterpret_cast<const bf16x8*>(ks + key_at[i] + own + t * 16u * I::kChunks * 16u);
                };
                read_keys(0);
#pragma unroll
                for (uint32_t t = 0; t < 2u * kTiles; ++t) {
                    if (t + 1u < 2u * kTiles) read_keys(t + 1u);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int n = 0; n < N; ++n) s[t / 2][n][t & 1u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (uint32_t i = 0; i < (uint32_t)I::kKeySteps; ++i)
#pragma unroll
                        for (int n = 0; n < N; ++n)
                            s[t / 2][n][t & 1u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t & 1u][i], q[n][i], s[t / 2][n][t & 1u], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                // the first values are read while weights are made: tile i of the output for places 32 u .. 32 u + 31
                u32x4 y[kAhead];
                auto read_values = [&](uint32_t iu) __attribute__((always_inline)) {
                    const uint32_t i = iu / kTiles, u = iu % kTiles;
                    u32x4 z;
#pragma unroll
                    for (uint32_t t = 0; t < 2; ++t) {
                        const s16x4 z1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4*)(vs + value_at[i] + own + (u * 32u + t * 16u) * I::kChunks * 16u));
                        const u32x2 z2 = __builtin_bit_cast(u32x2, z1);
                        z[2 * t] = z2[0];
                        z[2 * t + 1] = z2[1];
                    }
                    return z;
                };
#pragma unroll
                for (uint32_t i = 0; i < kAhead; ++i) y[i] = read_values(i);
                uint32_t seen[kTiles][N] = {};
                bf16x8 weights[kTiles][N];
                if (masked) {
#pragma unroll
                    for (uint32_t u = 0; u < kTiles; ++u)
#pragma unroll
                        for (int n = 0; n < N; ++n) seen[u][n] = seen_bits(args, w, column[n], low[n], b0 + u * 32u);
                }
                weigh(s, masked, seen, factor, g, m, sum, o, weights);
#pragma unroll
                for (uint32_t iu = 0; iu < I::kOut * kTiles; ++iu) {
                    const uint32_t i = iu / kTiles, u = iu % kTiles;
                    const bf16x8 v1 = __builtin_bit_cast(bf16x8, y[iu % kAhead]);
                    if (iu + kAhead < I::kOut * kTiles) y[iu % kAhead] = read_values(iu + kAhead);
#pragma unroll
                    for (int n = 0; n < N; ++n) o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, weights[u][n], o[n][i], 0, 0, 0);
                }
                if (masked && uniform(lds_odd[buffer] == base)) {
#pragma unroll
                    for (uint32_t u = 0; u < kTiles; ++u) I::add_odd(args, table, values, head, b0 + u * 32u, w.end, seen[u], weights[u], o, lane);
                }
            };
            if (kQueries == 2 && two) work(std::integral_constant<int, kQueries>());
            else if (one) work(std::integral_constant<int, 1>());
            __builtin_amdgcn_sched_barrier(0);
            it.store(args, lds_k[buffer ^ 1u], lds_v[buffer ^ 1u], base + kStep, w.end, masked_from(base + kStep, kStep), &lds_odd[buffer ^ 1u],
                     threadIdx.x);
            {
                // the places behind them (past the end: the last one again)
                const uint32_t tid = opaque(threadIdx.x);
                it.load(args, keys, values, head, id, in_block, tid);
                I::lookup(args, table, base + 3 * kStep, w.end, tid & 63u, id, in_block);
            }
            __syncthreads();
        }

        const bool direct = step == 0 && last_step == w.steps;
        const uint32_t slot = 2u * worker + (step == 0 ? 1u : 0u);
        const uint32_t lane = opaque(threadIdx.x) & 63u, r = lane & 15u, g = lane >> 4;
        if constexpr (kSplits == 2) {
            // the second half of the places joins the first, through the keys' LDS (all have left the loop)
            static_assert(sizeof(lds_k) >= kQueries * 64 * (I::kOut * 16 + 8), "");
            f32x4* to = reinterpret_cast<f32x4*>(group == 0 ? lds_k : lds_v);
            float* ml = reinterpret_cast<float*>(to + kQueries * I::kOut * 64);
            if (split == 1) {
#pragma unroll
                for (int n = 0; n < kQueries; ++n) {
#pragma unroll
                    for (int i = 0; i < I::kOut; ++i) to[(n * I::kOut + i) * 64 + (int)lane] = o[n][i];
                    ml[(2 * n) * 64 + (int)lane] = m[n];
                    ml[(2 * n + 1) * 64 + (int)lane] = sum[n][0];
                }
            }
            __syncthreads();
            if (split == 0) {
#pragma unroll
                for (int n = 0; n < kQueries; ++n) {
                    const float other = ml[(2 * n) * 64 + (int)lane], top = __builtin_fmaxf(m[n], other), zero = top == kNone ? 0.0f : top;
                    const float f0 = __builtin_amdgcn_exp2f(m[n] - zero), f1 = __builtin_amdgcn_exp2f(other - zero);
                    m[n] = top;
                    sum[n][0] = sum[n][0] * f0 + ml[(2 * n + 1) * 64 + (int)lane] * f1;
#pragma unroll
                    for (int i = 0; i < I::kOut; ++i) o[n][i] = o[n][i] * f0 + to[(n * I::kOut + i) * 64 + (int)lane] * f1;
                }
            }
            __syncthreads();  // the next item's keys come here
        }
#pragma unroll
        for (int n = 0; n < kQueries; ++n) {
            if (split != 0) break;
            const float all = sum[n][0];
            const uint32_t row = group * 16u + (uint32_t)n * 16u * kGroups + r;
            if (!direct && first_row + row < rows) {
                float* to = sh.parts + ((int64_t)slot * R + row) * DP + g * 4u;
#pragma unroll
                for (int i = 0; i < I::kOut; ++i) *reinterpret_cast<f32x4*>(to + i * 16) = o[n][i];
                if (g == 0) {
                    sh.sums[((int64_t)slot * R + row) * 2] = m[n];
                    sh.sums[((int64_t)slot * R + row) * 2 + 1] = all;
                }
            } else if (direct && first_row + row < rows) {
                const uint32_t j = sh.group.div(first_row + row), h = head * sh.group.d + (first_row + row - j * sh.group.d);
                uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (int64_t)(w.cb + j) * a.out_stride +
                                                           (int64_t)h * a.out_head_stride + g * 4u);
                const float inverse = 1.0f / all;
#pragma unroll
                for (int i = 0; i < I::kOut; ++i) {
                    u32x2 y;
                    y[0] = all == 0.0f ? 0u : pack_bf16(o[n][i][0] * inverse, o[n][i][1] * inverse);
                    y[1] = all == 0.0f ? 0u : pack_bf16(o[n][i][2] * inverse, o[n][i][3] * inverse);
                    if (kWhole || i * 16 < c.dim) *reinterpret_cast<u32x2*>(to + i * 8) = y;
                }
            }
        }
        at += last_step - step;
        if (at == stop && step == 0 && last_step < w.steps) {
            more = (uint32_t)(((uint64_t)(w.steps - last_step) + per - 1u) / per);
            if (threadIdx.x == 0) sh.cuts[worker] = Cut{more, first_row, rows, w.cb, head, {}};
        }
    }
    if (more == 0 && threadIdx.x == 0) sh.cuts[worker].more = 0;
}

template <int DP, bool kWhole, bool kFp8>
void launch_rows(const AttendArgs& a, const Shape& s, hipStream_t stream) {
    const dim3 grid(s.workers), block(s.rows == 256 ? 512 : 256);
    if constexpr (DP == 256) {
        hipLaunchKernelGGL((attend_rows_kernel<DP, kWhole, kFp8, 1, 4>), grid, block, 0, stream, a, s);
    } else {
        if (s.rows == 64) hipLaunchKernelGGL((attend_rows_kernel<DP, kWhole, kFp8, 2, 2>), grid, block, 0, stream, a, s);
        else if (s.rows == 128) hipLaunchKernelGGL((attend_rows_kernel<DP, kWhole, kFp8, 2, 4>), grid, block, 0, stream, a, s);
        else hipLaunchKernelGGL((attend_rows_kernel<DP, kWhole, kFp8, 2, 8>), grid, block, 0, stream, a, s);
    }
}

template <int DP>
void launch_format(const AttendArgs& a, const Shape& s, hipStream_t stream) {
    const bool whole = a.cache.c.dim == DP;
    if (a.cache.c.format == TOPK_CACHE_FP8) whole ? launch_rows<DP, true, true>(a, s, stream) : launch_rows<DP, false, true>(a, s, stream);
    else whole ? launch_rows<DP, true, false>(a, s, stream) : launch_rows<DP, false, false>(a, s, stream);
}

}  // namespace

void launch_attend_rows(const AttendArgs& a, const Shape& s, hipStream_t stream) {
    const int dp = padded_dim(a);
    if (dp == 64) launch_format<64>(a, s, stream);
    else if (dp == 128) launch_format<128>(a, s, stream);
    else launch_format<256>(a, s, stream);
}

}  // namespace topk
