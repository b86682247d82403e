// Penalties, biases and masks on logits, for gfx950.
//
// For row r of column c (column j of lane l), with n the token's count in the
// lane's output and its first j drafts:
//   seen (in the prompt, or n > 0):  x = x > 0 ? x / rep : x * rep
//   n > 0:                           x = x - (freq * n + pres)
//   biased:                          x = x + bias
//   forbidden by the mask:           x = -Inf
//
// Column-contiguous: one kernel.  A workgroup takes a couple of thousand rows
// of some of a lane's columns.  It streams them (in place: only what the mask
// forbids), finds the rows that a penalty or bias touches from one bit per row
// of the history, and rewrites those in every column from the original.
//
// Row-interleaved: a part that streams the matrix (out of place it copies the
// elements; it writes -Inf where the mask forbids them) and one that rewrites
// the elements that a penalty or a bias touches: a few thousand of a column's
// 248,046 rows.  It reads the originals and leaves forbidden elements alone.
// Out of place it is a second launch.  In place the two write different
// elements and are one launch: one lane's 8 columns 8.2 us, in two 12.7; 448
// columns, of whose elements 5 % are forbidden, 57 and 76.  (Forbidden elements
// are then written alone, not with the vector around them: the same time but
// where half of 448 columns' are forbidden, 134 and 132.)
//
// Reading every count would add 4 bytes per row and lane to the 2 to 8 that an
// element costs; the bits add an eighth of a byte, and a list of the touched
// rows keeps the arithmetic (some 40 instructions an element) off the lanes
// that have none: element by element in the streaming threads it took 16 us
// where the list takes 7 (56 columns in place).
//
// What bounds it (one MI355X, replayed from a graph).  Large matrices: memory.
// 448 interleaved columns of 248,046 rows, bf16: 82 us for the dense part (461
// MB, 5.6 TB/s, the rate of a plain copy) and 19 for the touched rows; 448
// column-contiguous ones 91.  64 columns of 131,072 rows, fp32, half of them in
// use: 11.2 us (34 MB).  Small ones: the chain launch, col_start and history
// bits, list, counts and elements, store: 6.7 us for one lane's 8 columns (8
// MB), 7.7 for 56 in place (scattered elements), 12 with masks (14 MB of -Inf).
//
// The penalised value is a chain of four operations.  Each is carried out in
// binary64, and the last result is rounded to binary32 and then to the type:
// what is left where a penalty nearly cancels a logit is right, and touched
// elements are too rare for it to cost time.
#include "topk_round.hpp"

#include "topk_col_common.hpp"

namespace topk {

namespace {

template <class DT>
__device__ __forceinline__ float to_float(uint32_t raw) {
    return __builtin_bit_cast(float, DT::kPerVec == 8 ? raw << 16 : raw);
}

// To nearest, ties to even; NaN stays NaN.
template <class DT>
__device__ __forceinline__ uint32_t from_double(double y) {
    const float f = (float)y;
    const uint32_t b = __builtin_bit_cast(uint32_t, f);
    if constexpr (DT::kPerVec == 8) {
        if (f != f) return (b >> 16) | 0x40u;
        return (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
    } else {
        return b;
    }
}

template <class DT>
constexpr uint32_t kMinusInf = DT::kPerVec == 8 ? 0xFF80u : 0xFF800000u;

// The operations as they are written, each rounded (no fused ones).
struct LaneRules {
    double rep, inv, pres, freq;
    __device__ LaneRules(float r, float p, float f) : rep((double)r), inv(1.0 / rep), pres((double)p), freq((double)f) {}
    // x / rep, rounded to nearest, of binary32 values.  q is off by at most two of
    // its last places, so x - q rep takes some 26 bits and is exact; adding its
    // quotient, off by less than 2^-51 of a last place, rounds as x / rep does,
    // which with operands of 24 bits is no nearer than 2^-25 of a last place to
    // where the rounding changes.  Where an operand is infinite or zero, q is the
    // quotient.  Eight lanes in place 7.70 us, with a division 7.83, with q alone
    // 7.60; one lane with every row in its history 8.85, 9.42 and 8.48.
    __device__ __forceinline__ double quotient(double x) const {
        const double q = x * inv, rest = __builtin_fma(-q, rep, x);
        return __builtin_isfinite(rest) ? __builtin_fma(rest, inv, q) : q;
    }
    // what n occurrences take off
    __device__ __forceinline__ double penalty(uint32_t n) const {
#pragma clang fp contract(off)
        return n ? freq * (double)n + pres : 0.0;
    }
    __device__ __forceinline__ double apply(double x, bool seen, double penalty, bool biased, double bias) const {
#pragma clang fp contract(off)
        const double y = (seen ? x > 0.0 ? quotient(x) : x * rep : x) - penalty;
        return biased ? y + bias : y;
    }
};

// The mask row of a column, or NULL if it has none.
__device__ __forceinline__ const uint32_t* mask_row(const AdjustArgs& a, uint32_t c) {
    if (!a.mask) return nullptr;
    const int64_t m = a.mask_index ? (int64_t)a.mask_index[c] : (int64_t)c;
    return m >= 0 && m < a.mask_count ? a.mask + m * a.mask_ld : nullptr;
}

// 16 bytes at element alignment (global memory takes any).  kOnce: past the
// caches, for matrices that they could not hold until they are read again.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
template <bool kOnce, class T>
__device__ __forceinline__ u32x4 load16(const T* p) {
    if constexpr (kOnce) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    else return *reinterpret_cast<const u32x4_any*>(p);
}
template <bool kOnce, class T>
__device__ __forceinline__ void store16(T* p, const u32x4& v) {
    if constexpr (kOnce) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
    else *reinterpret_cast<u32x4_any*>(p) = v;
}

// v with the elements whose bit in `allowed` is clear set to -Inf.
template <class DT>
__device__ __forceinline__ u32x4 masked(const u32x4& v, uint32_t allowed) {
    u32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w = q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
        if constexpr (DT::kPerVec == 8) {
            if (!(allowed >> (2 * q) & 1u)) w = (w & 0xFFFF0000u) | kMinusInf<DT>;
            if (!(allowed >> (2 * q + 1) & 1u)) w = (w & 0xFFFFu) | (kMinusInf<DT> << 16);
        } else {
            if (!(allowed >> q & 1u)) w = kMinusInf<DT>;
        }
        if (q == 0) r.x = w;
        else if (q == 1) r.y = w;
        else if (q == 2) r.z = w;
        else r.w = w;
    }
    return r;
}

// ------------------------------------------------------------ touched rows ---

// The ROWS rows of a workgroup: runs of RUN that lie `tiles` runs apart.  The
// ids of a vocabulary sorted by use put most of a history into the first rows;
// in one contiguous tile they hold up a launch that has little else to do.
// Runs of 256 rows are the most that a workgroup rewrites in one go, and whole
// cache lines; a launch that streams much reads one tile in a piece.
template <uint32_t kRows, uint32_t kRun>
struct Rows {
    static constexpr uint32_t RUN = kRun, ROWS = kRows, WORDS = ROWS / 32;
    static_assert(WORDS <= (uint32_t)kBlock, "one word of the rows' bits per thread");
    uint32_t tiles, tile;
    __device__ __forceinline__ uint32_t row(uint32_t at) const { return (at / RUN * tiles + tile) * RUN + at % RUN; }
    // the place of row r, or ROWS if it is another workgroup's
    __device__ __forceinline__ uint32_t place(uint32_t r, uint32_t V) const {
        const uint32_t run = r / RUN, i = run / tiles;
        return r < V && run - i * tiles == tile ? i * RUN + r % RUN : ROWS;
    }
};

template <uint32_t kRows, bool kBias>
struct TouchedRows {
    alignas(16) uint32_t bias_at[kBias ? kRows : 4];  // 1 + the last list entry of a place, or 0
    uint32_t touched[kRows / 32];  // places with a history, a draft or a bias
    uint32_t drafted[kRows / 32];  // places that are drafts
    uint16_t list[kRows];          // the touched places, in any order
    uint32_t n;
};

__device__ __forceinline__ uint32_t scalar(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// What hangs on the lane alone, read at once.
template <class R, bool kBias>
struct Lane {
    uint32_t cb, ce, db, de, bb, be;  // its columns, the drafts before its last column, its biases
    float rep, pres, freq;
    uint32_t word;                    // the history's bits of this thread's 32 places
    __device__ __forceinline__ Lane(const AdjustArgs& a, const R& rows, uint32_t l) {
        const uint32_t tid = threadIdx.x;
        const int32_t* cs = a.cols.at(l);
        const int32_t* ds = a.draft_parts.at(l);
        const int32_t* bs = a.bias_parts.at(l);
        const uint32_t r = rows.row(min_u32(tid, R::WORDS - 1u) * 32u);
        const uint32_t* sp = a.seen ? a.seen + (int64_t)l * a.seen_ld + (min_u32(r, a.V - 1u) >> 5) : safe<uint32_t>();
        const int32_t c0 = cs[0], c1 = cs[1], d0 = ds[0], d1 = ds[1], b0 = bs[0], b1 = bs[1];
        rep = *(a.repetition ? a.repetition + l : safe<float>());
        pres = *(a.presence ? a.presence + l : safe<float>());
        freq = *(a.frequency ? a.frequency + l : safe<float>());
        word = *sp;
        a.cols.cut(l, c0, c1, cb, ce);
        a.draft_parts.cut(l, d0, d1, db, de);
        a.bias_parts.cut(l, b0, b1, bb, be);
        if (!a.drafts) de = db;
        if (ce > cb) de = min_u32(de, db + (ce - cb - 1u));
        // (equal in all threads, which the compiler cannot know of such reads)
        cb = scalar(cb), ce = scalar(ce), db = scalar(db), de = scalar(de), bb = scalar(bb), be = scalar(be);
        if (!a.repetition) rep = 1.0f;
        if (!a.presence) pres = 0.0f;
        if (!a.frequency) freq = 0.0f;
        if (tid >= R::WORDS || r >= a.V || !a.seen) word = 0;
        else if (a.V - r < 32u) word &= (1u << (a.V - r)) - 1u;  // bits past the last row mean nothing
    }
};

// Fills sh (list and n are valid after the next barrier) with the touched places
// of the words that are `part` modulo parts (a power of two).  bias0, draft0:
// the lane's entries bb + thread and db + thread.
template <class R, bool kBias>
__device__ __forceinline__ void make_list(const AdjustArgs& a, const R& rows, const Lane<R, kBias>& lane, uint32_t draft0,
                                          uint32_t bias0, TouchedRows<R::ROWS, kBias>& sh, uint32_t part = 0, uint32_t parts = 1) {
    constexpr uint32_t kRows = R::ROWS;
    const uint32_t tid = threadIdx.x, ln = tid & 63u;
    if (tid == 0) sh.n = 0;
    if (tid < kRows / 32) {
        sh.touched[tid] = (tid & (parts - 1u)) == part ? lane.word : 0u;
        sh.drafted[tid] = 0;
    }
    if constexpr (kBias)
        for (uint32_t i = tid; i < kRows / 4; i += kBlock) reinterpret_cast<u32x4*>(sh.bias_at)[i] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    if (a.drafts || kBias) {
        for (uint32_t i = lane.db + tid; i < lane.de; i += kBlock) {
            const uint32_t at = rows.place(i == lane.db + tid ? draft0 : (uint32_t)a.drafts[i], a.V);
            if (at == kRows || (at >> 5 & (parts - 1u)) != part) continue;
            atomicOr(&sh.touched[at >> 5], 1u << (at & 31u));
            atomicOr(&sh.drafted[at >> 5], 1u << (at & 31u));
        }
        if constexpr (kBias) {
            for (uint32_t i = lane.bb + tid; i < lane.be; i += kBlock) {
                const uint32_t at = rows.place(i == lane.bb + tid ? bias0 : (uint32_t)a.bias_ids[i], a.V);
                if (at == kRows || (at >> 5 & (parts - 1u)) != part) continue;
                atomicOr(&sh.touched[at >> 5], 1u << (at & 31u));
                atomicMax(&sh.bias_at[at], i - lane.bb + 1u);
            }
        }
        __syncthreads();
    }
    // a ballot per 64 places, one LDS atomic per wave
    constexpr uint32_t Q = kRows / kBlock;
    unsigned long long some[Q];
    uint32_t total = 0;
#pragma unroll
    for (uint32_t q = 0; q < Q; ++q) {
        some[q] = __ballot(sh.touched[q * (kBlock / 32u) + (tid >> 5)] >> (tid & 31u) & 1u);
        total += (uint32_t)__popcll(some[q]);
    }
    if (total == 0) return;
    uint32_t pos = 0;
    if (ln == 0) pos = atomicAdd(&sh.n, total);
    pos = (uint32_t)__builtin_amdgcn_readfirstlane((int)pos);
#pragma unroll
    for (uint32_t q = 0; q < Q; ++q) {
        if (some[q] >> ln & 1ull) sh.list[pos + lanes_below(some[q])] = (uint16_t)(q * kBlock + tid);
        pos += (uint32_t)__popcll(some[q]);
    }
}

template <class R, bool kBias>
__device__ __forceinline__ void first_entries(const AdjustArgs& a, const Lane<R, kBias>& lane, uint32_t& draft0, uint32_t& bias0) {
    const uint32_t tid = threadIdx.x;
    bias0 = kBias ? (uint32_t)a.bias_ids[min_u32(lane.bb + tid, a.bias_parts.total - 1u)] : 0u;
    draft0 = a.drafts ? (uint32_t)a.drafts[min_u32(lane.db + tid, a.draft_parts.total - 1u)] : 0u;
}

// Which of a lane's drafts are one row (of a row known to be a draft).
struct DraftsOfRow {
    uint64_t first = 0;  // bit i: draft i of the first 64
    template <class L>
    __device__ __forceinline__ void find(const AdjustArgs& a, const L& lane, uint32_t row) {
#pragma unroll 8
        for (uint32_t i = 0; i < min_u32(lane.de - lane.db, 64u); ++i)
            first |= (uint32_t)a.drafts[lane.db + i] == row ? 1ull << i : 0ull;
    }
    // among the first j
    template <class L>
    __device__ __forceinline__ uint32_t before(const AdjustArgs& a, const L& lane, uint32_t row, uint32_t j) const {
        uint32_t n = (uint32_t)__popcll(j < 64u ? first & ((1ull << j) - 1u) : first);
        for (uint32_t i = lane.db + 64u; i < min_u32(lane.de, lane.db + j); ++i) n += (uint32_t)a.drafts[i] == row ? 1u : 0u;
        return n;
    }
};

// ------------------------------------------------------ column-contiguous ---

// What becomes of the matrix: changed in place; copied, the rows in short runs;
// copied a tile in a piece; the same past the caches.
enum { kModeInPlace, kModeShort, kModeLong, kModeOnce };

// Lane l0 + blockIdx.y, its columns blockIdx.z * U, .. + U - 1, then
// gridDim.z * U further on.  The columns share the search for the rows that a
// penalty or bias touches and the reading of their counts.
//
// At these sizes the time is that of the chain of dependent reads: reads of
// one link are issued together, at addresses cut to the last valid one instead
// of behind branches.
template <class DT, int kMode, uint32_t U, bool kBias, bool kMask>
__global__ __launch_bounds__(kBlock) void adjust_col(AdjustArgs a, uint32_t l0) {
    using storage = typename DT::storage;
    constexpr uint32_t EPV = DT::kPerVec, ALL = (1u << EPV) - 1u, ROWS = kBlock * EPV;
    constexpr bool kInPlace = kMode == kModeInPlace, kOnce = kMode == kModeOnce;
    using R = Rows<ROWS, kMode == kModeInPlace || kMode == kModeShort ? 256 : ROWS>;
    __shared__ TouchedRows<ROWS, kBias> sh;
    const uint32_t l = l0 + blockIdx.y, tid = threadIdx.x, V = a.V;
    const R rows{gridDim.x, blockIdx.x};
    const bool sparse = a.counts || a.drafts || kBias;
    const Lane<R, kBias> lane(a, rows, l);
    const uint32_t cb = lane.cb, ce = lane.ce;
    const uint32_t c_first = cb + blockIdx.z * U, c_step = gridDim.z * U;
    if (c_first >= ce) return;
    uint32_t draft0, bias0;
    first_entries(a, lane, draft0, bias0);

    // The streamed part copies (out of place) and masks.
    const uint32_t r = rows.row(tid * EPV);          // this thread's rows
    const uint32_t nvec = V / EPV;                   // whole vectors of a column
    const bool whole = r / EPV < nvec;
    // the vector read: the column's last whole one for the rows behind it
    const uint32_t rr = whole ? r : nvec ? V - EPV : 0u;
    u32x4 d[U];
    uint32_t m[U];
    auto load_columns = [&](uint32_t c0) {
        uint32_t none[U];
        const uint8_t* mp[U];
        if constexpr (kMask) {
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                const uint32_t c = min_u32(c0 + u, ce - 1u);
                const int64_t mi = a.mask_index ? (int64_t)a.mask_index[c] : (int64_t)c;
                const bool has = mi >= 0 && mi < a.mask_count;
                none[u] = has ? 0u : ALL;
                mp[u] = reinterpret_cast<const uint8_t*>(a.mask + (has ? mi * a.mask_ld : 0));
            }
        }
        if (nvec) {
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                if (!kInPlace) d[u] = load16<kOnce>(static_cast<const storage*>(a.x) + (int64_t)min_u32(c0 + u, ce - 1u) * a.ld + rr);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) m[u] = kMask ? (uint32_t)mp[u][min_u32(r, V - 1u) >> 3] : ALL;
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
            if (kMask) m[u] = (m[u] >> (r & 7u) & ALL) | none[u];
    };
    auto store_columns = [&](uint32_t c0) {
        if (kInPlace && whole) {
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                if (c0 + u < ce && m[u] != ALL && m[u]) d[u] = load16<false>(static_cast<const storage*>(a.x) + (int64_t)(c0 + u) * a.ld + r);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (c0 + u >= ce || r >= V || (kInPlace && m[u] == ALL)) continue;
            const storage* x = static_cast<const storage*>(a.x) + (int64_t)(c0 + u) * a.ld;
            storage* out = static_cast<storage*>(a.out) + (int64_t)(c0 + u) * a.out_ld;
            if (whole) {
                store16<kOnce>(out + r, kMask ? masked<DT>(d[u], m[u]) : d[u]);
            } else if (nvec) {
                const uint32_t skip = EPV - (V - r);  // elements of the vector read that other threads write
#pragma unroll
                for (uint32_t e = 0; e < EPV; ++e) {
                    const bool ok = m[u] << skip >> e & 1u;
                    if (e >= skip && (!kInPlace || !ok)) out[rr + e] = !kInPlace && ok ? (storage)vec_elem<DT>(d[u], (int)e) : (storage)kMinusInf<DT>;
                }
            } else {
                for (uint32_t e = 0; r + e < V; ++e) {
                    const bool ok = m[u] >> e & 1u;
                    if (!kInPlace || !ok) out[r + e] = ok ? x[r + e] : (storage)kMinusInf<DT>;
                }
            }
        }
    };
    constexpr bool stream = !kInPlace || kMask;
    if constexpr (stream) load_columns(c_first);

    if (sparse) make_list(a, rows, lane, draft0, bias0, sh);
    if constexpr (stream) {
        store_columns(c_first);
        for (uint32_t c0 = c_first + c_step; c0 < ce; c0 += c_step) {
            load_columns(c0);
            store_columns(c0);
        }
    }
    if (!sparse) return;
    // For the list, and for the streamed stores, which those below replace.
    // (Reading the first rows' elements before the streamed stores took longer:
    // 12.1 to 14.2 us with masks, 7.4 to 7.9 in place.)
    __syncthreads();

    const LaneRules rules(lane.rep, lane.pres, lane.freq);
    const uint32_t n_rows = sh.n;
    const int32_t* counts = a.counts ? a.counts + (int64_t)l * a.counts_ld : nullptr;
    for (uint32_t k = tid; k < n_rows; k += kBlock) {
        const uint32_t at = sh.list[k], row = rows.row(at);
        uint32_t counted = (uint32_t)*(counts ? counts + row : safe<int32_t>());
        const uint32_t b = kBias ? sh.bias_at[kBias ? at : 0] : 0u;
        const float bias_value = kBias ? a.bias_values[b ? lane.bb + b - 1u : 0u] : 0.0f;
        DraftsOfRow drafts;
        bool drafted = false, seen = false;
        uint32_t times = 0;
        double penalty = 0.0;
        for (uint32_t c0 = c_first; c0 < ce; c0 += c_step) {
            uint32_t raw[U], ok[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                raw[u] = (uint32_t)(static_cast<const storage*>(a.x) + (int64_t)min_u32(c0 + u, ce - 1u) * a.ld)[row];
            if constexpr (kMask) {
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) {
                    const uint32_t c = min_u32(c0 + u, ce - 1u);
                    const int64_t mi = a.mask_index ? (int64_t)a.mask_index[c] : (int64_t)c;
                    const bool has = mi >= 0 && mi < a.mask_count;
                    ok[u] = a.mask[(has ? mi * a.mask_ld : 0) + (row >> 5)] >> (row & 31u) | (has ? 0u : 1u);
                }
            }
            if (c0 == c_first) {
                if (!counts) counted = 0;
                times = counted & 0x7FFFFFFFu;
                penalty = rules.penalty(times);
                seen = counted != 0;
                drafted = a.drafts && (sh.drafted[at >> 5] >> (at & 31u) & 1u);
                if (drafted) drafts.find(a, lane, row);
            }
            uint32_t y[U];
            bool write[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                bool seen_u = seen;
                double penalty_u = penalty;
                if (drafted) {
                    const uint32_t n = times + drafts.before(a, lane, row, c0 + u - cb);
                    seen_u = seen || n;
                    penalty_u = rules.penalty(n);
                }
                // (a forbidden element stays -Inf, a later column's draft changes nothing here)
                write[u] = c0 + u < ce && (!kMask || (ok[u] & 1u)) && (seen_u || b);
                y[u] = from_double<DT>(rules.apply((double)to_float<DT>(raw[u]), seen_u, penalty_u, b != 0, (double)bias_value));
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                if (write[u]) (static_cast<storage*>(a.out) + (int64_t)(c0 + u) * a.out_ld)[row] = (storage)y[u];
        }
    }
}

// -------------------------------------------------------- row-interleaved ---

constexpr uint32_t kRowTileVecs = 64;  // at most 64 vectors of a row per workgroup

// A workgroup takes 1 << tx_log vectors of a row; each thread one of them over U
// rows, which one word of each column's mask covers, all in flight together.
// In place only forbidden elements are written, so that others may rewrite the
// allowed ones meanwhile.
template <class DT, int kMode, bool kMask, uint32_t U>
__device__ __forceinline__ void row_dense(const AdjustArgs& a, uint32_t tx_log, uint32_t row_tile, uint32_t column_tile,
                                          uint8_t* active) {
    using storage = typename DT::storage;
    constexpr uint32_t EPV = DT::kPerVec, ALL = (1u << EPV) - 1u;
    constexpr bool kInPlace = kMode == kModeInPlace, kOnce = kMode == kModeOnce;
    const uint32_t tid = threadIdx.x, V = a.V;
    const uint32_t tile_c = (column_tile << tx_log) * EPV, tile_n = EPV << tx_log;
    const uint32_t vc = tid & ((1u << tx_log) - 1u);
    // The row's last vector, if it is not whole, moves up: what it shares with
    // the one before it both write alike.
    uint32_t c = tile_c + vc * EPV;
    if (c < a.C && c + EPV > a.C && a.C >= tile_c + EPV) c = a.C - EPV;
    const uint32_t r0 = row_tile * (kBlock >> tx_log) * U + (tid >> tx_log) * U;
    uint32_t words[EPV];
    if constexpr (kMask) {
        int64_t mi[EPV];
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) {
            const uint32_t ce = min_u32(c + e, a.C - 1u);
            mi[e] = a.mask_index ? (int64_t)a.mask_index[ce] : (int64_t)ce;
        }
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) {
            const bool has = mi[e] >= 0 && mi[e] < a.mask_count;
            words[e] = a.mask[(has ? mi[e] * a.mask_ld : 0) + (min_u32(r0, V - 1u) >> 5)];
            mi[e] = has ? 0 : -1;
        }
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) words[e] = (words[e] >> (r0 & 31u)) | (uint32_t)mi[e];
    }
    uint32_t mine = c + EPV <= a.C ? ALL : c < a.C ? (1u << (a.C - c)) - 1u : 0u;  // bit e: column c + e is a lane's
    if (a.cols.start) {
        for (uint32_t i = tid; i < tile_n; i += kBlock) active[i] = 0;
        __syncthreads();
        for (uint32_t l = tid; l < a.lanes; l += kBlock) {
            uint32_t b, e;
            a.cols.range(l, b, e);
            e = min_u32(e, tile_c + tile_n);
            for (uint32_t k = b < tile_c ? tile_c : b; k < e; ++k) active[k - tile_c] = 1;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) mine &= c < a.C && active[c - tile_c + e] ? ~0u : ~(1u << e);
    }
    if (mine == 0 || r0 >= V) return;
    const uint32_t n = min_u32(U, V - r0);
    const storage* x = static_cast<const storage*>(a.x) + (int64_t)r0 * a.ld + c;
    storage* out = static_cast<storage*>(a.out) + (int64_t)r0 * a.out_ld + c;
    auto allowed = [&](uint32_t r) {
        if (!kMask) return ALL;
        uint32_t m = 0;
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) m |= (words[e] >> r & 1u) << e;
        return m;
    };
    u32x4 d[U];
    if constexpr (kInPlace) {
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t no = ~allowed(u) & mine;
            if (u >= n) break;
            if (no == ALL) {
                store16<false>(out + (int64_t)u * a.out_ld, masked<DT>(u32x4{0u, 0u, 0u, 0u}, 0u));
                continue;
            }
#pragma unroll
            for (uint32_t e = 0; e < EPV; ++e)
                if (no >> e & 1u) out[(int64_t)u * a.out_ld + e] = (storage)kMinusInf<DT>;
        }
        return;
    }
    if (mine == ALL) {
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) d[u] = load16<kOnce>(x + (int64_t)min_u32(u, n - 1u) * a.ld);
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
            if (u < n) store16<kOnce>(out + (int64_t)u * a.out_ld, kMask ? masked<DT>(d[u], allowed(u)) : d[u]);
        return;
    }
    // A vector with columns that are nobody's, or a row of less than one: read
    // whole, where the matrix reaches that far, and written by the element.
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
        const uint32_t r = min_u32(u, n - 1u);
        if ((int64_t)(V - 1u - (r0 + r)) * a.ld + a.C >= (int64_t)c + EPV) {
            d[u] = load16<false>(x + (int64_t)r * a.ld);
        } else {
            storage v[EPV] = {};
#pragma unroll
            for (uint32_t e = 0; e < EPV; ++e)
                if (mine >> e & 1u) v[e] = x[(int64_t)r * a.ld + e];
            __builtin_memcpy(&d[u], v, 16);
        }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
        const uint32_t m = allowed(u);
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e)
            if (u < n && (mine >> e & 1u))
                out[(int64_t)u * a.out_ld + e] = m >> e & 1u ? (storage)vec_elem<DT>(d[u], (int)e) : (storage)kMinusInf<DT>;
    }
}

template <class DT, int kMode, bool kMask, uint32_t U>
__global__ __launch_bounds__(kBlock) void adjust_row_dense(AdjustArgs a, uint32_t tx_log, uint32_t tile0) {
    __shared__ uint8_t active[kRowTileVecs * DT::kPerVec];
    row_dense<DT, kMode, kMask, U>(a, tx_log, blockIdx.x, tile0 + blockIdx.y, active);
}

constexpr uint32_t kSparseRows = 4096;

// Lane l, its touched rows in tile `tile` of `tiles`, 1 << w_log threads to a
// row; of the parts (a power of two) workgroups with the same rows, each takes
// every parts-th group of 32.
template <class DT, bool kBias, bool kMask>
__device__ __forceinline__ void row_sparse(const AdjustArgs& a, uint32_t tile, uint32_t tiles, uint32_t l, uint32_t part, uint32_t parts,
                                           uint32_t w_log, TouchedRows<kSparseRows, kBias>& sh) {
    using storage = typename DT::storage;
    const uint32_t tid = threadIdx.x;
    using R = Rows<kSparseRows, 256>;
    const R rows{tiles, tile};
    const Lane<R, kBias> lane(a, rows, l);
    if (lane.ce == lane.cb) return;
    uint32_t draft0, bias0;
    first_entries(a, lane, draft0, bias0);
    make_list(a, rows, lane, draft0, bias0, sh, part, parts);
    __syncthreads();

    const LaneRules rules(lane.rep, lane.pres, lane.freq);
    const uint32_t n_rows = sh.n, step = kBlock >> w_log;
    const int32_t* counts = a.counts ? a.counts + (int64_t)l * a.counts_ld : nullptr;
    for (uint32_t j = tid & ((1u << w_log) - 1u); j < lane.ce - lane.cb; j += 1u << w_log) {
        const uint32_t c = lane.cb + j;
        const uint32_t* mask = kMask ? mask_row(a, c) : nullptr;
        constexpr uint32_t U = 2;  // rows whose reads are in flight together
        for (uint32_t k0 = tid >> w_log; k0 < n_rows; k0 += step * U) {
            uint32_t at[U], row[U], counted[U], raw[U], ok[U], b[U];
            float bias[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                at[u] = sh.list[min_u32(k0 + u * step, n_rows - 1u)];
                row[u] = rows.row(at[u]);
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                counted[u] = (uint32_t)*(counts ? counts + row[u] : safe<int32_t>());
                raw[u] = (uint32_t)static_cast<const storage*>(a.x)[(int64_t)row[u] * a.ld + c];
                ok[u] = kMask ? *(mask ? mask + (row[u] >> 5) : safe<uint32_t>()) : 0u;
                b[u] = kBias ? sh.bias_at[kBias ? at[u] : 0] : 0u;
                bias[u] = kBias ? a.bias_values[b[u] ? lane.bb + b[u] - 1u : 0u] : 0.0f;
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                if (k0 + u * step >= n_rows || (mask && !(ok[u] >> (row[u] & 31u) & 1u))) continue;  // stays -Inf
                const uint32_t word = counts ? counted[u] : 0u;
                uint32_t times = word & 0x7FFFFFFFu;
                if (a.drafts && (sh.drafted[at[u] >> 5] >> (at[u] & 31u) & 1u)) {
                    DraftsOfRow drafts;
                    drafts.find(a, lane, row[u]);
                    times += drafts.before(a, lane, row[u], j);
                }
                const bool seen = word != 0 || times;
                // (a later column's draft changes nothing here)
                if (seen || b[u])
                    static_cast<storage*>(a.out)[(int64_t)row[u] * a.out_ld + c] = (storage)from_double<DT>(
                        rules.apply((double)to_float<DT>(raw[u]), seen, rules.penalty(times), b[u] != 0, (double)bias[u]));
            }
        }
    }
}

template <class DT, bool kBias, bool kMask>
__global__ __launch_bounds__(kBlock) void adjust_row_sparse(AdjustArgs a, uint32_t l0, uint32_t w_log) {
    __shared__ TouchedRows<kSparseRows, kBias> sh;
    row_sparse<DT, kBias, kMask>(a, blockIdx.x, gridDim.x, l0 + blockIdx.y, blockIdx.z, gridDim.z, w_log, sh);
}

// In place, with masks: the two write different elements, so one launch does
// both.  The first n_sparse workgroups take the touched rows from lane l0 on,
// `parts` to each of a lane's `tiles`, the others the masks, a column tile after
// the other.
template <class DT, bool kBias, uint32_t U>
__global__ __launch_bounds__(kBlock) void adjust_row_in_place(AdjustArgs a, uint32_t l0, uint32_t n_sparse, uint32_t tiles, uint32_t parts,
                                                              uint32_t w_log, uint32_t row_tiles, uint32_t tx_log) {
    __shared__ TouchedRows<kSparseRows, kBias> sh;
    __shared__ uint8_t active[kRowTileVecs * DT::kPerVec];
    if (blockIdx.x < n_sparse) {
        const uint32_t p = blockIdx.x / tiles, l = p / parts;
        row_sparse<DT, kBias, true>(a, blockIdx.x - p * tiles, tiles, l0 + l, p - l * parts, parts, w_log, sh);
    } else {
        const uint32_t i = blockIdx.x - n_sparse, t = i / row_tiles;
        row_dense<DT, kModeInPlace, true, U>(a, tx_log, i - t * row_tiles, t, active);
    }
}

// ----------------------------------------------------------------- launch ---

constexpr int64_t kRowVecs = 1 << 20;
constexpr int64_t kInPlaceWgs = 1 << 22;  // a grid has at most 2^32 threads

// A matrix that, read and written, exceeds the 256 MB Infinity Cache goes past
// the caches: 448 columns of 248,046 bf16 rows 102 to 96 us (column-contiguous)
// and 117 to 108 (interleaved), 56 columns 13.0 but 15.7.
bool past_caches(const AdjustArgs& a, int element_bytes) {
    return 2 * (int64_t)a.V * a.C * element_bytes > (int64_t(256) << 20);
}

template <class DT, int kMode, uint32_t U, bool kBias, bool kMask>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t rows = kBlock * DT::kPerVec, tiles = (a.V + rows - 1) / rows;
    // A workgroup per U columns of a lane of average size.  Where nothing is
    // streamed most of one is the list: more columns share it as soon as not all
    // workgroups run at once (in place, 448 columns of 248,046 rows 27.2 and 19.3
    // us, 256 columns 19.0 and 13.2; dense histories of 672 columns of 50,958
    // rows 37.1 but 40.3).
    uint32_t z = min(((a.C + a.lanes - 1) / a.lanes + U - 1) / U, (uint32_t)kGridY);
    if (kMode == kModeInPlace && !kMask)
        while (z > 1 && (uint64_t)tiles * a.lanes * z > 2048) z = (z + 1) / 2;
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const uint32_t n = (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY);
        hipLaunchKernelGGL((adjust_col<DT, kMode, U, kBias, kMask>), dim3(tiles, n, z), dim3(kBlock), 0, stream, a, (uint32_t)l0);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, int kMode, uint32_t U>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    if (a.bias_ids) return a.mask ? launch_col<DT, kMode, U, true, true>(a, stream) : launch_col<DT, kMode, U, true, false>(a, stream);
    return a.mask ? launch_col<DT, kMode, U, false, true>(a, stream) : launch_col<DT, kMode, U, false, false>(a, stream);
}

// Columns of a workgroup: one, as long as all workgroups run at once (the
// scattered reads of the touched rows then spread over the CUs), else four
// that share a list.  7 columns of 16,384 rows 4.4 us by ones, 7.0 by fours;
// of 248,046 rows 5.7 and 8.9; 56 columns 17.4 and 16.6, in place 12.1 and 7.3.
// Lanes of one column have nothing to share: 256 of them 73 and 119 us (of two,
// 64 lanes 37 and 39, in place 21 and 14).
template <class DT, int kMode>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t rows = kBlock * DT::kPerVec;
    const uint64_t wgs = (uint64_t)((a.V + rows - 1) / rows) * (a.C > a.lanes ? a.C : a.lanes);
    return wgs <= 2048 || a.C < 2 * (uint64_t)a.lanes ? launch_col<DT, kMode, 1>(a, stream) : launch_col<DT, kMode, 4>(a, stream);
}

template <class DT>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    if (a.x == a.out) return launch_col<DT, kModeInPlace>(a, stream);
    const int e = 16 / DT::kPerVec;
    if (past_caches(a, e)) return launch_col<DT, kModeOnce>(a, stream);
    // Short runs cost where the columns do not start on cache lines: a run of
    // 512 bytes then touches five lines for four.  32 columns, histories of
    // 500 and 4,000 tokens: 131,072 rows 5.8 and 6.3 us in short runs, 6.4 and
    // 9.1 in long ones; 248,046 rows 11.2 and 12.1, and 9.8 and 11.4.
    const bool lines = ((uintptr_t)a.x | (uintptr_t)a.out | (uint64_t)a.ld * e | (uint64_t)a.out_ld * e) % 128 == 0;
    return lines ? launch_col<DT, kModeShort>(a, stream) : launch_col<DT, kModeLong>(a, stream);
}

// How the row kernels cut the work.
template <class DT>
struct RowCut {
    uint32_t vecs, tx_log = 0, rows;          // masks and copies: vectors of a row, of a workgroup, rows of a thread
    uint32_t tiles, parts = 1, w_log = 0;     // touched rows
    explicit RowCut(const AdjustArgs& a) {
        vecs = (a.C + DT::kPerVec - 1) / DT::kPerVec;
        while ((1u << tx_log) < vecs && (1u << tx_log) < kRowTileVecs) ++tx_log;
        // Without penalties: 8 columns of 248,046 rows 7.3 us in fours, 10.3 in
        // sixteens; 56 columns 17.8 and 15.7; 448 columns 120 and 92.
        rows = (int64_t)a.V * vecs >= kRowVecs ? 16 : 4;
        tiles = (a.V + kSparseRows - 1) / kSparseRows;
        const uint32_t cols = (a.C + a.lanes - 1) / a.lanes;
        while (w_log < 6 && (1u << w_log) < cols) ++w_log;
        // In few tiles a history may touch nearly all rows; as long as the CUs have
        // room, several workgroups share them: 41 lanes of 9 columns, 1,532 rows,
        // in place 37 us by ones, 8.8 by sixteens.
        while (parts < 16 && tiles * parts < 32 && (uint64_t)tiles * a.lanes * parts < 1024) parts *= 2;
    }
    uint32_t row_tiles(const AdjustArgs& a) const {
        const uint32_t n = (kBlock >> tx_log) * rows;
        return (a.V + n - 1) / n;
    }
    uint32_t col_tiles() const { return (vecs + (1u << tx_log) - 1) >> tx_log; }
};

template <class DT, int kMode, bool kMask>
hipError_t launch_row_dense(const AdjustArgs& a, hipStream_t stream) {
    const RowCut<DT> cut(a);
    for (uint32_t t = 0; t < cut.col_tiles(); t += (uint32_t)kGridY) {
        const dim3 grid(cut.row_tiles(a), min(cut.col_tiles() - t, (uint32_t)kGridY));
        // (a matrix past the caches has more than kRowVecs vectors)
        if (kMode == kModeOnce || cut.rows == 16)
            hipLaunchKernelGGL((adjust_row_dense<DT, kMode, kMask, 16>), grid, dim3(kBlock), 0, stream, a, cut.tx_log, t);
        else
            hipLaunchKernelGGL((adjust_row_dense<DT, kMode == kModeOnce ? kModeLong : kMode, kMask, 4>), grid, dim3(kBlock), 0, stream, a,
                               cut.tx_log, t);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kBias, bool kMask>
hipError_t launch_row_sparse(const AdjustArgs& a, hipStream_t stream) {
    const RowCut<DT> cut(a);
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const dim3 grid(cut.tiles, (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY), cut.parts);
        hipLaunchKernelGGL((adjust_row_sparse<DT, kBias, kMask>), grid, dim3(kBlock), 0, stream, a, (uint32_t)l0, cut.w_log);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kBias, uint32_t U>
hipError_t launch_row_in_place(const AdjustArgs& a, const RowCut<DT>& cut, bool sparse, hipStream_t stream) {
    // the masks with the first of the lanes (all of them, unless those are very many)
    const int64_t each = (int64_t)cut.tiles * cut.parts, most = each < kInPlaceWgs ? kInPlaceWgs / each : 1;
    for (int64_t l0 = 0; l0 < (sparse ? (int64_t)a.lanes : 1); l0 += most) {
        const uint32_t n = sparse ? (uint32_t)(each * (a.lanes - l0 < most ? a.lanes - l0 : most)) : 0u;
        const uint32_t masks = l0 == 0 ? cut.row_tiles(a) * cut.col_tiles() : 0u;
        hipLaunchKernelGGL((adjust_row_in_place<DT, kBias, U>), dim3(n + masks), dim3(kBlock), 0, stream, a, (uint32_t)l0, n, cut.tiles,
                           cut.parts, cut.w_log, cut.row_tiles(a), cut.tx_log);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kBias>
hipError_t launch_row_in_place(const AdjustArgs& a, bool sparse, hipStream_t stream) {
    const RowCut<DT> cut(a);
    return cut.rows == 16 ? launch_row_in_place<DT, kBias, 16>(a, cut, sparse, stream)
                          : launch_row_in_place<DT, kBias, 4>(a, cut, sparse, stream);
}

template <class DT>
hipError_t launch_row_sparse(const AdjustArgs& a, hipStream_t stream) {
    if (a.bias_ids) return a.mask ? launch_row_sparse<DT, true, true>(a, stream) : launch_row_sparse<DT, true, false>(a, stream);
    return a.mask ? launch_row_sparse<DT, false, true>(a, stream) : launch_row_sparse<DT, false, false>(a, stream);
}

template <class DT, int kMode>
hipError_t launch_row_copy(const AdjustArgs& a, hipStream_t stream) {
    return a.mask ? launch_row_dense<DT, kMode, true>(a, stream) : launch_row_dense<DT, kMode, false>(a, stream);
}

template <class DT>
hipError_t launch_dt(int layout, const AdjustArgs& a, hipStream_t stream) {
    const bool sparse = a.counts || a.drafts || a.bias_ids;
    const bool in_place = a.x == a.out;
    if (in_place && !sparse && !a.mask) return hipSuccess;
    if (layout == TOPK_COL_CONTIG) return launch_col<DT>(a, stream);
    if (in_place && a.mask) return a.bias_ids ? launch_row_in_place<DT, true>(a, sparse, stream) : launch_row_in_place<DT, false>(a, sparse, stream);
    if (!in_place)
        if (const hipError_t e = past_caches(a, 16 / DT::kPerVec) ? launch_row_copy<DT, kModeOnce>(a, stream)
                                                                  : launch_row_copy<DT, kModeLong>(a, stream);
            e != hipSuccess)
            return e;
    return sparse ? launch_row_sparse<DT>(a, stream) : hipSuccess;
}

}  // namespace

hipError_t launch_adjust(int dtype, int layout, const AdjustArgs& a, hipStream_t stream) {
    return dtype == TOPK_BF16 ? launch_dt<Bf16>(layout, a, stream) : launch_dt<F32>(layout, a, stream);
}

}  // namespace topk
