// Penalties, biases and masks on logits, for gfx950.
//
// For row r of column c (column j of lane l), with n the token's count in the
// lane's output and its first j drafts:
//   seen (in the prompt, or n > 0):  x = x > 0 ? x / rep : x * rep
//   n > 0:                           x = x - (freq * n + pres)
//   biased:                          x = x + bias
//   forbidden by the mask:           x = -Inf
//
// Column-contiguous: one kernel.  A workgroup takes a few thousand rows of all
// of a lane's columns.  It streams them (in place: only what the mask
// forbids), finds the rows that a penalty or bias touches from one bit per row
// of the history, and rewrites those in every column from the original.
//
// Row-interleaved: two kernels.  The dense one streams the matrix: it copies
// the elements (nothing to copy in place) and writes -Inf where the mask
// forbids them.  The sparse one rewrites the elements that a penalty or a
// bias touches: a few thousand of a column's 248,046 rows.  It reads the
// originals, so it follows the dense one out of place and precedes it in
// place; forbidden elements it leaves alone.
//
// The penalised value is a chain of four operations.  It is carried in
// binary64 (division as a product with the rounded reciprocal, off by 2^-52)
// and rounded to binary32 and then to the type: the chain adds nothing to the
// final rounding that could be seen, and it is too rare to cost time.
#include "topk_round.hpp"

#include "topk_col_common.hpp"

namespace topk {

namespace {

constexpr uint32_t kTile = 8192;  // rows per workgroup (row-interleaved, sparse)

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

struct LaneRules {
    double rep, inv, pres, freq;
    __device__ LaneRules(float r, float p, float f, bool has_r = true)
        : rep(has_r ? (double)r : 1.0), inv(1.0 / rep), pres((double)p), freq((double)f) {}
    __device__ explicit LaneRules(const AdjustArgs& a, uint32_t l)
        : LaneRules(a.repetition ? a.repetition[l] : 1.0f, a.presence ? a.presence[l] : 0.0f,
                    a.frequency ? a.frequency[l] : 0.0f) {}
    __device__ __forceinline__ double apply(double x, bool prompt, uint32_t n, double bias) const {
        if (prompt || n) x = x > 0.0 ? x * inv : x * rep;
        if (n) x -= freq * (double)n + pres;
        return x + bias;
    }
};

// The mask row of a column, or NULL if it has none.
__device__ __forceinline__ const uint32_t* mask_row(const AdjustArgs& a, uint32_t c) {
    if (!a.mask) return nullptr;
    const int64_t m = a.mask_index ? (int64_t)a.mask_index[c] : (int64_t)c;
    return m >= 0 && m < a.mask_count ? a.mask + m * a.mask_ld : nullptr;
}

// 16 bytes at element alignment (global memory takes any).
template <class T>
__device__ __forceinline__ u32x4 load16(const T* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
template <class T>
__device__ __forceinline__ void store16(T* p, const u32x4& v) {
    __builtin_memcpy(p, &v, 16);
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

// ------------------------------------------------------ column-contiguous ---

// Rows of a workgroup: one 16-byte vector per thread, in runs of 256 rows that
// lie `tiles` runs apart.  The ids of a vocabulary sorted by use put most of a
// history into the first rows; in one contiguous tile they would hold up the
// whole launch.  256 rows are the most that a workgroup rewrites in one go,
// and whole cache lines.
template <class DT>
struct ColRows {
    static constexpr uint32_t EPV = DT::kPerVec, RUN = 256, ROWS = kBlock * EPV, WORDS = ROWS / 32;
    uint32_t tiles, tile;
    __device__ __forceinline__ uint32_t row(uint32_t at) const { return (at / RUN * tiles + tile) * RUN + at % RUN; }
    // the place of row r, or ROWS if it is another workgroup's
    __device__ __forceinline__ uint32_t place(uint32_t r, uint32_t V) const {
        const uint32_t run = r / RUN, i = run / tiles;
        return r < V && run - i * tiles == tile ? i * RUN + r % RUN : ROWS;
    }
};

template <class DT, bool kBias>
struct ColShared {
    using Rows = ColRows<DT>;
    alignas(16) uint32_t bias_at[kBias ? Rows::ROWS : 4];  // 1 + the last list entry of a place, or 0
    uint32_t touched[Rows::WORDS];  // places with a history, a draft or a bias
    uint32_t drafted[Rows::WORDS];  // places that are drafts
    uint16_t list[Rows::ROWS];      // the touched places, in any order
    uint32_t n;
};

constexpr uint32_t kColsAtOnce = 4;  // columns whose vectors a thread has in flight

// An address that can be read in place of an absent array's, so that a read
// needs no branch (a branch around it would make the next ones wait).
template <class T>
__device__ __forceinline__ const T* or_safe(const T* p) {
    return p ? p : (const T*)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
}

// Lane l0 + blockIdx.y, its columns blockIdx.z * U, .. + U - 1, then
// gridDim.z * U further on.  The columns share the search for the rows that a
// penalty or bias touches and the reading of their counts.
//
// At these sizes the time is that of the chain of dependent reads: reads of
// one link are issued together, at addresses cut to the last valid one instead
// of behind branches.
template <class DT, bool kInPlace, bool kBias, bool kMask>
__global__ __launch_bounds__(kBlock) void adjust_col(AdjustArgs a, uint32_t l0) {
    using storage = typename DT::storage;
    using Rows = ColRows<DT>;
    constexpr uint32_t EPV = DT::kPerVec, ALL = (1u << EPV) - 1u, U = kColsAtOnce;
    __shared__ ColShared<DT, kBias> sh;
    const uint32_t l = l0 + blockIdx.y, tid = threadIdx.x, V = a.V;
    const Rows rows{gridDim.x, blockIdx.x};
    const bool sparse = a.counts || a.drafts || kBias;

    // all that hangs on the lane alone
    const int32_t* cs = a.cols.start ? a.cols.start + l : or_safe<int32_t>(nullptr);
    const int32_t* ds = a.draft_parts.start ? a.draft_parts.start + l : or_safe<int32_t>(nullptr);
    const int32_t* bs = kBias ? a.bias_parts.start + l : or_safe<int32_t>(nullptr);
    const float* rp = a.repetition ? a.repetition + l : or_safe<float>(nullptr);
    const float* pp = a.presence ? a.presence + l : or_safe<float>(nullptr);
    const float* fp = a.frequency ? a.frequency + l : or_safe<float>(nullptr);
    const uint32_t wr = rows.row(min_u32(tid, Rows::WORDS - 1u) * 32u);  // this thread's 32 rows
    const uint32_t* sp = a.seen ? a.seen + (int64_t)l * a.seen_ld + (min_u32(wr, V - 1u) >> 5) : or_safe<uint32_t>(nullptr);
    const int32_t c0s = cs[0], c1s = cs[1], d0s = ds[0], d1s = ds[1], b0s = bs[0], b1s = bs[1];
    const float rep = *rp, pres = *pp, freq = *fp;
    uint32_t word = *sp;
    uint32_t cb, ce, db, de, bb, be;
    a.cols.cut(l, c0s, c1s, cb, ce);
    a.draft_parts.cut(l, d0s, d1s, db, de);
    a.bias_parts.cut(l, b0s, b1s, bb, be);
    const uint32_t c_first = cb + blockIdx.z * U, c_step = gridDim.z * U;
    if (c_first >= ce) return;
    if (!a.drafts) de = db;
    de = min_u32(de, db + (ce - cb - 1u));  // the last draft precedes the last column

    // The streamed part copies (out of place) and masks.
    const uint32_t r = rows.row(tid * EPV);          // this thread's rows
    const uint32_t nvec = V / EPV;                   // whole vectors of a column
    const bool whole = r / EPV < nvec;
    const uint32_t rr = whole ? r : 0u;              // a vector that can be read, if there is one
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
                if (!kInPlace) d[u] = load16(static_cast<const storage*>(a.x) + (int64_t)min_u32(c0 + u, ce - 1u) * a.ld + rr);
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
                if (c0 + u < ce && m[u] != ALL && m[u]) d[u] = load16(static_cast<const storage*>(a.x) + (int64_t)(c0 + u) * a.ld + r);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (c0 + u >= ce || r >= V || (kInPlace && m[u] == ALL)) continue;
            const storage* x = static_cast<const storage*>(a.x) + (int64_t)(c0 + u) * a.ld;
            storage* out = static_cast<storage*>(a.out) + (int64_t)(c0 + u) * a.out_ld;
            if (whole) {
                store16(out + r, kMask ? masked<DT>(d[u], m[u]) : d[u]);
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

    // the touched places as a list
    if (sparse) {
        if (tid >= Rows::WORDS || wr >= V || !a.seen) word = 0;
        else if (V - wr < 32u) word &= (1u << (V - wr)) - 1u;  // bits past the last row mean nothing
        if (tid == 0) sh.n = 0;
        if (a.drafts || kBias) {
            if (tid < Rows::WORDS) {
                sh.touched[tid] = word;
                sh.drafted[tid] = 0;
            }
            if constexpr (kBias)
                for (uint32_t i = tid; i < Rows::ROWS / 4; i += kBlock) reinterpret_cast<u32x4*>(sh.bias_at)[i] = u32x4{0u, 0u, 0u, 0u};
            __syncthreads();
            for (uint32_t i = db + tid; i < de; i += kBlock) {
                const uint32_t at = rows.place((uint32_t)a.drafts[i], V);
                if (at == Rows::ROWS) continue;
                atomicOr(&sh.touched[at >> 5], 1u << (at & 31u));
                atomicOr(&sh.drafted[at >> 5], 1u << (at & 31u));
            }
            if constexpr (kBias) {
                for (uint32_t i = bb + tid; i < be; i += kBlock) {
                    const uint32_t at = rows.place((uint32_t)a.bias_ids[i], V);
                    if (at == Rows::ROWS) continue;
                    atomicOr(&sh.touched[at >> 5], 1u << (at & 31u));
                    atomicMax(&sh.bias_at[at], i - bb + 1u);
                }
            }
            __syncthreads();
            word = tid < Rows::WORDS ? sh.touched[tid] : 0u;
        } else {
            __syncthreads();
        }
        if (word) {
            uint32_t pos = atomicAdd(&sh.n, (uint32_t)__popc(word));
            for (; word; word &= word - 1u) sh.list[pos++] = (uint16_t)(tid * 32u + (uint32_t)__builtin_ctz(word));
        }
    }
    if constexpr (stream) {
        store_columns(c_first);
        for (uint32_t c0 = c_first + c_step; c0 < ce; c0 += c_step) {
            load_columns(c0);
            store_columns(c0);
        }
    }
    if (!sparse) return;
    __syncthreads();  // for the list, and for the streamed stores, which those below replace

    const LaneRules rules(rep, a.presence ? pres : 0.0f, a.frequency ? freq : 0.0f, a.repetition != nullptr);
    const uint32_t n_rows = sh.n;
    const int32_t* counts = a.counts ? a.counts + (int64_t)l * a.counts_ld : nullptr;
    for (uint32_t k = tid; k < n_rows; k += kBlock) {
        const uint32_t at = sh.list[k], row = rows.row(at);
        uint32_t counted = (uint32_t)*(counts ? counts + row : or_safe<int32_t>(nullptr));
        const uint32_t b = kBias ? sh.bias_at[kBias ? at : 0] : 0u;
        const float bias_value = kBias ? a.bias_values[b ? bb + b - 1u : 0u] : 0.0f;
        uint64_t drafts = 0;  // bit i: draft i of the first 64 is this row
        bool drafted = false;
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
                if (a.drafts) {
                    drafted = sh.drafted[at >> 5] >> (at & 31u) & 1u;
                    if (drafted)
#pragma unroll 8
                        for (uint32_t i = 0; i < min_u32(de - db, 64u); ++i) drafts |= (uint32_t)a.drafts[db + i] == row ? 1ull << i : 0ull;
                }
            }
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                if (c0 + u >= ce || (kMask && !(ok[u] & 1u))) continue;  // a forbidden element stays -Inf
                uint32_t times = counted & 0x7FFFFFFFu;
                if (drafted) {
                    const uint32_t j = c0 + u - cb;  // drafts before the column
                    times += (uint32_t)__popcll(j < 64u ? drafts & ((1ull << j) - 1u) : drafts);
                    for (uint32_t i = db + 64u; i < min_u32(de, db + j); ++i) times += (uint32_t)a.drafts[i] == row ? 1u : 0u;
                }
                // (a later column's draft changes nothing here)
                if (counted >> 31 || times || b)
                    (static_cast<storage*>(a.out) + (int64_t)(c0 + u) * a.out_ld)[row] = (storage)from_double<DT>(
                        rules.apply((double)to_float<DT>(raw[u]), counted >> 31, times, b ? (double)bias_value : 0.0));
            }
        }
    }
}

// -------------------------------------------------------- row-interleaved ---

constexpr uint32_t kRowTileVecs = 64;  // at most 64 vectors of a row per workgroup

// Row-interleaved: a workgroup takes 1 << tx_log vectors of a row; each
// thread one of them over 32 rows, which one word of each column's mask
// covers.
template <class DT, bool kInPlace>
__global__ __launch_bounds__(kBlock) void adjust_row_dense(AdjustArgs a, uint32_t tx_log, uint32_t tile0) {
    using storage = typename DT::storage;
    constexpr uint32_t EPV = DT::kPerVec, ALL = (1u << EPV) - 1u;
    __shared__ uint8_t active[kRowTileVecs * EPV];
    const uint32_t tid = threadIdx.x;
    const uint32_t tile_c = ((tile0 + blockIdx.y) << tx_log) * EPV, tile_n = EPV << tx_log;
    if (a.cols.start) {
        for (uint32_t i = tid; i < tile_n; i += kBlock) active[i] = 0;
        __syncthreads();
        for (uint32_t l = tid; l < a.lanes; l += kBlock) {
            uint32_t b, e;
            a.cols.range(l, b, e);
            e = min_u32(e, tile_c + tile_n);
            for (uint32_t c = b < tile_c ? tile_c : b; c < e; ++c) active[c - tile_c] = 1;
        }
        __syncthreads();
    }
    const uint32_t vc = tid & ((1u << tx_log) - 1u);
    const uint32_t c = tile_c + vc * EPV;
    const uint32_t rows = (kBlock >> tx_log) * 32u;
    const uint32_t r0 = blockIdx.x * rows + (tid >> tx_log) * 32u;
    if (c >= a.C || r0 >= a.V) return;
    uint32_t mine = 0;  // bit e: column c + e is a lane's
    uint32_t words[EPV];
#pragma unroll
    for (uint32_t e = 0; e < EPV; ++e) {
        words[e] = 0xFFFFFFFFu;
        if (c + e < a.C && (!a.cols.start || active[vc * EPV + e])) {
            mine |= 1u << e;
            if (const uint32_t* m = mask_row(a, c + e)) words[e] = m[r0 >> 5];
        }
    }
    const uint32_t n = min_u32(32u, a.V - r0);
    const storage* x = static_cast<const storage*>(a.x) + (int64_t)r0 * a.ld + c;
    storage* out = static_cast<storage*>(a.out) + (int64_t)r0 * a.out_ld + c;
#pragma unroll 4
    for (uint32_t r = 0; r < n; ++r, x += a.ld, out += a.out_ld) {
        uint32_t allowed = 0;
#pragma unroll
        for (uint32_t e = 0; e < EPV; ++e) allowed |= (words[e] >> r & 1u) << e;
        if (kInPlace && allowed == ALL) continue;
        if (mine == ALL) {
            store16(out, masked<DT>(load16(x), allowed));
        } else {
            for (uint32_t e = 0; e < EPV; ++e)
                if ((mine >> e & 1u) && (!kInPlace || !(allowed >> e & 1u)))
                    out[e] = allowed >> e & 1u ? x[e] : (storage)kMinusInf<DT>;
        }
    }
}

template <bool kBias>
struct SparseShared {
    uint32_t touched[kTile / 32];           // rows of the tile with a history, a draft or a bias
    uint32_t drafted[kTile / 32];           // rows that are drafts
    uint32_t bias_at[kBias ? kTile : 1];    // 1 + the last list entry of a row, or 0
    uint16_t rows[kTile];                   // the touched rows
    uint32_t wave_sum[kWaves];
};

// Lane l0 + blockIdx.y, rows [blockIdx.x * kTile, ...), all the lane's columns.
template <class DT, bool kBias>
__global__ __launch_bounds__(kBlock) void adjust_row_sparse(AdjustArgs a, uint32_t l0) {
    using storage = typename DT::storage;
    __shared__ SparseShared<kBias> sh;
    static_assert(kTile / 32 == kBlock, "one word of the tile's rows per thread");
    const uint32_t tid = threadIdx.x, l = l0 + blockIdx.y, t0 = blockIdx.x * kTile;
    uint32_t cb, ce;
    a.cols.range(l, cb, ce);
    if (ce == cb) return;
    const uint32_t ncols = ce - cb;

    uint32_t word = 0;
    if (a.seen && t0 + tid * 32u < a.V) {
        word = a.seen[(int64_t)l * a.seen_ld + (t0 >> 5) + tid];
        const uint32_t left = a.V - (t0 + tid * 32u);
        if (left < 32u) word &= (1u << left) - 1u;  // bits past the last row mean nothing
    }
    sh.touched[tid] = word;
    sh.drafted[tid] = 0;
    if constexpr (kBias)
        for (uint32_t i = tid; i < kTile; i += kBlock) sh.bias_at[i] = 0;
    __syncthreads();
    uint32_t db = 0, de = 0;
    if (a.drafts) {
        a.draft_parts.range(l, db, de);
        de = min_u32(de, db + ncols - 1u);  // the last draft precedes the last column
        for (uint32_t i = db + tid; i < de; i += kBlock) {
            const uint32_t r = (uint32_t)a.drafts[i] - t0;
            if (r < kTile && r < a.V - t0) {
                atomicOr(&sh.touched[r >> 5], 1u << (r & 31u));
                atomicOr(&sh.drafted[r >> 5], 1u << (r & 31u));
            }
        }
    }
    uint32_t bb = 0, be = 0;
    if constexpr (kBias) {
        a.bias_parts.range(l, bb, be);
        for (uint32_t i = bb + tid; i < be; i += kBlock) {
            const uint32_t r = (uint32_t)a.bias_ids[i] - t0;
            if (r < kTile && r < a.V - t0) {
                atomicOr(&sh.touched[r >> 5], 1u << (r & 31u));
                atomicMax(&sh.bias_at[r], i - bb + 1u);
            }
        }
    }
    __syncthreads();

    // the touched rows as a list
    word = sh.touched[tid];
    const uint32_t lane = tid & 63u, mine = (uint32_t)__popc(word);
    uint32_t upto = mine;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63u) sh.wave_sum[tid >> 6] = upto;
    __syncthreads();
    uint32_t base = upto - mine, nrows = 0;
#pragma unroll
    for (uint32_t w = 0; w < (uint32_t)kWaves; ++w) {
        if (w < tid >> 6) base += sh.wave_sum[w];
        nrows += sh.wave_sum[w];
    }
    for (; word; word &= word - 1u) sh.rows[base++] = (uint16_t)(tid * 32u + (uint32_t)__builtin_ctz(word));
    __syncthreads();

    const LaneRules rules(a, l);
    const uint64_t items = (uint64_t)nrows * ncols;
    for (uint64_t it = tid; it < items; it += kBlock) {
        // neighbouring threads: neighbouring columns of a row
        const uint32_t i = (uint32_t)(it / ncols), j = (uint32_t)(it % ncols);
        const uint32_t r = sh.rows[i], row = t0 + r, c = cb + j;
        const uint32_t w = a.counts ? (uint32_t)a.counts[(int64_t)l * a.counts_ld + row] : 0u;
        uint32_t n = w & 0x7FFFFFFFu;
        if (sh.drafted[r >> 5] >> (r & 31u) & 1u)
            for (uint32_t d = db; d < min_u32(de, db + j); ++d) n += (uint32_t)a.drafts[d] == row ? 1u : 0u;
        const uint32_t at = kBias ? sh.bias_at[kBias ? r : 0] : 0u;
        if (!(w >> 31) && n == 0 && at == 0) continue;  // a later column's draft
        const uint32_t* mask = mask_row(a, c);
        if (mask && !(mask[row >> 5] >> (row & 31u) & 1u)) continue;
        const double v = (double)to_float<DT>((uint32_t)static_cast<const storage*>(a.x)[(int64_t)row * a.ld + c]);
        const double bias = at ? (double)a.bias_values[bb + at - 1u] : 0.0;
        static_cast<storage*>(a.out)[(int64_t)row * a.out_ld + c] = (storage)from_double<DT>(rules.apply(v, w >> 31, n, bias));
    }
}

// ----------------------------------------------------------------- launch ---

template <class DT, bool kInPlace, bool kBias, bool kMask>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t rows = ColRows<DT>::ROWS, tiles = (a.V + rows - 1) / rows;
    // a workgroup per kColsAtOnce columns of a lane of average size
    const uint32_t z = min(((a.C + a.lanes - 1) / a.lanes + kColsAtOnce - 1) / kColsAtOnce, (uint32_t)kGridY);
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const uint32_t n = (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY);
        hipLaunchKernelGGL((adjust_col<DT, kInPlace, kBias, kMask>), dim3(tiles, n, z), dim3(kBlock), 0, stream, a, (uint32_t)l0);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kInPlace>
hipError_t launch_col(const AdjustArgs& a, hipStream_t stream) {
    if (a.bias_ids)
        return a.mask ? launch_col<DT, kInPlace, true, true>(a, stream) : launch_col<DT, kInPlace, true, false>(a, stream);
    return a.mask ? launch_col<DT, kInPlace, false, true>(a, stream) : launch_col<DT, kInPlace, false, false>(a, stream);
}

template <class DT, bool kInPlace>
hipError_t launch_row_dense(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t vecs = (a.C + DT::kPerVec - 1) / DT::kPerVec;
    uint32_t tx_log = 0;
    while ((1u << tx_log) < vecs && (1u << tx_log) < kRowTileVecs) ++tx_log;
    const uint32_t rows = (kBlock >> tx_log) * 32u;
    const uint32_t col_tiles = (vecs + (1u << tx_log) - 1) >> tx_log;
    for (uint32_t t = 0; t < col_tiles; t += (uint32_t)kGridY) {
        const dim3 grid((a.V + rows - 1) / rows, min(col_tiles - t, (uint32_t)kGridY));
        hipLaunchKernelGGL((adjust_row_dense<DT, kInPlace>), grid, dim3(kBlock), 0, stream, a, tx_log, t);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kBias>
hipError_t launch_row_sparse(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t tiles = (a.V + kTile - 1) / kTile;
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const dim3 grid(tiles, (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY));
        hipLaunchKernelGGL((adjust_row_sparse<DT, kBias>), grid, dim3(kBlock), 0, stream, a, (uint32_t)l0);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT>
hipError_t launch_dt(int layout, const AdjustArgs& a, hipStream_t stream) {
    const bool sparse = a.counts || a.drafts || a.bias_ids;
    const bool in_place = a.x == a.out;
    if (in_place && !sparse && !a.mask) return hipSuccess;
    if (layout == TOPK_COL_CONTIG)
        return in_place ? launch_col<DT, true>(a, stream) : launch_col<DT, false>(a, stream);
    if (!in_place)
        if (const hipError_t e = launch_row_dense<DT, false>(a, stream); e != hipSuccess) return e;
    if (sparse) {
        const hipError_t e = a.bias_ids ? launch_row_sparse<DT, true>(a, stream) : launch_row_sparse<DT, false>(a, stream);
        if (e != hipSuccess) return e;
    }
    return in_place && a.mask ? launch_row_dense<DT, true>(a, stream) : hipSuccess;
}

}  // namespace

hipError_t launch_adjust(int dtype, int layout, const AdjustArgs& a, hipStream_t stream) {
    return dtype == TOPK_BF16 ? launch_dt<Bf16>(layout, a, stream) : launch_dt<F32>(layout, a, stream);
}

}  // namespace topk
