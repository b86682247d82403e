// Penalties, biases and masks on logits, for gfx950.
//
// For row r of column c (column j of lane l), with n the token's count in the
// lane's output and its first j drafts:
//   seen (in the prompt, or n > 0):  x = x > 0 ? x / rep : x * rep
//   n > 0:                           x = x - (freq * n + pres)
//   biased:                          x = x + bias
//   forbidden by the mask:           x = -Inf
//
// Two kernels.  The dense one streams the matrix: it copies the elements
// (nothing to copy in place) and writes -Inf where the mask forbids them.
// The sparse one rewrites the elements that a penalty or a bias touches: a
// few thousand of a column's 248,046 rows.  It reads the originals, so it
// follows the dense one out of place and precedes it in place; forbidden
// elements it leaves alone.
//
// The penalised value is a chain of four operations.  It is carried in
// binary64 (division as a product with the rounded reciprocal, off by 2^-52)
// and rounded to binary32 and then to the type: the chain adds nothing to the
// final rounding that could be seen, and it is too rare to cost time.
#include "topk_round.hpp"

#include "topk_col_common.hpp"

namespace topk {

namespace {

constexpr uint32_t kTile = 8192;  // rows per workgroup

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
    __device__ explicit LaneRules(const AdjustArgs& a, uint32_t l)
        : rep(a.repetition ? (double)a.repetition[l] : 1.0), inv(1.0 / rep),
          pres(a.presence ? (double)a.presence[l] : 0.0), freq(a.frequency ? (double)a.frequency[l] : 0.0) {}
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

// ------------------------------------------------------------------ dense ---

// Column-contiguous: column c0 + blockIdx.y, rows [blockIdx.x * kTile, ...).
template <class DT, bool kInPlace>
__global__ __launch_bounds__(kBlock) void adjust_dense_col(AdjustArgs a, uint32_t c0) {
    using storage = typename DT::storage;
    constexpr uint32_t EPV = DT::kPerVec, ALL = (1u << EPV) - 1u;
    const uint32_t c = c0 + blockIdx.y, tid = threadIdx.x, t0 = blockIdx.x * kTile;
    if (a.cols.start) {  // does the column belong to a lane?
        bool mine = false;
        for (uint32_t l = tid; l < a.lanes; l += kBlock) {
            uint32_t b, e;
            a.cols.range(l, b, e);
            mine |= c >= b && c < e;
        }
        if (!__syncthreads_or(mine)) return;
    }
    const uint32_t* mask = mask_row(a, c);
    if (kInPlace && !mask) return;
    const storage* x = static_cast<const storage*>(a.x) + (int64_t)c * a.ld;
    storage* out = static_cast<storage*>(a.out) + (int64_t)c * a.out_ld;
#pragma unroll
    for (uint32_t i = 0; i < kTile / (kBlock * EPV); ++i) {
        const uint32_t r0 = t0 + (i * kBlock + tid) * EPV;
        if (r0 >= a.V) continue;
        const uint32_t allowed = mask ? (mask[r0 >> 5] >> (r0 & 31u)) & ALL : ALL;
        if (kInPlace && allowed == ALL) continue;
        if (r0 + EPV <= a.V) {
            store16(out + r0, masked<DT>(load16(x + r0), allowed));
        } else {
            for (uint32_t e = 0; r0 + e < a.V; ++e)
                if (!kInPlace || !(allowed >> e & 1u))
                    out[r0 + e] = allowed >> e & 1u ? x[r0 + e] : (storage)kMinusInf<DT>;
        }
    }
}

constexpr uint32_t kRowTileVecs = 64;  // at most 64 vectors of a row per workgroup

// Row-interleaved: a workgroup takes 1 << tx_log vectors of a row; each
// thread one of them over 32 rows, which one word of each column's mask
// covers.
template <class DT, bool kInPlace>
__global__ __launch_bounds__(kBlock) void adjust_dense_row(AdjustArgs a, uint32_t tx_log, uint32_t tile0) {
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

// ----------------------------------------------------------------- sparse ---

template <bool kBias>
struct SparseShared {
    uint32_t touched[kTile / 32];           // rows of the tile with a history, a draft or a bias
    uint32_t drafted[kTile / 32];           // rows that are drafts
    uint32_t bias_at[kBias ? kTile : 1];    // 1 + the last list entry of a row, or 0
    uint16_t rows[kTile];                   // the touched rows
    uint32_t wave_sum[kWaves];
};

// Lane l0 + blockIdx.y, rows [blockIdx.x * kTile, ...), all the lane's columns.
template <class DT, bool kRow, bool kBias>
__global__ __launch_bounds__(kBlock) void adjust_sparse(AdjustArgs a, uint32_t l0) {
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
        // neighbouring threads: neighbouring rows of a column, or columns of a row
        const uint32_t i = kRow ? (uint32_t)(it / ncols) : (uint32_t)(it % nrows);
        const uint32_t j = kRow ? (uint32_t)(it % ncols) : (uint32_t)(it / nrows);
        const uint32_t r = sh.rows[i], row = t0 + r, c = cb + j;
        const uint32_t w = a.counts ? (uint32_t)a.counts[(int64_t)l * a.counts_ld + row] : 0u;
        uint32_t n = w & 0x7FFFFFFFu;
        if (sh.drafted[r >> 5] >> (r & 31u) & 1u)
            for (uint32_t d = db; d < min_u32(de, db + j); ++d) n += (uint32_t)a.drafts[d] == row ? 1u : 0u;
        const uint32_t at = kBias ? sh.bias_at[kBias ? r : 0] : 0u;
        if (!(w >> 31) && n == 0 && at == 0) continue;  // a later column's draft
        const uint32_t* mask = mask_row(a, c);
        if (mask && !(mask[row >> 5] >> (row & 31u) & 1u)) continue;
        const int64_t xi = kRow ? (int64_t)row * a.ld + c : (int64_t)c * a.ld + row;
        const int64_t oi = kRow ? (int64_t)row * a.out_ld + c : (int64_t)c * a.out_ld + row;
        const double v = (double)to_float<DT>((uint32_t)static_cast<const storage*>(a.x)[xi]);
        const double bias = at ? (double)a.bias_values[bb + at - 1u] : 0.0;
        static_cast<storage*>(a.out)[oi] = (storage)from_double<DT>(rules.apply(v, w >> 31, n, bias));
    }
}

// ----------------------------------------------------------------- launch ---

template <class DT, bool kInPlace>
hipError_t launch_dense(int layout, const AdjustArgs& a, hipStream_t stream) {
    if (layout == TOPK_COL_CONTIG) {
        const uint32_t tiles = (a.V + kTile - 1) / kTile;
        for (int64_t c0 = 0; c0 < a.C; c0 += kGridY) {
            const uint32_t n = (uint32_t)(a.C - c0 < kGridY ? a.C - c0 : kGridY);
            hipLaunchKernelGGL((adjust_dense_col<DT, kInPlace>), dim3(tiles, n), dim3(kBlock), 0, stream, a, (uint32_t)c0);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const uint32_t vecs = (a.C + DT::kPerVec - 1) / DT::kPerVec;
    uint32_t tx_log = 0;
    while ((1u << tx_log) < vecs && (1u << tx_log) < kRowTileVecs) ++tx_log;
    const uint32_t rows = (kBlock >> tx_log) * 32u;
    const uint32_t col_tiles = (vecs + (1u << tx_log) - 1) >> tx_log;
    for (uint32_t t = 0; t < col_tiles; t += (uint32_t)kGridY) {
        const dim3 grid((a.V + rows - 1) / rows, min(col_tiles - t, (uint32_t)kGridY));
        hipLaunchKernelGGL((adjust_dense_row<DT, kInPlace>), grid, dim3(kBlock), 0, stream, a, tx_log, t);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT, bool kRow>
hipError_t launch_sparse(const AdjustArgs& a, hipStream_t stream) {
    const uint32_t tiles = (a.V + kTile - 1) / kTile;
    for (int64_t l0 = 0; l0 < a.lanes; l0 += kGridY) {
        const dim3 grid(tiles, (uint32_t)(a.lanes - l0 < kGridY ? a.lanes - l0 : kGridY));
        if (a.bias_ids)
            hipLaunchKernelGGL((adjust_sparse<DT, kRow, true>), grid, dim3(kBlock), 0, stream, a, (uint32_t)l0);
        else
            hipLaunchKernelGGL((adjust_sparse<DT, kRow, false>), grid, dim3(kBlock), 0, stream, a, (uint32_t)l0);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class DT>
hipError_t launch_dt(int layout, const AdjustArgs& a, hipStream_t stream) {
    const bool sparse = a.counts || a.drafts || a.bias_ids;
    const bool in_place = a.x == a.out;
    if (!in_place)
        if (const hipError_t e = launch_dense<DT, false>(layout, a, stream); e != hipSuccess) return e;
    if (sparse) {
        const hipError_t e = layout == TOPK_COL_CONTIG ? launch_sparse<DT, false>(a, stream) : launch_sparse<DT, true>(a, stream);
        if (e != hipSuccess) return e;
    }
    return in_place && a.mask ? launch_dense<DT, true>(layout, a, stream) : hipSuccess;
}

}  // namespace

hipError_t launch_adjust(int dtype, int layout, const AdjustArgs& a, hipStream_t stream) {
    return dtype == TOPK_BF16 ? launch_dt<Bf16>(layout, a, stream) : launch_dt<F32>(layout, a, stream);
}

}  // namespace topk
