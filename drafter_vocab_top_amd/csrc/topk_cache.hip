// The paged cache, for gfx950: keys and values written into their slots
// (quantised on the way), and an accepted path's moved together.
//
// Quantising: the row's largest finite magnitude a gives e, the smallest whole
// number with a <= 448 * 2^e, from a's exponent field and the comparison of
// its fraction with that of 448 = 1.75 * 2^8; x * 2^-e is exact, the conversion
// to e4m3 rounds once.
#include "topk_cache.hpp"

namespace topk {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight elements as binary32.
template <class DT>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
    if constexpr (DT::kPerVec == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v[i];
            x[2 * i] = __builtin_bit_cast(float, w << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
        }
    } else {
        const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint32_t*>(base) + at);
        const u32x4 v0 = p[0], v1 = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w0 = v0[i], w1 = v1[i];
            x[i] = __builtin_bit_cast(float, w0);
            x[4 + i] = __builtin_bit_cast(float, w1);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_of(float x) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

// Eight elements of a key and of its value for each thread, kGroup threads (a
// power of two) for each row; the row's last threads have none where dim / 8 is
// no power of two.  Memory bounds long calls: 98,304 rows of 128 bfloat16
// elements into an e4m3 cache are 76 MB in 18 us (with keys and values in
// threads of their own 22; two rows for each thread 18), short ones the chain
// slot, row, store: 384 rows 3 us.
template <class DT, bool kFp8, int kGroup>
__global__ __launch_bounds__(256) void write_kernel(CacheWriteArgs a) {
    const topk_cache& c = a.cache.c;
    const uint32_t part = threadIdx.x % kGroup;
    const uint32_t row = blockIdx.x * (256u / kGroup) + threadIdx.x / kGroup, rows = (uint32_t)(a.w.C * c.heads);
    const uint32_t col = row < rows ? row / (uint32_t)c.heads : 0u, head = row < rows ? row % (uint32_t)c.heads : 0u;
    const int64_t slot = a.w.slots[col];
    const bool live = row < rows && (int32_t)(part * 8u) < c.dim && slot >= 0 && slot < c.blocks * c.block_size;
    float x[2][8] = {};
    if (live) {
        load8<DT>(a.w.keys, (int64_t)col * a.w.key_stride + (int64_t)head * a.w.key_head_stride + part * 8u, x[0]);
        load8<DT>(a.w.values, (int64_t)col * a.w.value_stride + (int64_t)head * a.w.value_head_stride + part * 8u, x[1]);
    }
    const uint32_t block = a.cache.block.div(live ? (uint32_t)slot : 0u), in_block = (live ? (uint32_t)slot : 0u) - block * a.cache.block.d;
    const uint32_t row16 = a.cache.row16(block, in_block);
    const int64_t at = (int64_t)head * c.head_stride + part * 8u;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        void* to = past16(n ? c.values : c.keys, row16);
        if constexpr (!kFp8) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = bf16_of(x[n][2 * i]) | (bf16_of(x[n][2 * i + 1]) << 16);
            if (live) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(to) + at) = v;
        } else {
            uint32_t largest = 0;  // of the finite magnitudes, as patterns
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = __builtin_bit_cast(uint32_t, x[n][i]) & 0x7FFFFFFFu;
                if (m < 0x7F800000u) largest = max_u32(largest, m);
            }
#pragma unroll
            for (int s = 1; s < kGroup; s <<= 1) largest = max_u32(largest, (uint32_t)__shfl_xor((int)largest, s));
            const int32_t e = max_i32((int32_t)(largest >> 23) - 135 + ((largest & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
            u32x2 v = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float y[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    y[k] = __builtin_isfinite(x[n][i + k]) ? __builtin_ldexpf(x[n][i + k], -e) : __builtin_nanf("");
                if (i % 4 == 0) v[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], (int)v[i / 4], false);
                else v[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], (int)v[i / 4], true);
            }
            if (live) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(to) + at) = v;
            if (live && part == 0)
                (n ? c.value_scales : c.key_scales)[a.cache.scale_row(block, in_block) + (int64_t)head * c.scale_head_stride] =
                    (uint8_t)(e + 127);
        }
    }
}

template <class DT, bool kFp8, int kGroup>
hipError_t write_grid(const CacheWriteArgs& a, hipStream_t stream) {
    const int64_t rows = a.w.C * a.cache.c.heads;
    const dim3 grid((uint32_t)((rows + 256 / kGroup - 1) / (256 / kGroup)));
    hipLaunchKernelGGL((write_kernel<DT, kFp8, kGroup>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <class DT, bool kFp8>
hipError_t write_dim(const CacheWriteArgs& a, hipStream_t stream) {
    const int32_t threads = a.cache.c.dim / 8;
    if (threads <= 8) return write_grid<DT, kFp8, 8>(a, stream);
    if (threads <= 16) return write_grid<DT, kFp8, 16>(a, stream);
    return write_grid<DT, kFp8, 32>(a, stream);
}

// One thread for 16 bytes of a row (of every slot that moves), or one scale.  A
// workgroup first lists the moves of its lane: threads look up one entry of the
// path each, so the reads that hang on each other (path, table) are made once
// and not once for every few rows.  Then a thread reads kAhead places before it
// writes the first of them: place i comes from a later one, and what a batch
// reads lies behind all that was written before it.  64 lanes' paths of 13 in 32
// layers of 4 heads of 128 (54 MB): 14.7 us, 3.7 TB/s (kAhead 2: 15.7); one lane's
// 3.4 (kAhead 16: 3.8).
template <bool kFp8>
__global__ __launch_bounds__(256) void move_kernel(CacheMoveArgs a, uint32_t row_vectors, uint32_t vectors, uint32_t scales, uint32_t first_lane) {
    constexpr uint32_t kAhead = 8;
    __shared__ uint32_t from16[256], to16[256], scale_from[256], scale_to[256], counts[4];
    const topk_cache& c = a.cache.c;
    constexpr int32_t size = kFp8 ? 1 : 2;
    const uint32_t tid = threadIdx.x, wave = tid >> 6, t = blockIdx.x * 256u + tid;
    const uint32_t l = first_lane + blockIdx.y;
    const bool vector = t < vectors, scale = kFp8 && !vector && t - vectors < scales;
    // layer, keys or values, head and vector of the head's row
    const uint32_t item = vector ? t / row_vectors : scale ? t - vectors : 0u, part = vector ? t % row_vectors : 0u;
    const uint32_t head = item % (uint32_t)c.heads, both = item / (uint32_t)c.heads;
    const int64_t layer = both >> 1;
    const bool values = both & 1u;
    uint8_t* base = scale ? (values ? c.value_scales : c.key_scales) + layer * c.scale_layer_stride + (int64_t)head * c.scale_head_stride
                          : static_cast<uint8_t*>(values ? c.values : c.keys) + (layer * c.layer_stride + (int64_t)head * c.head_stride) * size + part * 16u;
    const int64_t len = max_i32(a.lens[l], 0), places = min(a.table_ld * c.block_size, (int64_t)0x7FFFFFFF);
    const int32_t* table = a.table + (int64_t)l * a.table_ld;
    const int32_t* columns = a.columns + (int64_t)l * a.width;
    for (uint32_t first = 0; first < a.width; first += 256u) {
        const uint32_t i = first + tid;
        const int32_t from = i < a.width ? columns[i] : -1;
        const int64_t src = len + from, dst = len + i;
        bool moves = from > (int32_t)i && src < places;
        uint32_t sb = 0, db = 0;
        int32_t s = -1, d = -1;
        if (moves) {
            sb = a.cache.block.div((uint32_t)src);
            db = a.cache.block.div((uint32_t)dst);
            s = table[sb];
            d = table[db];
        }
        moves = moves && s >= 0 && s < c.blocks && d >= 0 && d < c.blocks;
        const unsigned long long mask = __ballot(moves);
        if (first) __syncthreads();  // (the list before is done with)
        if ((tid & 63u) == 0) counts[wave] = (uint32_t)__builtin_popcountll(mask);
        __syncthreads();
        uint32_t at = lanes_below(mask), n = 0;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            at += k < wave ? counts[k] : 0u;
            n += counts[k];
        }
        if (moves) {
            const uint32_t sr = (uint32_t)src - sb * a.cache.block.d, dr = (uint32_t)dst - db * a.cache.block.d;
            from16[at] = a.cache.row16((uint32_t)s, sr);
            to16[at] = a.cache.row16((uint32_t)d, dr);
            if constexpr (kFp8) {
                scale_from[at] = a.cache.scale_row((uint32_t)s, sr);
                scale_to[at] = a.cache.scale_row((uint32_t)d, dr);
            }
        }
        __syncthreads();
        if (vector) {
            for (uint32_t k = 0; k < n; k += kAhead) {
                u32x4 v[kAhead];
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u) v[u] = *reinterpret_cast<const u32x4*>(past16(base, from16[min_u32(k + u, n - 1u)]));
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u)
                    if (k + u < n) *reinterpret_cast<u32x4*>(past16(base, to16[k + u])) = v[u];
            }
        } else if (scale) {
            for (uint32_t k = 0; k < n; k += kAhead) {
                uint8_t v[kAhead];
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u) v[u] = base[scale_from[min_u32(k + u, n - 1u)]];
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u)
                    if (k + u < n) base[scale_to[k + u]] = v[u];
            }
        }
    }
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t stream) {
    const bool fp8 = a.cache.c.format == TOPK_CACHE_FP8;
    if (a.w.dtype == TOPK_BF16) return fp8 ? write_dim<Bf16, true>(a, stream) : write_dim<Bf16, false>(a, stream);
    return fp8 ? write_dim<F32, true>(a, stream) : write_dim<F32, false>(a, stream);
}

hipError_t launch_cache_move(const CacheMoveArgs& a, hipStream_t stream) {
    const topk_cache& c = a.cache.c;
    const bool fp8 = c.format == TOPK_CACHE_FP8;
    const uint32_t row_vectors = (uint32_t)c.dim * (fp8 ? 1u : 2u) / 16u;
    const int64_t items = 2 * c.layers * c.heads, vectors = items * row_vectors, scales = fp8 ? items : 0;
    for (int64_t l = 0; l < a.lanes; l += kGridY) {
        const dim3 grid((uint32_t)((vectors + scales + 255) / 256), (uint32_t)(a.lanes - l < kGridY ? a.lanes - l : kGridY));
        if (fp8)
            hipLaunchKernelGGL(move_kernel<true>, grid, dim3(256), 0, stream, a, row_vectors, (uint32_t)vectors, (uint32_t)scales, (uint32_t)l);
        else
            hipLaunchKernelGGL(move_kernel<false>, grid, dim3(256), 0, stream, a, row_vectors, (uint32_t)vectors, 0u, (uint32_t)l);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace topk
