// Attention of a round's columns over the paged cache, for gfx950.
//
//   out = sum_p w_p v_p / sum_p w_p,  w_p = exp(s_p - m),  s_p = scale (q . k_p)
//
// One wave per column and query head: 64 places at a time, a lane for each
// place's score, then a lane for each element of the weighted sum; the running
// maximum m, the sum of the weights and the output are rescaled when m grows.
#include "topk_cache.hpp"

namespace topk {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x = __builtin_fmaxf(x, __shfl_xor(x, s));
    return x;
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
    return x;
}

__device__ __forceinline__ float scale_of(uint8_t b) { return __builtin_ldexpf(1.0f, (int)b - 127); }

__device__ __forceinline__ float bf16_value(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

template <bool kFp8>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs args) {
    __shared__ float qs[4][TOPK_MAX_DIM];
    const topk_attend_args& a = args.a;
    const topk_cache& c = args.cache.c;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t h = blockIdx.x;  // query head
    const uint32_t kh = h / (uint32_t)(a.heads / c.heads);
    for (int64_t l = blockIdx.y; l < a.lanes; l += gridDim.y) {
        uint32_t cb, ce;
        args.cols.range((uint32_t)l, cb, ce);
        const uint32_t n = ce - cb;
        const uint32_t len = (uint32_t)max_i32(a.lens[l], 0);
        const uint32_t end = (uint32_t)min((uint64_t)len + n, (uint64_t)args.places);
        const int32_t* table = a.table + l * a.table_ld;
        for (uint32_t j0 = 0; j0 < n; j0 += 4u) {
            const uint32_t j = j0 + wave;
            const int64_t col = (int64_t)cb + min_u32(j, n - 1u);
            __syncthreads();
            for (uint32_t d = lane; d < (uint32_t)c.dim; d += 64u)
                qs[wave][d] = bf16_value(static_cast<const uint16_t*>(a.q)[col * a.q_stride + (int64_t)h * a.q_head_stride + d]);
            __syncthreads();
            if (j >= n) continue;
            int64_t lo = 0;  // the first visible place before len
            if (a.window) lo = (a.positions ? max((int64_t)a.positions[col], (int64_t)len) : (int64_t)len + j) - a.window + 1;
            float m = -__builtin_inff(), sum = 0.0f, o[4] = {};
            for (uint32_t p0 = (uint32_t)min(max(lo, (int64_t)0), (int64_t)len) & ~63u; p0 < end; p0 += 64u) {
                const uint32_t p = min_u32(p0 + lane, end - 1u);
                bool seen = p0 + lane < end;
                if (p < len) {
                    seen = seen && (int64_t)p >= lo;
                } else {
                    const uint32_t i = p - len;
                    if (a.mask) seen = seen && (int64_t)(i >> 5) < a.mask_ld && (a.mask[col * a.mask_ld + (i >> 5)] >> (i & 31u) & 1u);
                    else seen = seen && i <= j && (!a.window || j - i < (uint32_t)a.window);
                }
                const uint32_t b = args.cache.block.div(p);
                const int32_t id = min_i32(max_i32(table[b], 0), (int32_t)c.blocks - 1);
                const uint32_t r = p - b * args.cache.block.d;
                const int64_t at = (int64_t)id * c.block_stride + (int64_t)r * c.slot_stride + (int64_t)kh * c.head_stride;
                const int64_t sat = (int64_t)id * c.scale_block_stride + (int64_t)r * c.scale_slot_stride + (int64_t)kh * c.scale_head_stride;
                float s = 0.0f;
                for (int32_t d = 0; d < c.dim; ++d) {
                    float k;
                    if constexpr (kFp8)
                        k = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(c.keys)[at + d], 0);
                    else
                        k = bf16_value(static_cast<const uint16_t*>(c.keys)[at + d]);
                    s += qs[wave][d] * k;
                }
                if constexpr (kFp8) s *= scale_of(c.key_scales[sat]);
                s = seen ? s * (a.scale * kLog2e) : -__builtin_inff();
                const float top = __builtin_fmaxf(m, wave_max(s));
                const float zero = top == -__builtin_inff() ? 0.0f : top;
                const float old = __builtin_amdgcn_exp2f(m - zero);
                float w = __builtin_amdgcn_exp2f(s - zero);
                m = top;
                sum = sum * old + wave_sum(w);
                w = (float)(__bf16)w;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] *= old;
                const unsigned long long visible = __ballot(seen);
                for (int k = 0; k < 64; ++k) {
                    if (!(visible >> k & 1ull)) continue;
                    const float wk = __shfl(w, k);
                    const int64_t ak = __shfl(at, k);
                    float f = 1.0f;
                    if constexpr (kFp8) f = scale_of(c.value_scales[__shfl(sat, k)]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t d = (int32_t)lane + 64 * i;
                        if (d >= c.dim) continue;
                        if constexpr (kFp8) o[i] += wk * (f * __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(c.values)[ak + d], 0));
                        else o[i] += wk * bf16_value(static_cast<const uint16_t*>(c.values)[ak + d]);
                    }
                }
            }
            __bf16* to = static_cast<__bf16*>(a.out) + col * a.out_stride + (int64_t)h * a.out_head_stride;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t d = (int32_t)lane + 64 * i;
                if (d < c.dim) to[d] = (__bf16)(m == -__builtin_inff() ? 0.0f : o[i] / sum);
            }
        }
    }
}

}  // namespace

int64_t attend_workspace(const AttendArgs&) { return 0; }

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.a.heads, (uint32_t)(a.a.lanes < kGridY ? a.a.lanes : kGridY));
    if (a.cache.c.format == TOPK_CACHE_FP8) hipLaunchKernelGGL(attend_kernel<true>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(attend_kernel<false>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace topk
