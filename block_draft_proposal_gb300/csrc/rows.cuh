// Rows of fp32 or bf16 values in steps of 8 per thread, and E4M3 encoding: what the
// kernels of the cache, the norms, the block quantisation and the rotary positions share.
#pragma once

#include <float.h>

#include "kernels.h"

namespace dflash2 {

// 8 values as they are (rows that are only moved keep their bits, NaN payloads
// included), and as fp32.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T> __device__ __forceinline__ Raw8<T> load_raw8(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
// The same of memory that the kernel also writes (a call in place).
template <typename T> __device__ __forceinline__ Raw8<T> load_raw8_written(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
template <typename T> __device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
}
__device__ __forceinline__ void as_floats(const Raw8<float> &r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(r.w[i].x), x[4 * i + 1] = __uint_as_float(r.w[i].y);
        x[4 * i + 2] = __uint_as_float(r.w[i].z), x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
}
__device__ __forceinline__ void as_floats(const Raw8<__nv_bfloat16> &r, float (&x)[8]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The exponent of an E4M3 cache's row: the smallest e in [kKvMinExp, kKvMaxExp] with
// amax <= 448 * 2^e.  448 = 1.75 * 2^8, so e is amax's binade minus 8, one more when its
// significand exceeds 1.75.
__device__ __forceinline__ int row_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kKvMinExp), kKvMaxExp);
}
__device__ __forceinline__ uint8_t encode1(float x) {
    return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float decode1(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
    return __half2float(__half(h));
}
// The codes of x * s, nearest even, saturating at 448, NaN as NaN.
__device__ __forceinline__ uint32_t encode4(const float *x, float s) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * s, x[1] * s), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * s, x[3] * s), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s) {
    return make_uint2(encode4(x, s), encode4(x + 4, s));
}

// ---- E4M3 blocks: one fp32 scale per 128 values of a row ---------------------
constexpr int kQuantBlock = 128;
constexpr int kQuantLanes = kQuantBlock / 8;  // neighbouring lanes that hold a block
constexpr float kQuantFloor = 7.888609e-31f;  // 2^-100: below it 448 / amax would leave fp32

// The block's scale and codes from its 16 lanes' values (8 each, in order; values past
// the row's end as zeros).  amax is the largest finite magnitude; a block without one
// has scale 1.  Infinities, which E4M3 has no code for, become NaN codes like NaN: a
// product with them stays visible.  The divisions are IEEE and nothing is contracted, so
// the codes are fixed by the values.
__device__ __forceinline__ void block_scale(float amax, float *scale, float *inv) {
    const bool some = amax > 0.0f;
    amax = fmaxf(amax, kQuantFloor);
    *scale = some ? __fdiv_rn(amax, 448.0f) : 1.0f;
    *inv = some ? __fdiv_rn(448.0f, amax) : 0.0f;
}
__device__ __forceinline__ float finite_amax(float (&x)[8]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        if (a <= FLT_MAX)
            amax = fmaxf(amax, a);
        else
            x[i] = __uint_as_float(0x7FFFFFFFu);
    }
    return amax;
}
// One block of 16 lanes.
__device__ __forceinline__ uint2 quantise_block(float (&x)[8], float *scale) {
    float amax = 0.0f;  // fmaxf leaves NaN out
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    const auto fold = [&]() {
#pragma unroll
        for (int o = kQuantLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    };
    fold();
    if (__any_sync(0xFFFFFFFFu, amax > FLT_MAX)) {
        amax = finite_amax(x);
        fold();
    }
    float inv;
    block_scale(amax, scale, &inv);
    return encode8(x, inv);
}
// Four blocks of the same 16 lanes at a time: the lanes' maxima are folded so that a
// quarter of the lanes ends with each block's (5 shuffles in place of 16), and the
// divisions are made once for the four.  The lane's `scale` is that of block quant_lane().
constexpr int kQuantUnroll = 4;
__device__ __forceinline__ int quant_lane() { return (threadIdx.x >> 2) & 3; }
__device__ __forceinline__ void quantise_blocks(float (&x)[kQuantUnroll][8], float *scale, uint2 (&codes)[kQuantUnroll]) {
    float m[kQuantUnroll];
#pragma unroll
    for (int c = 0; c < kQuantUnroll; ++c) {
        m[c] = 0.0f;  // fmaxf leaves NaN out
#pragma unroll
        for (int i = 0; i < 8; ++i) m[c] = fmaxf(m[c], fabsf(x[c][i]));
    }
    const auto fold = [&]() {
        const bool h8 = threadIdx.x & 8, h4 = threadIdx.x & 4;
        const float s0 = __shfl_xor_sync(0xFFFFFFFFu, h8 ? m[0] : m[2], 8);
        const float s1 = __shfl_xor_sync(0xFFFFFFFFu, h8 ? m[1] : m[3], 8);
        const float a0 = fmaxf(h8 ? m[2] : m[0], s0), a1 = fmaxf(h8 ? m[3] : m[1], s1);
        float k = fmaxf(h4 ? a1 : a0, __shfl_xor_sync(0xFFFFFFFFu, h4 ? a0 : a1, 4));
        k = fmaxf(k, __shfl_xor_sync(0xFFFFFFFFu, k, 2));
        return fmaxf(k, __shfl_xor_sync(0xFFFFFFFFu, k, 1));
    };
    float amax = fold();
    if (__any_sync(0xFFFFFFFFu, amax > FLT_MAX)) {
#pragma unroll
        for (int c = 0; c < kQuantUnroll; ++c) m[c] = finite_amax(x[c]);
        amax = fold();
    }
    float inv;
    block_scale(amax, scale, &inv);
#pragma unroll
    for (int c = 0; c < kQuantUnroll; ++c)
        codes[c] = encode8(x[c], __shfl_sync(0xFFFFFFFFu, inv, (threadIdx.x & 16) | (4 * c)));
}
// Stores 8 codes, n of them when the row ends (vec: 8-byte aligned and whole).
__device__ __forceinline__ void store_codes(uint8_t *p, int n, bool vec, uint2 c) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2 *>(p) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace dflash2
