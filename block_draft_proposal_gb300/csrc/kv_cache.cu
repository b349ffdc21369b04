// Paged key/value cache: write (with E4M3 quantisation) and read back.
//
// Both operators move each byte once and compute next to nothing; HBM bounds them
// once the rows fill the GPU, a launch below that.
//
// Fast path (head_dim 64, 128 or 256): a warp takes the keys or the values of one
// token, so the slot is read and split into page and offset once for all heads;
// kLanes = head_dim / 8 lanes hold a row, 8 values each, and a thread has four
// rows' loads in flight.  The row's largest magnitude is a shuffle over its lanes.
// (A warp per two rows of any token, with its divisions for every row, was bound by
// instructions: 51 us for 20011 tokens x 8 heads written as E4M3, 165 us for 100003
// tokens read.)  A write's first rows are loaded beside its slot (24 us, 29 before).
// Measured, 8 heads of 128, bf16 rows and an E4M3 cache: 20011 tokens written and read back
// in 40 us, 6.1 TB/s; 100003 tokens read in 92 us, 6.7 TB/s; 512 tokens written to a bf16
// cache in 9 us, the call.
#include "kernels.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 256;

struct KvArgs {
    const void *k, *v;  // packed rows (write: input; read: unused)
    void *ko, *vo;      // packed rows (read: output)
    int64_t k_stride, v_stride;
    const int64_t *slots;
    int32_t n_tokens, n_rows;  // n_rows = 2 * n_tokens * kv_heads
    int32_t kv_heads, head_dim, page_size;
    int64_t n_slots;
    void *kc, *vc;
    uint8_t *ke, *ve;
    int32_t *err;
};

// 8 values as they are (a native cache copies rows bit for bit, NaN payloads
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

// The smallest e in [kKvMinExp, kKvMaxExp] with amax <= 448 * 2^e: 448 = 1.75 * 2^8,
// so e is amax's binade minus 8, one more when its significand exceeds 1.75.
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

struct Row {
    int64_t token;
    int64_t at;  // row of the cache arrays, or -1 (skip / zero)
    int head;
    bool values;
};
// Row of head 0 of a token in the cache arrays, or -1; the rows of the next heads
// follow at page_size.  `first` is the one lane that reports a bad slot.
__device__ __forceinline__ int64_t find_token(const KvArgs &a, int64_t token, bool first) {
    const int64_t slot = __ldg(a.slots + token);
    if (slot >= a.n_slots) {
        if (first && a.err) atomicOr(a.err, DFLASH2_DEVERR_ID_RANGE);
        return -1;
    }
    if (slot < 0) return -1;
    int64_t page, off;
    if (a.n_slots <= 0xFFFFFFFFll) {  // 32-bit division when the slots allow it
        page = (uint32_t)slot / (uint32_t)a.page_size;
        off = (uint32_t)slot - (uint32_t)page * (uint32_t)a.page_size;
    } else {
        page = slot / a.page_size;
        off = slot - page * a.page_size;
    }
    return page * a.kv_heads * a.page_size + off;
}
__device__ __forceinline__ Row find_row(const KvArgs &a, int32_t r, bool first) {
    Row o;
    const uint32_t th = (uint32_t)r / (uint32_t)a.kv_heads;
    o.head = r - (int32_t)(th * (uint32_t)a.kv_heads);
    o.values = th & 1u;
    o.token = th >> 1;
    const int64_t at = find_token(a, o.token, first);
    o.at = at < 0 ? -1 : at + (int64_t)o.head * a.page_size;
    return o;
}

constexpr int kUnroll = 4;

template <typename T, bool kE4M3, int kLanes>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvArgs a) {
    constexpr int kDim = kLanes * 8, kRows = 32 / kLanes;  // rows a warp holds at once
    grid_dep_wait();
    const int lane = threadIdx.x % kLanes, sub = (threadIdx.x & 31) / kLanes;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = w >> 1;
    if (token >= a.n_tokens) return;
    const bool values = w & 1;
    int64_t at = -1;
    const T *src = (values ? (const T *)a.v + token * a.v_stride : (const T *)a.k + token * a.k_stride) + lane * 8;
    void *cache = values ? a.vc : a.kc;
    uint8_t *exps = values ? a.ve : a.ke;
    for (int h0 = sub; h0 - sub < a.kv_heads; h0 += kRows * kUnroll) {
        Raw8<T> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            raw[u] = Raw8<T>{};
            if (h0 + u * kRows < a.kv_heads) raw[u] = load_raw8(src + (int64_t)(h0 + u * kRows) * kDim);
        }
        if (h0 == sub) {  // the slot, beside the first rows
            at = find_token(a, token, (threadIdx.x & 31) == 0 && !values);
            if (at < 0) return;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kRows;
            const int64_t row = at + (int64_t)h * a.page_size;
            if constexpr (!kE4M3) {
                if (h < a.kv_heads) store_raw8((T *)cache + row * kDim + lane * 8, raw[u]);
            } else {
                float x[8], amax = 0.0f;
                as_floats(raw[u], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const int e = row_exponent(amax);
                const float s = pow2i(-e);
                uint32_t c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float *y = x + 4 * i;
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * s, y[1] * s),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * s, y[3] * s),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    c[i] = lo | (hi << 16);
                }
                if (h < a.kv_heads) {
                    *reinterpret_cast<uint2 *>((uint8_t *)cache + row * kDim + lane * 8) = make_uint2(c[0], c[1]);
                    if (lane == 0) exps[row] = (uint8_t)(e + 127);
                }
            }
        }
    }
}

template <typename T, bool kE4M3, int kLanes>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a) {
    constexpr int kDim = kLanes * 8, kRows = 32 / kLanes;
    grid_dep_wait();
    const int lane = threadIdx.x % kLanes, sub = (threadIdx.x & 31) / kLanes;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = w >> 1;
    if (token >= a.n_tokens) return;
    const bool values = w & 1;
    const int64_t at = find_token(a, token, (threadIdx.x & 31) == 0 && !values);
    const void *cache = values ? a.vc : a.kc;
    const uint8_t *exps = values ? a.ve : a.ke;
    T *dst = (T *)(values ? a.vo : a.ko) + token * a.kv_heads * kDim + lane * 8;
    for (int h0 = sub; h0 < a.kv_heads; h0 += kRows * kUnroll) {
        Raw8<T> raw[kUnroll];
        uint2 c[kUnroll];
        int e[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kRows;
            const int64_t row = at + (int64_t)h * a.page_size;
            raw[u] = Raw8<T>{};
            c[u] = make_uint2(0u, 0u);
            e[u] = 127;
            if (at < 0 || h >= a.kv_heads) continue;
            if constexpr (kE4M3) {
                c[u] = __ldg(reinterpret_cast<const uint2 *>((const uint8_t *)cache + row * kDim) + lane);
                e[u] = __ldg(exps + row);
            } else {
                raw[u] = load_raw8((const T *)cache + row * kDim + lane * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kRows;
            if (h >= a.kv_heads) continue;
            if constexpr (kE4M3) {
                float x[8];
                const float s = pow2i(kv_exponent((uint8_t)e[u]));
                const uint32_t b[2] = {c[u].x, c[u].y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(b[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(y));
                    x[2 * i] = f.x * s;
                    x[2 * i + 1] = f.y * s;
                }
                store8(dst + (int64_t)h * kDim, x);
            } else {
                store_raw8(dst + (int64_t)h * kDim, raw[u]);
            }
        }
    }
}

// Any head_dim up to 256 and any alignment: a warp per row, one value per lane
// and step.
template <typename T, bool kE4M3>
__global__ void __launch_bounds__(kThreads) kv_write_scalar(const KvArgs a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= a.n_rows) return;
    const Row row = find_row(a, (int32_t)r, lane == 0);
    if (row.at < 0) return;
    const int d = a.head_dim;
    const T *src = (row.values ? (const T *)a.v + row.token * a.v_stride
                               : (const T *)a.k + row.token * a.k_stride) +
                   (int64_t)row.head * d;
    if constexpr (!kE4M3) {
        T *dst = (T *)(row.values ? a.vc : a.kc) + row.at * d;
        for (int j = lane; j < d; j += 32) dst[j] = src[j];
    } else {
        float amax = 0.0f;
        for (int j = lane; j < d; j += 32) amax = fmaxf(amax, fabsf(to_f32(src[j])));
        amax = warp_max(amax);
        const int e = row_exponent(amax);
        const float s = pow2i(-e);
        uint8_t *dst = (uint8_t *)(row.values ? a.vc : a.kc) + row.at * d;
        for (int j = lane; j < d; j += 32) dst[j] = encode1(to_f32(src[j]) * s);
        if (lane == 0) (row.values ? a.ve : a.ke)[row.at] = (uint8_t)(e + 127);
    }
}

template <typename T, bool kE4M3>
__global__ void __launch_bounds__(kThreads) kv_read_scalar(const KvArgs a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= a.n_rows) return;
    const Row row = find_row(a, (int32_t)r, lane == 0);
    const int d = a.head_dim;
    T *dst = (row.values ? (T *)a.vo : (T *)a.ko) + (row.token * a.kv_heads + row.head) * d;
    for (int j = lane; j < d; j += 32) {
        if constexpr (kE4M3) {
            float x = 0.0f;
            if (row.at >= 0)
                x = decode1(((const uint8_t *)(row.values ? a.vc : a.kc))[row.at * d + j]) *
                    pow2i(kv_exponent((row.values ? a.ve : a.ke)[row.at]));
            from_f32(dst + j, x);
        } else {
            dst[j] = row.at >= 0 ? ((const T *)(row.values ? a.vc : a.kc))[row.at * d + j] : T(0.0f);
        }
    }
}

template <typename T, bool kE4M3, bool kWrite, int kLanes>
dflash2_status launch_lanes(const KvArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((2ll * a.n_tokens + kThreads / 32 - 1) / (kThreads / 32));
    if constexpr (kWrite)
        launch_k(kv_write_kernel<T, kE4M3, kLanes>, dim3(grid), dim3(kThreads), 0, st, a);
    else
        launch_k(kv_read_kernel<T, kE4M3, kLanes>, dim3(grid), dim3(kThreads), 0, st, a);
    return launch_status();
}

template <typename T, bool kE4M3, bool kWrite>
dflash2_status launch_kv(const KvArgs &a, bool aligned, cudaStream_t st) {
    if (aligned && a.head_dim == 64) return launch_lanes<T, kE4M3, kWrite, 8>(a, st);
    if (aligned && a.head_dim == 128) return launch_lanes<T, kE4M3, kWrite, 16>(a, st);
    if (aligned && a.head_dim == 256) return launch_lanes<T, kE4M3, kWrite, 32>(a, st);
    const unsigned grid = (unsigned)(((int64_t)a.n_rows + kThreads / 32 - 1) / (kThreads / 32));
    if constexpr (kWrite)
        launch_k(kv_write_scalar<T, kE4M3>, dim3(grid), dim3(kThreads), 0, st, a);
    else
        launch_k(kv_read_scalar<T, kE4M3>, dim3(grid), dim3(kThreads), 0, st, a);
    return launch_status();
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks both entry points share; fills what is common.
dflash2_status check_kv(KvArgs *a, const int64_t *slots, int64_t n_tokens, int32_t kv_heads,
                        int32_t head_dim, int32_t page_size, int64_t num_pages, int32_t dtype,
                        int32_t kv_format) {
    if (dtype != DFLASH2_F32 && dtype != DFLASH2_BF16) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (kv_format != DFLASH2_KV_NATIVE && kv_format != DFLASH2_KV_E4M3)
        return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (head_dim < 1 || head_dim > 256 || kv_heads < 1 || page_size < 1 || num_pages < 0 ||
        n_tokens < 0 || num_pages > (INT64_MAX >> 9) / page_size / kv_heads ||
        n_tokens >= (1ll << 30) / kv_heads + ((1ll << 30) % kv_heads ? 1 : 0))
        return DFLASH2_ERR_INVALID_ARG;
    a->slots = slots;
    a->n_tokens = (int32_t)n_tokens;
    a->n_rows = (int32_t)(2 * n_tokens * kv_heads);
    a->kv_heads = kv_heads;
    a->head_dim = head_dim;
    a->page_size = page_size;
    a->n_slots = num_pages * page_size;
    return DFLASH2_OK;
}

template <bool kWrite>
dflash2_status dispatch_kv(const KvArgs &a, bool aligned, int32_t dtype, int32_t kv_format,
                           cudaStream_t st) {
    if (dtype == DFLASH2_F32)
        return kv_format == DFLASH2_KV_E4M3 ? launch_kv<float, true, kWrite>(a, aligned, st)
                                            : launch_kv<float, false, kWrite>(a, aligned, st);
    return kv_format == DFLASH2_KV_E4M3 ? launch_kv<__nv_bfloat16, true, kWrite>(a, aligned, st)
                                        : launch_kv<__nv_bfloat16, false, kWrite>(a, aligned, st);
}

}  // namespace
}  // namespace dflash2

using namespace dflash2;

extern "C" dflash2_status dflash2_kv_cache_write(
    const void *k, const void *v, int64_t k_row_stride, int64_t v_row_stride, const int64_t *slots,
    int64_t n_tokens, int32_t kv_heads, int32_t head_dim, int32_t page_size, int64_t num_pages,
    int32_t dtype, int32_t kv_format, void *k_cache, void *v_cache, uint8_t *k_exp, uint8_t *v_exp,
    int32_t *err_word, void *stream) {
    KvArgs a{};
    dflash2_status st = check_kv(&a, slots, n_tokens, kv_heads, head_dim, page_size, num_pages,
                                 dtype, kv_format);
    if (st != DFLASH2_OK) return st;
    const int64_t width = (int64_t)kv_heads * head_dim;
    if (k_row_stride < width || v_row_stride < width) return DFLASH2_ERR_INVALID_ARG;
    if (n_tokens == 0) return DFLASH2_OK;
    const bool q8 = kv_format == DFLASH2_KV_E4M3;
    if (!k || !v || !slots || !k_cache || !v_cache || (q8 && (!k_exp || !v_exp)))
        return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == DFLASH2_F32 ? 4 : 2;
    if (!aligned_to(k, el) || !aligned_to(v, el) || !aligned_to(slots, 8) ||
        (!q8 && (!aligned_to(k_cache, el) || !aligned_to(v_cache, el))) ||
        (err_word && !aligned_to(err_word, 4)))
        return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    a.k = k, a.v = v, a.k_stride = k_row_stride, a.v_stride = v_row_stride;
    a.kc = k_cache, a.vc = v_cache, a.ke = k_exp, a.ve = v_exp, a.err = err_word;
    const uintptr_t held = q8 ? 8 : 16;
    const bool aligned = aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(k_cache, held) &&
                         aligned_to(v_cache, held) && k_row_stride * (int64_t)el % 16 == 0 &&
                         v_row_stride * (int64_t)el % 16 == 0;
    return dispatch_kv<true>(a, aligned, dtype, kv_format, static_cast<cudaStream_t>(stream));
}

extern "C" dflash2_status dflash2_kv_cache_read(
    const void *k_cache, const void *v_cache, const uint8_t *k_exp, const uint8_t *v_exp,
    const int64_t *slots, int64_t n_tokens, int32_t kv_heads, int32_t head_dim, int32_t page_size,
    int64_t num_pages, int32_t dtype, int32_t kv_format, void *k_out, void *v_out,
    int32_t *err_word, void *stream) {
    KvArgs a{};
    dflash2_status st = check_kv(&a, slots, n_tokens, kv_heads, head_dim, page_size, num_pages,
                                 dtype, kv_format);
    if (st != DFLASH2_OK) return st;
    if (n_tokens == 0) return DFLASH2_OK;
    const bool q8 = kv_format == DFLASH2_KV_E4M3;
    if (!k_out || !v_out || !slots || !k_cache || !v_cache || (q8 && (!k_exp || !v_exp)))
        return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == DFLASH2_F32 ? 4 : 2;
    if (!aligned_to(k_out, el) || !aligned_to(v_out, el) || !aligned_to(slots, 8) ||
        (!q8 && (!aligned_to(k_cache, el) || !aligned_to(v_cache, el))) ||
        (err_word && !aligned_to(err_word, 4)))
        return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    a.ko = k_out, a.vo = v_out;
    a.kc = const_cast<void *>(k_cache), a.vc = const_cast<void *>(v_cache);
    a.ke = const_cast<uint8_t *>(k_exp), a.ve = const_cast<uint8_t *>(v_exp);
    a.err = err_word;
    const uintptr_t held = q8 ? 8 : 16;
    const bool aligned = aligned_to(k_out, 16) && aligned_to(v_out, 16) &&
                         aligned_to(k_cache, held) && aligned_to(v_cache, held);
    return dispatch_kv<false>(a, aligned, dtype, kv_format, static_cast<cudaStream_t>(stream));
}
