// Paged key/value cache: write (with E4M3 quantisation) and read back.
//
// A row is one (token, keys or values, head): head_dim values.  Rows are
// numbered (token * 2 + which) * kv_heads + head, so neighbouring rows are
// neighbours in the packed tensor and the cache's 64 .. 512 byte rows are the
// scattered side.  Both operators move each byte once and compute next to
// nothing; HBM bounds them once the rows fill the GPU, a launch below that.
//
// Fast path (head_dim 64, 128 or 256): kLanes = head_dim / 8 lanes hold a row,
// 8 values each, and every lane group takes kUnroll rows at once so that a
// thread has that many 16-byte loads in flight.  The row's largest magnitude is a
// shuffle over those lanes.
#include "kernels.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -48, kMaxExp = 48;

struct KvArgs {
    const void *k, *v;  // packed rows (write: input; read: unused)
    void *ko, *vo;      // packed rows (read: output)
    int64_t k_stride, v_stride;
    const int64_t *slots;
    int32_t n_rows;  // 2 * n_tokens * kv_heads
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
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
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

// The smallest e in [kMinExp, kMaxExp] with amax <= 448 * 2^e: 448 = 1.75 * 2^8,
// so e is amax's binade minus 8, one more when its significand exceeds 1.75.
__device__ __forceinline__ int row_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kMinExp), kMaxExp);
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
// `first` is the one lane of the row that reports a bad slot.
__device__ __forceinline__ Row find_row(const KvArgs &a, int32_t r, bool first) {
    Row o;
    const uint32_t th = (uint32_t)r / (uint32_t)a.kv_heads;
    o.head = r - (int32_t)(th * (uint32_t)a.kv_heads);
    o.values = th & 1u;
    o.token = th >> 1;
    const int64_t slot = __ldg(a.slots + o.token);
    o.at = -1;
    if (slot >= a.n_slots) {
        if (first && a.err) atomicOr(a.err, DFLASH2_DEVERR_ID_RANGE);
    } else if (slot >= 0) {
        int64_t page, off;
        if (a.n_slots <= 0xFFFFFFFFll) {  // 32-bit division when the slots allow it
            page = (uint32_t)slot / (uint32_t)a.page_size;
            off = (uint32_t)slot - (uint32_t)page * (uint32_t)a.page_size;
        } else {
            page = slot / a.page_size;
            off = slot - page * a.page_size;
        }
        o.at = (page * a.kv_heads + o.head) * a.page_size + off;
    }
    return o;
}

template <typename T, bool kE4M3, int kLanes, int kUnroll>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvArgs a) {
    constexpr int kDim = kLanes * 8;
    grid_dep_wait();
    const int lane = threadIdx.x % kLanes;
    const int32_t groups = kThreads / kLanes;
    const int64_t r0 = (int64_t)blockIdx.x * groups * kUnroll + threadIdx.x / kLanes;
    Row row[kUnroll];
    float x[kUnroll][8];
    Raw8<T> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = r0 + u * groups;
        row[u].at = -1;
        if (r >= a.n_rows) continue;
        row[u] = find_row(a, (int32_t)r, lane == 0);
        if (row[u].at < 0) continue;
        const T *src = row[u].values ? (const T *)a.v + row[u].token * a.v_stride
                                     : (const T *)a.k + row[u].token * a.k_stride;
        src += (int64_t)row[u].head * kDim + lane * 8;
        if constexpr (kE4M3)
            load8(src, x[u]);
        else
            raw[u] = load_raw8(src);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if constexpr (!kE4M3) {
            if (row[u].at >= 0)
                store_raw8((T *)(row[u].values ? a.vc : a.kc) + row[u].at * kDim + lane * 8, raw[u]);
        } else {
            float amax = 0.0f;
            if (row[u].at >= 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[u][i]));
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            if (row[u].at >= 0) {
                const int e = row_exponent(amax);
                const float s = pow2i(-e);
                uint32_t w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float *y = x[u] + 4 * i;
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * s, y[1] * s),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * s, y[3] * s),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    w[i] = lo | (hi << 16);
                }
                uint8_t *dst = (uint8_t *)(row[u].values ? a.vc : a.kc) + row[u].at * kDim + lane * 8;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
                if (lane == 0) (row[u].values ? a.ve : a.ke)[row[u].at] = (uint8_t)(e + 127);
            }
        }
    }
}

template <typename T, bool kE4M3, int kLanes, int kUnroll>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a) {
    constexpr int kDim = kLanes * 8;
    grid_dep_wait();
    const int lane = threadIdx.x % kLanes;
    const int32_t groups = kThreads / kLanes;
    const int64_t r0 = (int64_t)blockIdx.x * groups * kUnroll + threadIdx.x / kLanes;
    Row row[kUnroll];
    Raw8<T> raw[kUnroll];
    uint2 c[kUnroll];
    int e[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = r0 + u * groups;
        raw[u] = Raw8<T>{};
        c[u] = make_uint2(0u, 0u);
        e[u] = 0;
        row[u].token = -1;
        if (r >= a.n_rows) continue;
        row[u] = find_row(a, (int32_t)r, lane == 0);
        if (row[u].at < 0) continue;
        const void *src = row[u].values ? a.vc : a.kc;
        if constexpr (kE4M3) {
            c[u] = __ldg(reinterpret_cast<const uint2 *>((const uint8_t *)src + row[u].at * kDim) + lane);
            e[u] = (int)__ldg((row[u].values ? a.ve : a.ke) + row[u].at) - 127;
        } else {
            raw[u] = load_raw8((const T *)src + row[u].at * kDim + lane * 8);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (row[u].token < 0) continue;
        T *dst = (row[u].values ? (T *)a.vo : (T *)a.ko) +
                 (row[u].token * a.kv_heads + row[u].head) * kDim + lane * 8;
        if constexpr (kE4M3) {
            float x[8];
            const float s = ldexpf(1.0f, e[u]);
            const uint32_t w[2] = {c[u].x, c[u].y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                x[2 * i] = f.x * s;
                x[2 * i + 1] = f.y * s;
            }
            store8(dst, x);
        } else {
            store_raw8(dst, raw[u]);
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
                    ldexpf(1.0f, (int)(row.values ? a.ve : a.ke)[row.at] - 127);
            from_f32(dst + j, x);
        } else {
            dst[j] = row.at >= 0 ? ((const T *)(row.values ? a.vc : a.kc))[row.at * d + j] : T(0.0f);
        }
    }
}

// Rows per lane group: four once the rows fill every SM several times over
// (measured at 100003 tokens x 8 heads), one below that, where more CTAs in
// flight answer sooner (measured at 512 tokens x 8 heads).
constexpr int kManyRows = 152 * 8 * (kThreads / 16) * 4;

template <typename T, bool kE4M3, bool kWrite, int kLanes>
dflash2_status launch_lanes(const KvArgs &a, cudaStream_t st) {
    const int groups = kThreads / kLanes;
    const int per = a.n_rows >= kManyRows ? 4 : 1;
    const unsigned grid = (unsigned)(((int64_t)a.n_rows + groups * per - 1) / (groups * per));
    void (*fn)(const KvArgs);
    if constexpr (kWrite)
        fn = per == 4 ? kv_write_kernel<T, kE4M3, kLanes, 4> : kv_write_kernel<T, kE4M3, kLanes, 1>;
    else
        fn = per == 4 ? kv_read_kernel<T, kE4M3, kLanes, 4> : kv_read_kernel<T, kE4M3, kLanes, 1>;
    launch_k(fn, dim3(grid), dim3(kThreads), 0, st, a);
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
