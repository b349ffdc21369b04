// Rotary positions with several axes, of queries and keys, and the write of the rotated
// keys and the values into the paged cache.
//
//   angle(i, j) = positions[axis[j], i] * f[j]       token i, pair j of rotary_dim / 2
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
//   pairs (j, j + rotary_dim / 2), or adjacent (2j, 2j + 1); the rest of a row is copied
//
// Frequencies are 64-bit fractions of a turn, so position * frequency modulo 2^64 is the
// angle modulo a turn: exact for every 64-bit position, where an fp32 product has lost
// 0.06 rad at position 10^6, and one integer multiplication.
//
// Every value moves once: HBM bounds it, a launch where tokens are few.  A lane holds the
// same two steps of 8 values of every row, chosen so that both halves of its pairs are
// its own (for halves: step u and u + rotary_dim / 16; rows whose halves or addresses allow
// no 8 go in steps of 4), so its sines and cosines are read
// from shared memory once per token and the rows need no exchange between lanes but the
// E4M3 maximum.  A block computes its tokens' sines and cosines once and keeps several
// groups' loads in flight per warp (computed by every warp of a token, at 18 instructions a
// value, 20011 tokens x 56 rows took 172 us).
// Measured, heads of 128, bf16: 20011 tokens, 40 + 8 heads with the write into an E4M3 cache
// 90 us, 5.9 TB/s; 32 + 8 heads into a bf16 cache 84 us; 512 tokens 4.1 us; one 2.9 us.
// Steps of 4, 10000 tokens, 8 + 8 heads of 72 into a bf16 cache: 24 us, 2.9 TB/s (value by
// value 108).
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace dflash2 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;

struct RotaryArgs {
    const void *q, *k, *v;
    void *qo, *ko;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;
    const int64_t *positions;  // [axes, n_tokens]
    const uint64_t *freq;
    const uint8_t *axis;
    int32_t axes, pairs;       // pairs = rotary_dim / 2
    int32_t adjacent;
    float magnitude;
    int64_t n_tokens;
    int32_t q_rows, k_rows, v_rows;  // heads of each, 0 if absent
    int32_t head_dim, kv_heads, page_size;
    const int64_t *slots;      // NULL: no cache
    int64_t n_slots;
    void *kc, *vc;
    uint8_t *ke, *ve;
    int32_t parts;             // warps a token's rows are split over (a power of two; scalar: any)
    int32_t *err;
};

// Cosine and sine of phase / 2^64 turns, within 0.8 of a last place (0.5 of it the final
// rounding), also where one of them is next to 0.
// The nearest quarter turn leaves exactly; the rest x, at most pi / 4, is held in two
// floats (the fraction of a turn in one costs pi 2^-25 of angle, more than all other
// roundings), and the Taylor series' small terms are added to x and to 1 last.
// A rest of few bits, as slow pairs have at the first positions, is held in floats of its own
// size: in the fixed steps of the others its sine would be off by 0.9 of a last place at 2^38 and
// lost below 2^7.  (Floats of their own size for all: 20011 tokens 91.4 us for 89.7, 20000 with 5 rows
// each 23.1 for 21.5.)
__device__ __forceinline__ float2 turn_by(uint64_t phase) {
    const int64_t quarter = (((int64_t)phase >> 61) + 1) >> 1;
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // |rest| <= 2^61
    const int32_t high = (int32_t)((rest + (1ll << 37)) >> 38);          // 24 bits
    const int32_t low = (int32_t)((rest - ((int64_t)high << 38)) >> 7);  // and the next 30
    constexpr float kPi = 0x1.921fb6p-24f, kPiLow = -0x1.777a5cp-49f;    // pi / 2^25
    float hi = (float)high, lo = 0x1p-31f * (float)low;
    if (__builtin_expect(abs(high) < 8, 0)) {
        const float whole = __ll2float_rn(rest);
        hi = 0x1p-38f * whole, lo = 0x1p-38f * __ll2float_rn(rest - __float2ll_rz(whole));
    }
    const float x = __fmul_rn(hi, kPi);
    const float x_low = __fmaf_rn(lo, kPi, __fmaf_rn(hi, kPiLow, __fmaf_rn(hi, kPi, -x)));
    const float xx = __fmul_rn(x, x), xx_half = 0.5f * xx;
    const float xx_low = __fmaf_rn(x + x, x_low, __fmaf_rn(x, x, -xx));
    float s = __fmaf_rn(xx, 1.0f / 362880, -1.0f / 5040);
    s = __fmaf_rn(xx, __fmaf_rn(xx, s, 1.0f / 120), -1.0f / 6);
    s = __fadd_rn(x, __fmaf_rn(x, __fmul_rn(xx, s), __fmaf_rn(-xx_half, x_low, x_low)));
    float c = __fmaf_rn(xx, -1.0f / 3628800, 1.0f / 40320);
    c = __fmaf_rn(xx, __fmaf_rn(xx, c, -1.0f / 720), 1.0f / 24);
    c = __fmaf_rn(__fmul_rn(xx, xx), c, -0.5f * xx_low);
    const float one = __fsub_rn(1.0f, xx_half);  // and what its rounding lost
    c = __fadd_rn(one, __fadd_rn(__fsub_rn(__fsub_rn(1.0f, one), xx_half), c));
    const bool swap = quarter & 1;
    const float cosine = swap ? s : c, sine = swap ? c : s;
    return make_float2((quarter + 1) & 2 ? -cosine : cosine, quarter & 2 ? -sine : sine);
}

// Cosine and sine (times the magnitude) of a token's pair.
__device__ __forceinline__ float2 turn_of(const RotaryArgs &a, int64_t token, int pair) {
    const int axis = __ldg(a.axis + pair);
    uint64_t phase = 0;
    if (axis < a.axes)
        phase = (uint64_t)__ldg(a.positions + axis * a.n_tokens + token) * __ldg(a.freq + pair);
    else if (a.err)
        atomicOr(a.err, DFLASH2_DEVERR_ID_RANGE);
    const float2 x = turn_by(phase);
    return make_float2(x.x * a.magnitude, x.y * a.magnitude);
}

// Head 0's row of a token in the cache arrays, or -1.
__device__ __forceinline__ int64_t cache_row(const RotaryArgs &a, int64_t token, bool report) {
    if (!a.slots) return -1;
    const int64_t slot = __ldg(a.slots + token);
    if (slot >= a.n_slots) {
        if (report && a.err) atomicOr(a.err, DFLASH2_DEVERR_ID_RANGE);
        return -1;
    }
    if (slot < 0) return -1;
    const int64_t page = slot / a.page_size;
    return page * a.kv_heads * a.page_size + (slot - page * a.page_size);
}

// A step: 8 values, or 4.
template <typename T> struct Raw4 {
    uint2 w[sizeof(T) / 2];
};
template <typename T, int kStep> using Raw = std::conditional_t<kStep == 8, Raw8<T>, Raw4<T>>;
__device__ __forceinline__ void load_step(const float *p, Raw4<float> &r) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = make_uint2(w.x, w.y), r.w[1] = make_uint2(w.z, w.w);
}
__device__ __forceinline__ void load_step(const __nv_bfloat16 *p, Raw4<__nv_bfloat16> &r) {
    r.w[0] = *reinterpret_cast<const uint2 *>(p);
}
template <typename T> __device__ __forceinline__ void load_step(const T *p, Raw8<T> &r) { r = load_raw8_written(p); }
__device__ __forceinline__ void as_floats(const Raw4<float> &r, float (&x)[4]) {
    x[0] = __uint_as_float(r.w[0].x), x[1] = __uint_as_float(r.w[0].y);
    x[2] = __uint_as_float(r.w[1].x), x[3] = __uint_as_float(r.w[1].y);
}
__device__ __forceinline__ void as_floats(const Raw4<__nv_bfloat16> &r, float (&x)[4]) {
    x[0] = __uint_as_float(r.w[0].x << 16), x[1] = __uint_as_float(r.w[0].x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.w[0].y << 16), x[3] = __uint_as_float(r.w[0].y & 0xFFFF0000u);
}
__device__ __forceinline__ void store_step(float *p, const Raw4<float> &r) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0].x, r.w[0].y, r.w[1].x, r.w[1].y);
}
__device__ __forceinline__ void store_step(__nv_bfloat16 *p, const Raw4<__nv_bfloat16> &r) {
    *reinterpret_cast<uint2 *>(p) = r.w[0];
}
template <typename T> __device__ __forceinline__ void store_step(T *p, const Raw8<T> &r) { store_raw8(p, r); }
__device__ __forceinline__ void store_step(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_step(__nv_bfloat16 *p, const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
template <typename T> __device__ __forceinline__ void store_step(T *p, const float (&x)[8]) { store8(p, x); }
__device__ __forceinline__ void encode_step(uint8_t *c, const float (&x)[8], float s) {
    *reinterpret_cast<uint2 *>(c) = encode8(x, s);
}
__device__ __forceinline__ void encode_step(uint8_t *c, const float (&x)[4], float s) {
    *reinterpret_cast<uint32_t *>(c) = encode4(x, s);
}

// kLanes lanes (a power of two) hold a row of up to 2 kStep kLanes values, a warp kRows rows
// at once: a group.
// Groups whose loads are in flight, and blocks per SM, which give their registers: 20011
// tokens into an E4M3 cache 2 groups 94 us, 3: 90, 4: 108; into a bf16 cache 84, 86, 97; 8000
// tokens in fp32 with 3 blocks 63 us, with 2 and 3 groups 58.  Steps of 4, 10000 tokens of
// 16 + 16 heads of 80: bf16 cache 2 groups 48 us, 3: 45, 4: 43, 6: 42 (500 tokens 5 % slower);
// E4M3 55, 50, 53, 52.
template <typename T, bool kE4M3, int kStep>
constexpr int kInFlight = sizeof(T) == 4 || kE4M3 ? 3 : kStep == 4 ? 4 : 2;
template <typename T> constexpr int kBlocks = sizeof(T) == 4 ? 2 : 3;

template <typename T, bool kE4M3, int kStep, int kLanes>
__global__ void __launch_bounds__(kThreads, kBlocks<T>) rotary_kernel(const RotaryArgs a) {
    constexpr int kRows = 32 / kLanes, kAhead = kInFlight<T, kE4M3, kStep>, kHalf = kStep / 2;
    __shared__ float2 table[kWarps * kMaxPairs];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, tokens = kWarps / a.parts;
    const int64_t token0 = (int64_t)blockIdx.x * tokens, token = token0 + warp / a.parts;
    const int lane = threadIdx.x % kLanes, sub = (threadIdx.x & 31) / kLanes;
    const int total = a.q_rows + a.k_rows + a.v_rows, d = a.head_dim;
    const int groups = token < a.n_tokens ? (total + kRows - 1) / kRows : 0;

    // this lane's two steps, and whether each is turned
    const int steps = d / kStep, turned = 2 * a.pairs / kStep;
    int s0, s1;
    if (a.adjacent || lane >= turned / 2) {
        s0 = 2 * lane, s1 = s0 + 1;
    } else {
        s0 = lane, s1 = lane + turned / 2;
    }
    const bool on0 = s0 < steps, on1 = s1 < steps;
    const T *q = (const T *)a.q + token * a.q_stride, *k = (const T *)a.k + token * a.k_stride;
    const T *v = (const T *)a.v + token * a.v_stride;

    struct Pair {
        Raw<T, kStep> x, y;
    } raw[kAhead];
    const auto fetch = [&](int g, Pair &p) {
        int r = g * kRows + sub;
        p.x = p.y = Raw<T, kStep>{};
        if (g >= groups || r >= total) return;
        const T *src = q;
        if (r >= a.q_rows) {
            r -= a.q_rows, src = k;
            if (r >= a.k_rows) r -= a.k_rows, src = v;
        }
        src += r * d;
        if (on0) load_step(src + s0 * kStep, p.x);
        if (on1) load_step(src + s1 * kStep, p.y);
    };
    int g = warp % a.parts;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(g + i * a.parts, raw[i]);

    const int64_t at = groups && a.k_rows ? cache_row(a, token, (threadIdx.x & 31) == 0 && g == 0) : -1;
    // the sines and cosines of the block's tokens, each once
    for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
        const int t = i / a.pairs;
        if (token0 + t < a.n_tokens) table[i] = turn_of(a, token0 + t, i - t * a.pairs);
    }
    __syncthreads();
    if (groups == 0) return;
    const float2 *cs = table + warp / a.parts * a.pairs;
    float co[kStep], si[kStep];  // halves: of the step's pairs; adjacent: of half as many of each step
    const bool turn0 = s0 < turned, turn1 = s1 < turned;
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
        const int j = a.adjacent ? (i < kHalf ? kHalf * s0 + i : kHalf * s1 + i - kHalf) : kStep * s0 + i;
        const float2 x = j < a.pairs ? cs[j] : make_float2(1.0f, 0.0f);
        co[i] = x.x, si[i] = x.y;
    }
    const auto turn = [&](float (&x)[kStep], float (&y)[kStep]) {
        if (a.adjacent) {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                const float p = x[2 * i], o = x[2 * i + 1], p1 = y[2 * i], o1 = y[2 * i + 1];
                if (turn0) {
                    x[2 * i] = p * co[i] - o * si[i];
                    x[2 * i + 1] = o * co[i] + p * si[i];
                }
                if (turn1) {
                    y[2 * i] = p1 * co[kHalf + i] - o1 * si[kHalf + i];
                    y[2 * i + 1] = o1 * co[kHalf + i] + p1 * si[kHalf + i];
                }
            }
        } else if (turn0) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const float p = x[i], o = y[i];
                x[i] = p * co[i] - o * si[i];
                y[i] = o * co[i] + p * si[i];
            }
        }
    };
    T *q_out = (T *)a.qo + token * a.qo_stride, *k_out = (T *)a.ko + token * a.ko_stride;

    const auto finish = [&](int g, const Pair &p) {
        const int r = g * kRows + sub;
        float x[kStep], y[kStep];
        as_floats(p.x, x);
        as_floats(p.y, y);
        if ((g + 1) * kRows <= a.q_rows) {  // queries alone, the most
            turn(x, y);
            if (on0) store_step(q_out + r * d + s0 * kStep, x);
            if (on1) store_step(q_out + r * d + s1 * kStep, y);
            return;
        }
        const bool live = r < total, values = r >= a.q_rows + a.k_rows, key = !values && r >= a.q_rows;
        if (!values) turn(x, y);
        const int head = values ? r - a.q_rows - a.k_rows : key ? r - a.q_rows : r;
        if (live && !values && (!key || a.ko)) {
            T *dst = (key ? k_out : q_out) + head * d;
            if (on0) store_step(dst + s0 * kStep, x);
            if (on1) store_step(dst + s1 * kStep, y);
        }
        const bool held = live && (key || values) && at >= 0;
        const int64_t row = at + (int64_t)head * a.page_size;
        if constexpr (kE4M3) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < kStep; ++i) amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            if (!held) return;
            const int e = row_exponent(amax);
            uint8_t *c = (uint8_t *)(values ? a.vc : a.kc) + row * d;
            if (on0) encode_step(c + s0 * kStep, x, pow2i(-e));
            if (on1) encode_step(c + s1 * kStep, y, pow2i(-e));
            if (lane == 0) (values ? a.ve : a.ke)[row] = (uint8_t)(e + 127);
        } else if (held) {
            T *c = (T *)(values ? a.vc : a.kc) + row * d;
            if (values) {  // a value row keeps its bits
                if (on0) store_step(c + s0 * kStep, p.x);
                if (on1) store_step(c + s1 * kStep, p.y);
            } else {
                if (on0) store_step(c + s0 * kStep, x);
                if (on1) store_step(c + s1 * kStep, y);
            }
        }
    };
    while (g < groups) {  // the same for the whole warp
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (g >= groups) break;
            finish(g, raw[i]);
            fetch(g + kAhead * a.parts, raw[i]);
            g += a.parts;
        }
    }
}

// What no step of 4 fits, up to head_dim 256: a warp per kScalarRows rows of a token,
// a value per lane and step.  All of a row is read before any of it is written, so calls
// in place are safe here too.
constexpr int kScalarRows = 4;

template <typename T, bool kE4M3>
__global__ void __launch_bounds__(kThreads) rotary_scalar(const RotaryArgs a) {
    __shared__ float2 table[kWarps][kMaxPairs];
    grid_dep_wait();
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t token = w / a.parts;
    if (token >= a.n_tokens) return;
    const int part = (int)(w - token * a.parts), lane = threadIdx.x & 31;
    const int total = a.q_rows + a.k_rows + a.v_rows, d = a.head_dim;
    const int64_t at = cache_row(a, token, part == 0 && lane == 0);
    float2 *cs = table[threadIdx.x >> 5];
    for (int j = lane; j < a.pairs; j += 32) cs[j] = turn_of(a, token, j);
    __syncwarp();
    for (int r = part * kScalarRows; r < min(total, (part + 1) * kScalarRows); ++r) {
        const bool values = r >= a.q_rows + a.k_rows, key = !values && r >= a.q_rows;
        const int head = values ? r - a.q_rows - a.k_rows : key ? r - a.q_rows : r;
        const T *src = (values ? (const T *)a.v + token * a.v_stride
                               : key ? (const T *)a.k + token * a.k_stride : (const T *)a.q + token * a.q_stride) +
                       (int64_t)head * d;
        float x[8], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = lane + 32 * i;
            x[i] = 0.0f;
            if (j >= d) continue;
            x[i] = to_f32(src[j]);
            if (!values && j < 2 * a.pairs) {
                const bool second = a.adjacent ? j & 1 : j >= a.pairs;
                const int other = a.adjacent ? j ^ 1 : second ? j - a.pairs : j + a.pairs;
                const float2 t = cs[a.adjacent ? j >> 1 : second ? j - a.pairs : j];
                const float o = to_f32(src[other]);
                x[i] = second ? x[i] * t.x + o * t.y : x[i] * t.x - o * t.y;
            }
            amax = fmaxf(amax, fabsf(x[i]));
        }
        __syncwarp();
        T *dst = values ? nullptr : key ? (T *)a.ko + token * a.ko_stride : (T *)a.qo + token * a.qo_stride;
        if (key && !a.ko) dst = nullptr;
        const bool held = (key || values) && at >= 0;
        const int64_t row = at + (int64_t)head * a.page_size;
        int e = 0;
        if constexpr (kE4M3) {
            e = row_exponent(warp_max(amax));
            if (held && lane == 0) (values ? a.ve : a.ke)[row] = (uint8_t)(e + 127);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = lane + 32 * i;
            if (j >= d) continue;
            if (dst) from_f32(dst + (int64_t)head * d + j, x[i]);
            if (!held) continue;
            if constexpr (kE4M3)
                ((uint8_t *)(values ? a.vc : a.kc))[row * d + j] = encode1(x[i] * pow2i(-e));
            else if (values)
                ((T *)a.vc)[row * d + j] = src[j];
            else
                from_f32((T *)a.kc + row * d + j, x[i]);
        }
    }
}

template <typename T, bool kE4M3, int kStep, int kLanes>
void launch_lanes(RotaryArgs a, int sms, cudaStream_t st) {
    constexpr int rows = 32 / kLanes;
    // As few warps per token as leave a block per SM (512 tokens x 48 rows: 4.2 us, with
    // twice as many 6.3), one only where there are three per SM (20011 tokens x 56 rows 90
    // us, with two warps 94; 1536 tokens 11.6 and 9.0); no more than a token has groups.
    const int groups = (a.q_rows + a.k_rows + a.v_rows + rows - 1) / rows;
    a.parts = kWarps;
    while (a.parts > 1 &&
           (a.parts > groups || a.n_tokens * a.parts / 2 >= (a.parts > 2 ? 1ll : 3ll) * kWarps * sms))
        a.parts /= 2;
    const int64_t grid = (a.n_tokens * a.parts + kWarps - 1) / kWarps;
    launch_k(rotary_kernel<T, kE4M3, kStep, kLanes>, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
}

template <typename T, bool kE4M3, int kStep>
void launch_steps(const RotaryArgs &a, int sms, cudaStream_t st) {
    constexpr int kMost = 128 / kStep;  // lanes of a row of 256 values
    if (a.head_dim <= 64)
        launch_lanes<T, kE4M3, kStep, kMost / 4>(a, sms, st);
    else if (a.head_dim <= 128)
        launch_lanes<T, kE4M3, kStep, kMost / 2>(a, sms, st);
    else
        launch_lanes<T, kE4M3, kStep, kMost>(a, sms, st);
}

template <typename T, bool kE4M3>
dflash2_status launch_rotary(RotaryArgs a, int step, int sms, cudaStream_t st) {
    if (step == 8) {
        launch_steps<T, kE4M3, 8>(a, sms, st);
    } else if (step == 4) {
        launch_steps<T, kE4M3, 4>(a, sms, st);
    } else {
        a.parts = (a.q_rows + a.k_rows + a.v_rows + kScalarRows - 1) / kScalarRows;
        const int64_t warps = a.n_tokens * a.parts;
        launch_k(rotary_scalar<T, kE4M3>, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kThreads), 0, st, a);
    }
    return launch_status();
}

dflash2_status run_rotary(RotaryArgs a, int32_t dtype, int32_t kv_format, int32_t rotary_dim, bool cached, void *stream) {
    if (dtype != DFLASH2_F32 && dtype != DFLASH2_BF16) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (kv_format != DFLASH2_KV_NATIVE && kv_format != DFLASH2_KV_E4M3) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    const int64_t total = (int64_t)a.q_rows + a.k_rows + a.v_rows;
    const int64_t qw = (int64_t)a.q_rows * a.head_dim, kw = (int64_t)a.k_rows * a.head_dim;
    constexpr int64_t kMaxStride = 1ll << 32;
    const auto bad = [&](int64_t stride, int64_t width) { return stride < width || stride > kMaxStride; };
    if (a.head_dim < 1 || a.head_dim > 256 || rotary_dim < 2 || rotary_dim > a.head_dim || rotary_dim % 2 != 0 ||
        a.axes < 1 || a.axes > 255 || a.adjacent < 0 || a.adjacent > 1 || !(fabsf(a.magnitude) <= FLT_MAX) ||
        a.n_tokens < 0 || a.q_rows < 0 || a.k_rows < 0 || (cached && a.k_rows < 1) || total < 1 ||
        total > (1 << 16) || a.n_tokens > INT32_MAX / total || (a.q_rows && (bad(a.q_stride, qw) || bad(a.qo_stride, qw))) ||
        (a.k_rows && (bad(a.k_stride, kw) || (a.ko && bad(a.ko_stride, kw)))) || (cached && bad(a.v_stride, kw)))
        return DFLASH2_ERR_INVALID_ARG;
    const int64_t num_pages = a.n_slots;  // turned into slots below
    if (cached && (a.page_size < 1 || num_pages < 0 || num_pages > (INT64_MAX >> 9) / a.page_size / a.kv_heads))
        return DFLASH2_ERR_INVALID_ARG;
    if (a.n_tokens == 0) return DFLASH2_OK;
    const bool q8 = kv_format == DFLASH2_KV_E4M3;
    if (!a.positions || !a.freq || !a.axis || (a.q_rows && (!a.q || !a.qo)) || (a.k_rows && !a.k) ||
        (!cached && a.k_rows && !a.ko) ||
        (cached && (!a.v || !a.slots || !a.kc || !a.vc || (q8 && (!a.ke || !a.ve)))) ||
        (a.q == a.qo && a.q_rows && a.q_stride != a.qo_stride) || (a.k_rows && a.k == a.ko && a.k_stride != a.ko_stride))
        return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == DFLASH2_F32 ? 4 : 2;
    if ((a.q_rows && (!aligned_to(a.q, el) || !aligned_to(a.qo, el))) || (a.k_rows && !aligned_to(a.k, el)) ||
        !aligned_to(a.ko, el) || !aligned_to(a.positions, 8) || !aligned_to(a.freq, 8) || !aligned_to(a.err, 4) ||
        (cached && (!aligned_to(a.v, el) || !aligned_to(a.slots, 8) ||
                    (!q8 && (!aligned_to(a.kc, el) || !aligned_to(a.vc, el))))))
        return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    const dflash2_status st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    a.n_slots = cached ? num_pages * a.page_size : 0;
    // the widest step with aligned rows and pairs whose halves both begin at a step
    const auto steps_of = [&](int step) {
        const int64_t bytes = std::min<int64_t>(16, step * (int64_t)el);
        const auto rows = [&](const void *p, int64_t stride) {
            return aligned_to(p, (uintptr_t)bytes) && stride * (int64_t)el % bytes == 0;
        };
        const uintptr_t kept = q8 ? (uintptr_t)step : (uintptr_t)bytes;
        return a.head_dim % step == 0 && rotary_dim % (a.adjacent ? step : 2 * step) == 0 &&
               (!a.q_rows || (rows(a.q, a.q_stride) && rows(a.qo, a.qo_stride))) &&
               (!a.k_rows || (rows(a.k, a.k_stride) && (!a.ko || rows(a.ko, a.ko_stride)))) &&
               (!cached || (rows(a.v, a.v_stride) && aligned_to(a.kc, kept) && aligned_to(a.vc, kept)));
    };
    const int step = steps_of(8) ? 8 : steps_of(4) ? 4 : 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    if (cached && q8)
        return dtype == DFLASH2_F32 ? launch_rotary<float, true>(a, step, di.sm_count, s) : launch_rotary<B, true>(a, step, di.sm_count, s);
    return dtype == DFLASH2_F32 ? launch_rotary<float, false>(a, step, di.sm_count, s) : launch_rotary<B, false>(a, step, di.sm_count, s);
}

}  // namespace
}  // namespace dflash2

using namespace dflash2;

extern "C" dflash2_status dflash2_rotary(const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride,
                                         const int64_t *positions, int32_t axes, const uint64_t *freq,
                                         const uint8_t *axis, int32_t rotary_dim, int32_t adjacent, float magnitude,
                                         int64_t n_tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int32_t dtype, void *q_out, int64_t q_out_row_stride, void *k_out,
                                         int64_t k_out_row_stride, int32_t *err_word, void *stream) {
    RotaryArgs a{};
    a.q = q, a.q_stride = q_row_stride, a.k = k, a.k_stride = k_row_stride;
    a.positions = positions, a.axes = axes, a.freq = freq, a.axis = axis, a.pairs = rotary_dim / 2;
    a.adjacent = adjacent, a.magnitude = magnitude, a.n_tokens = n_tokens;
    a.q_rows = q_heads, a.k_rows = kv_heads, a.head_dim = head_dim, a.kv_heads = kv_heads;
    a.qo = q_out, a.qo_stride = q_out_row_stride, a.ko = k_out, a.ko_stride = k_out_row_stride, a.err = err_word;
    return run_rotary(a, dtype, DFLASH2_KV_NATIVE, rotary_dim, false, stream);
}

extern "C" dflash2_status dflash2_rotary_kv_write(
    const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride, const void *v, int64_t v_row_stride,
    const int64_t *positions, int32_t axes, const uint64_t *freq, const uint8_t *axis, int32_t rotary_dim,
    int32_t adjacent, float magnitude, const int64_t *slots, int64_t n_tokens, int32_t q_heads, int32_t kv_heads,
    int32_t head_dim, int32_t page_size, int64_t num_pages, int32_t dtype, int32_t kv_format, void *q_out,
    int64_t q_out_row_stride, void *k_out, int64_t k_out_row_stride, void *k_cache, void *v_cache, uint8_t *k_exp,
    uint8_t *v_exp, int32_t *err_word, void *stream) {
    RotaryArgs a{};
    a.q = q, a.q_stride = q_row_stride, a.k = k, a.k_stride = k_row_stride, a.v = v, a.v_stride = v_row_stride;
    a.positions = positions, a.axes = axes, a.freq = freq, a.axis = axis, a.pairs = rotary_dim / 2;
    a.adjacent = adjacent, a.magnitude = magnitude, a.slots = slots, a.n_tokens = n_tokens;
    a.q_rows = q_heads, a.k_rows = kv_heads, a.v_rows = kv_heads, a.head_dim = head_dim, a.kv_heads = kv_heads;
    a.page_size = page_size, a.n_slots = num_pages;
    a.qo = q_out, a.qo_stride = q_out_row_stride, a.ko = k_out, a.ko_stride = k_out_row_stride;
    a.kc = k_cache, a.vc = v_cache, a.ke = k_exp, a.ve = v_exp, a.err = err_word;
    return run_rotary(a, dtype, kv_format, rotary_dim, true, stream);
}
