// The norms around a sublayer (attention, MLP) with its gate and residual:
//
//   norm:  out = x / sqrt(mean(x^2) + eps) * (w + offset)
//   join:  h  = post ? rms(y) * (w_post + offset) : y
//          r' = r + branch_scale * act(gate) * h
//          out = rms(r') * (w_next + offset)          (if asked)
//
// and the E4M3 block quantisation of rows, alone or of `out` as it is made.  Every value
// is read and written once: the row stays in registers between the two sums of squares,
// which a join needs one after the other (three sums over r and h alone would do in one
// pass, but the next norm would lose what cancels in r + h).  r' goes into the next norm
// as computed in fp32, not as rounded for storage.
//
// HBM bounds them once the rows fill the GPU, a launch below that.  A thread holds 4 x 8 values
// (2 x 8 of rows that go value by value); a row takes as many threads as it needs (a warp
// up to 1024 values, 512 value by value), and the loads of y, r and the gate are
// all in flight at once.  The choice goes by the row's length alone, so a row's result does
// not depend on how many there are.
// Measured (graph replays, rotating inputs): norm of 20011 x 7168 bf16 83 us, 6.9 TB/s; join
// with an fp32 stream, a full sigmoid gate and both norms 284 us, 7.1 TB/s; bf16 join without
// a gate 164 us, 7.0 TB/s, to E4M3 blocks 165; norm of 20011 x 5120 to E4M3 blocks 57 us, 5.4
// TB/s; quantisation of 8192 x 7168 bf16 30 us, 6.0 TB/s; one row of 4096: norm 2.3 us, join
// 3.3 us.
#include <type_traits>

#include "rows.cuh"
#include "tcgen05.cuh"

namespace dflash2 {
namespace {

enum { kGateNone = DFLASH2_GATE_NONE, kGateChannel = DFLASH2_GATE_CHANNEL,
       kGateToken = DFLASH2_GATE_TOKEN, kGateFull = DFLASH2_GATE_FULL };

struct NormArgs {
    const void *x;  // residual stream (norm: the input)
    const void *y, *w_post, *gate, *w_next;
    int64_t x_stride, y_stride, gate_stride, r_stride;
    int32_t gate_kind, gate_act;
    float branch, w_off, eps;
    int64_t rows;
    int32_t hidden;
    void *r_out, *out;
    float *scale;   // E4M3 blocks if not NULL
    bool code_vec;  // rows of codes are 8-byte aligned
};

// 8 values of a thread, at first, first + step, ... of a row of n: steps of 1 and whole
// 16-byte pieces (kVec), or any.
template <typename T, bool kVec> struct Held {
    Raw8<T> raw;
    __device__ __forceinline__ void load(const T *row, int first, int, int n) {
        raw = Raw8<T>{};
        if (first < n) raw = load_raw8_written(row + first);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const { as_floats(raw, x); }
};
// (bits: a conversion beside its load waits for it, and the row's loads for one another)
template <typename T> struct Held<T, false> {
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    uint32_t v[8];
    __device__ __forceinline__ void load(const T *row, int first, int step, int n) {
        const Bits *p = reinterpret_cast<const Bits *>(row) + first;
        if (first + 7 * step < n) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i * step];
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = first + i * step < n ? p[i * step] : 0u;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(sizeof(T) == 4 ? v[i] : v[i] << 16);
    }
};
template <typename T, bool kVec>
__device__ __forceinline__ void put8(T *row, int first, int step, int n, const float (&x)[8]) {
    if constexpr (kVec) {
        if (first < n) store8(row + first, x);
    } else if (first + 7 * step < n) {
        T *p = row + first;
#pragma unroll
        for (int i = 0; i < 8; ++i) from_f32(p + i * step, x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (first + i * step < n) from_f32(row + first + i * step, x[i]);
    }
}

// Eight values two at a time, an issue slot for both.
__device__ __forceinline__ uint64_t two(const float (&x)[8], int i) { return f2(x[2 * i], x[2 * i + 1]); }
__device__ __forceinline__ void set_two(float (&x)[8], int i, uint64_t v) { unf2(v, x[2 * i], x[2 * i + 1]); }
__device__ __forceinline__ void add_squares(const float (&x)[8], uint64_t &sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fma2(two(x, i), two(x, i), sum);
}
__device__ __forceinline__ float both(uint64_t v) {
    float lo, hi;
    unf2(v, lo, hi);
    return lo + hi;
}
// x *= factor * (w + offset), or factor alone
__device__ __forceinline__ void scale8(float (&x)[8], float factor) {
#pragma unroll
    for (int i = 0; i < 4; ++i) set_two(x, i, mul2(two(x, i), f2(factor, factor)));
}
__device__ __forceinline__ void weigh8(float (&x)[8], const float (&w)[8], float offset) {
#pragma unroll
    for (int i = 0; i < 4; ++i) set_two(x, i, mul2(two(x, i), add2(two(w, i), f2(offset, offset))));
}

__device__ __forceinline__ float gate_value(float g, int act) {
    if (act == DFLASH2_GATE_SIGMOID) return __fdividef(1.0f, 1.0f + expf(-g));  // 2 ulp each
    return act == DFLASH2_GATE_TANH ? tanhf(g) : g;
}

// The sum over a row's threads, the same in each (fixed order).  `red` is used by one
// call of the row alone.
template <bool kWarpRow> __device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if constexpr (!kWarpRow) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f);
    }
    return v;
}

// Blocks of 256 threads per SM that the registers leave room for, by the bytes a value takes:
// rows in flight against what a thread holds of each.  20011 x 7168: join with an fp32 stream
// and a full gate 2: 315 us, 3: 284, 4: 309; bf16 join 2: 176, 4: 165; fp32 join of 20011 x
// 4096 2: 189, 3: 242; bf16 norm 4: 90, 5: 84.
// Value by value a thread holds 32 bits of each, so it takes two pieces in place of four, four
// blocks: bf16 join of 10000 x 5001 127 us (four pieces 181, one 240), with an fp32 stream and
// a full gate 165 (230), of 30000 x 1001 73 (71) and 91 (93).
// What these leave some joins is less than they hold, and they spill: bf16 rows 56 to 68 bytes, a bf16 stream
// with fp32 rows 164 to 200, E4M3 blocks of odd widths 274 to 288, rows of more than 16384 60 to 550.
template <typename TX, typename T, bool kVec, bool kJoin, int kChunks>
constexpr int kBlocks256 = kJoin ? (kChunks == 2                    ? 4
                                    : sizeof(TX) + sizeof(T) == 4   ? (kVec ? 4 : 3)
                                    : sizeof(TX) + sizeof(T) == 6 && kVec ? 3 : 2)
                           : kVec && sizeof(TX) + sizeof(T) == 4 ? 5 : 4;
template <typename TX, typename T, bool kVec, bool kJoin, int kChunks, int kThreads>
constexpr int kRowBlocks = kThreads <= 256 ? kBlocks256<TX, T, kVec, kJoin, kChunks>
                           : kThreads == 512 && kBlocks256<TX, T, kVec, kJoin, kChunks> > 3 ? 2 : 1;

// kThreads: a row's threads at most; 32 stands for a warp per row, 8 rows a block.  kChunks:
// a thread's pieces of 8 values.
// (kE4M3 in the type, not from a.scale: norms to E4M3 blocks 60 -> 58 us at 20011 x 5120.)
template <typename TX, typename T, bool kVec, bool kJoin, bool kE4M3, int kChunks, int kThreads>
__global__ void __launch_bounds__(kThreads == 32 ? 256 : kThreads, kRowBlocks<TX, T, kVec, kJoin, kChunks, kThreads>)
    sublayer_kernel(const NormArgs a) {
    static_assert(!kE4M3 || kChunks == kQuantUnroll, "blocks are quantised four at a time");
    constexpr bool kWarpRow = kThreads == 32;
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();  // a product that follows sets itself up meanwhile (1 x 4096 x 6144 after a
                        // norm 8.3 us in place of 9.6, 512 rows 20.5 for 21.4)
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int per = kWarpRow ? 32 : blockDim.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) return;  // a whole warp or block
    const int hidden = a.hidden;
    const float inv_n = 1.0f / (float)hidden;
    // Eight neighbouring values of each of a thread's pieces of the row; rows that are not whole
    // 16-byte pieces go value by value, neighbours in neighbouring threads, unless E4M3
    // blocks want them as above.
    constexpr bool apart = !kVec && !kE4M3;
    const int step = apart ? per : 1, origin = apart ? t : t * 8;
    const auto first = [&](int c) { return c * 8 * per + origin; };

    Held<TX, kVec> held[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) held[c].load((const TX *)a.x + row * a.x_stride, first(c), step, hidden);
    float r[kChunks][8];
    uint64_t sum = 0;
    if constexpr (kJoin) {
        Held<T, kVec> y[kChunks], g[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            y[c].load((const T *)a.y + row * a.y_stride, first(c), step, hidden);
            if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull)
                g[c].load((const T *)a.gate + (a.gate_kind == kGateFull ? row * a.gate_stride : 0), first(c), step, hidden);
        }
        const float token_gate =
            a.gate_kind == kGateToken
                ? gate_value(to_f32(((const T *)a.gate)[row * a.gate_stride]), a.gate_act) : 1.0f;
        float y_rms = 1.0f;
        if (a.w_post) {
            uint64_t s = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float v[8];
                y[c].get(v);
                add_squares(v, s);
            }
            y_rms = __frsqrt_rn(row_sum<kWarpRow>(both(s), red[0]) * inv_n + a.eps);
        }
        // the branch's scale goes with the row's root or its gate
        const float factor = y_rms * a.branch * token_gate;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float h[8], v[8];
            y[c].get(h);
            scale8(h, factor);
            if (a.w_post) {
                Held<T, kVec> w;
                w.load((const T *)a.w_post, first(c), step, hidden);
                w.get(v);
                weigh8(h, v, a.w_off);
            }
            held[c].get(r[c]);
            if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
                g[c].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = gate_value(v[i], a.gate_act);
#pragma unroll
                for (int i = 0; i < 4; ++i) set_two(r[c], i, fma2(two(h, i), two(v, i), two(r[c], i)));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) set_two(r[c], i, add2(two(r[c], i), two(h, i)));
            }
            put8<TX, kVec>((TX *)a.r_out + row * a.r_stride, first(c), step, hidden, r[c]);
        }
        if (!a.w_next) return;
    } else {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) held[c].get(r[c]);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) add_squares(r[c], sum);  // past the end r is 0, or the row NaN
    const float rms = __frsqrt_rn(row_sum<kWarpRow>(both(sum), red[1]) * inv_n + a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        Held<T, kVec> w;
        float v[8];
        w.load((const T *)a.w_next, first(c), step, hidden);
        w.get(v);
        scale8(r[c], rms);
        weigh8(r[c], v, a.w_off);
        if constexpr (!kE4M3) put8<T, kVec>((T *)a.out + row * hidden, first(c), step, hidden, r[c]);
    }
    if constexpr (kE4M3) {
        if (!kVec)
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (first(c) + i >= hidden) r[c][i] = 0.0f;
        uint2 codes[kChunks];
        float scale;
        quantise_blocks(r, &scale, codes);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if (first(c) < hidden)
                store_codes((uint8_t *)a.out + row * hidden + first(c), hidden - first(c), a.code_vec, codes[c]);
        const int block = (quant_lane() * per + t) / kQuantLanes;
        if ((t & 3) == 0 && block * kQuantBlock < hidden)
            a.scale[row * ((hidden + kQuantBlock - 1) / kQuantBlock) + block] = scale;
    }
}

template <typename TX, typename T, bool kVec, bool kJoin, bool kE4M3, int kChunks>
void launch_chunks(const NormArgs &a, cudaStream_t st) {
    const int threads = ((a.hidden + 8 * kChunks - 1) / (8 * kChunks) + 31) / 32 * 32;
    const dim3 grid((unsigned)a.rows);
    if (threads == 32)
        launch_k(sublayer_kernel<TX, T, kVec, kJoin, kE4M3, kChunks, 32>, dim3((unsigned)((a.rows + 7) / 8)), dim3(256),
                 0, st, a);
    else if (threads <= 256)
        launch_k(sublayer_kernel<TX, T, kVec, kJoin, kE4M3, kChunks, 256>, grid, dim3(threads), 0, st, a);
    else if (threads <= 512)
        launch_k(sublayer_kernel<TX, T, kVec, kJoin, kE4M3, kChunks, 512>, grid, dim3(threads), 0, st, a);
    else
        launch_k(sublayer_kernel<TX, T, kVec, kJoin, kE4M3, kChunks, 1024>, grid, dim3(threads), 0, st, a);
}

template <typename TX, typename T, bool kVec, bool kJoin, bool kE4M3>
dflash2_status launch_vec(const NormArgs &a, cudaStream_t st) {
    if constexpr (kVec || kE4M3)
        launch_chunks<TX, T, kVec, kJoin, kE4M3, kQuantUnroll>(a, st);
    else if (a.hidden <= 1024 * 16)  // what 1024 threads hold in two pieces
        launch_chunks<TX, T, false, kJoin, false, 2>(a, st);
    else
        launch_k(sublayer_kernel<TX, T, false, kJoin, false, 4, 1024>, dim3((unsigned)a.rows), dim3(1024), 0, st, a);
    return launch_status();
}

template <typename TX, typename T, bool kJoin>
dflash2_status launch_norm(const NormArgs &a, bool vec, cudaStream_t st) {
    if (a.scale) return vec ? launch_vec<TX, T, true, kJoin, true>(a, st) : launch_vec<TX, T, false, kJoin, true>(a, st);
    return vec ? launch_vec<TX, T, true, kJoin, false>(a, st) : launch_vec<TX, T, false, kJoin, false>(a, st);
}

template <bool kJoin>
dflash2_status dispatch_norm(NormArgs a, int32_t x_dtype, int32_t dtype, bool vec, cudaStream_t st) {
    a.code_vec = a.scale && a.hidden % 8 == 0 && aligned_to(a.out, 8);
    if (x_dtype == DFLASH2_F32)
        return dtype == DFLASH2_F32 ? launch_norm<float, float, kJoin>(a, vec, st)
                                    : launch_norm<float, __nv_bfloat16, kJoin>(a, vec, st);
    return dtype == DFLASH2_F32 ? launch_norm<__nv_bfloat16, float, kJoin>(a, vec, st)
                                : launch_norm<__nv_bfloat16, __nv_bfloat16, kJoin>(a, vec, st);
}

bool known(int32_t dtype) { return dtype == DFLASH2_F32 || dtype == DFLASH2_BF16; }
uintptr_t size_of(int32_t dtype) { return dtype == DFLASH2_F32 ? 4 : 2; }
constexpr int64_t kMaxStride = 1ll << 32;  // row strides: 2^31 rows of them stay in 64 bits

dflash2_status check_norm(const NormArgs &a, int32_t x_dtype, int32_t dtype) {
    if (!known(x_dtype) || !known(dtype)) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (a.rows < 0 || a.rows > INT32_MAX || a.hidden < 1 || a.hidden > 32768 || !(a.eps >= 0.0f) ||
        !(a.eps <= FLT_MAX) || !(fabsf(a.w_off) <= FLT_MAX) || a.x_stride < a.hidden || a.x_stride > kMaxStride)
        return DFLASH2_ERR_INVALID_ARG;
    return DFLASH2_OK;
}
// Rows in steps of 8 values: 16-byte aligned starts of whole steps.
bool vec_rows(const void *p, int64_t stride, uintptr_t el) {
    return aligned_to(p, 16) && stride * (int64_t)el % 16 == 0;
}

// ---- block quantisation of rows ----------------------------------------------
constexpr int kQuantThreads = 256;

// Sixteen lanes take four neighbouring blocks of a row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kQuantThreads)
    quantise_rows_kernel(const T *x, int64_t stride, int64_t rows, int32_t cols, uint8_t *q, float *scale,
                         bool code_vec) {
    grid_dep_wait();
    grid_dep_launch();  // a product that follows loads its weights meanwhile
    const int nb = (cols + kQuantBlock - 1) / kQuantBlock, groups = (nb + kQuantUnroll - 1) / kQuantUnroll;
    const int64_t g = ((int64_t)blockIdx.x * kQuantThreads + threadIdx.x) / kQuantLanes;
    const int64_t row = g / groups;
    const int block = (int)(g - row * groups) * kQuantUnroll, lane = threadIdx.x % kQuantLanes;
    const int left = row < rows ? cols - block * kQuantBlock - lane * 8 : 0;  // values from the first on
    Held<T, kVec> h[kQuantUnroll];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u)
        h[u].load(x + row * stride + block * kQuantBlock + lane * 8, u * kQuantBlock, 1, left);
    float v[kQuantUnroll][8], s;
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) h[u].get(v[u]);
    uint2 codes[kQuantUnroll];
    quantise_blocks(v, &s, codes);
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
        const int n = left - u * kQuantBlock;
        if (n > 0) store_codes(q + row * cols + (block + u) * kQuantBlock + lane * 8, n, code_vec, codes[u]);
    }
    if ((lane & 3) == 0 && row < rows && block + quant_lane() < nb) scale[row * nb + block + quant_lane()] = s;
}

}  // namespace

dflash2_status launch_quant_blocks_e4m3(const void *x, int64_t stride, int32_t dtype, int64_t rows, int32_t cols,
                                        uint8_t *q, float *scale, cudaStream_t st) {
    constexpr int kCols = kQuantBlock * kQuantUnroll;
    const int64_t grid = (rows * ((cols + kCols - 1) / kCols) * kQuantLanes + kQuantThreads - 1) / kQuantThreads;
    const bool vec = cols % 8 == 0 && vec_rows(x, stride, size_of(dtype));
    const bool code_vec = cols % 8 == 0 && aligned_to(q, 8);
    const dim3 g((unsigned)grid), t(kQuantThreads);
    using B = __nv_bfloat16;
    if (dtype == DFLASH2_F32) {
        const float *p = (const float *)x;
        if (vec)
            launch_k(quantise_rows_kernel<float, true>, g, t, 0, st, p, stride, rows, cols, q, scale, code_vec);
        else
            launch_k(quantise_rows_kernel<float, false>, g, t, 0, st, p, stride, rows, cols, q, scale, code_vec);
    } else {
        const B *p = (const B *)x;
        if (vec)
            launch_k(quantise_rows_kernel<B, true>, g, t, 0, st, p, stride, rows, cols, q, scale, code_vec);
        else
            launch_k(quantise_rows_kernel<B, false>, g, t, 0, st, p, stride, rows, cols, q, scale, code_vec);
    }
    return launch_status();
}

dflash2_status check_quant_blocks(const void *x, int64_t stride, int32_t dtype, int64_t rows, int32_t cols) {
    if (!known(dtype)) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || cols < 1 || cols > 1 << 30 || stride < cols || stride > kMaxStride || rows > INT32_MAX ||
        (int64_t)rows * ((cols + kQuantBlock - 1) / kQuantBlock) > 1ll << 34)
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0) return DFLASH2_OK;
    if (!x) return DFLASH2_ERR_INVALID_ARG;
    return aligned_to(x, size_of(dtype)) ? DFLASH2_OK : DFLASH2_ERR_MISALIGNED;
}

}  // namespace dflash2

using namespace dflash2;

extern "C" dflash2_status dflash2_quantize_blocks_e4m3(const void *x, int64_t x_row_stride, int64_t rows, int32_t cols,
                                                       int32_t dtype, uint8_t *q, float *scale, void *stream) {
    dflash2_status st = check_quant_blocks(x, x_row_stride, dtype, rows, cols);
    if (st != DFLASH2_OK || rows == 0) return st;
    if (!q || !scale) return DFLASH2_ERR_INVALID_ARG;
    if (!aligned_to(scale, 4)) return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    return launch_quant_blocks_e4m3(x, x_row_stride, dtype, rows, cols, q, scale, static_cast<cudaStream_t>(stream));
}

extern "C" dflash2_status dflash2_sublayer_norm(const void *x, int64_t x_row_stride, int32_t x_dtype,
                                                const void *weight, float weight_offset, float eps, int64_t rows,
                                                int32_t hidden, int32_t dtype, void *out, float *scale, void *stream) {
    NormArgs a{};
    a.x = x, a.x_stride = x_row_stride, a.w_next = weight, a.w_off = weight_offset, a.eps = eps;
    a.rows = rows, a.hidden = hidden, a.out = out, a.scale = scale;
    dflash2_status st = check_norm(a, x_dtype, dtype);
    if (st != DFLASH2_OK || rows == 0) return st;
    if (!x || !weight || !out) return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t xe = size_of(x_dtype), el = size_of(dtype);
    if (!aligned_to(x, xe) || !aligned_to(weight, el) || !aligned_to(out, scale ? 1 : el) || !aligned_to(scale, 4))
        return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    const bool vec = hidden % 8 == 0 && vec_rows(x, x_row_stride, xe) && aligned_to(weight, 16) &&
                     (scale || aligned_to(out, 16));
    return dispatch_norm<false>(a, x_dtype, dtype, vec, static_cast<cudaStream_t>(stream));
}

extern "C" dflash2_status dflash2_sublayer_join(
    const void *residual, int64_t residual_row_stride, int32_t residual_dtype, const void *y, int64_t y_row_stride,
    const void *post_weight, const void *gate, int32_t gate_kind, int64_t gate_row_stride, int32_t gate_act,
    float branch_scale, const void *next_weight, float weight_offset, float eps, int64_t rows, int32_t hidden,
    int32_t dtype, void *residual_out, int64_t residual_out_row_stride, void *out, float *scale, void *stream) {
    NormArgs a{};
    a.x = residual, a.x_stride = residual_row_stride, a.y = y, a.y_stride = y_row_stride;
    a.w_post = post_weight, a.gate = gate, a.gate_kind = gate_kind, a.gate_act = gate_act;
    a.gate_stride = gate_row_stride, a.branch = branch_scale, a.w_next = next_weight, a.w_off = weight_offset;
    a.eps = eps, a.rows = rows, a.hidden = hidden, a.r_out = residual_out, a.r_stride = residual_out_row_stride;
    a.out = out, a.scale = scale;
    dflash2_status st = check_norm(a, residual_dtype, dtype);
    if (st != DFLASH2_OK) return st;
    if (gate_kind < kGateNone || gate_kind > kGateFull || gate_act < DFLASH2_GATE_IDENTITY ||
        gate_act > DFLASH2_GATE_TANH || !(fabsf(branch_scale) <= FLT_MAX) || y_row_stride < hidden ||
        y_row_stride > kMaxStride || residual_out_row_stride < hidden || residual_out_row_stride > kMaxStride ||
        (gate_kind == kGateToken && (gate_row_stride < 1 || gate_row_stride > kMaxStride)) ||
        (gate_kind == kGateFull && (gate_row_stride < hidden || gate_row_stride > kMaxStride)))
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0) return DFLASH2_OK;
    if (!residual || !y || !residual_out || (gate_kind != kGateNone && !gate) || (next_weight && !out) ||
        (!next_weight && (out || scale)) || (residual_out == residual && residual_out_row_stride != residual_row_stride))
        return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t xe = size_of(residual_dtype), el = size_of(dtype);
    if (!aligned_to(residual, xe) || !aligned_to(residual_out, xe) || !aligned_to(y, el) ||
        !aligned_to(post_weight, el) || !aligned_to(next_weight, el) || (gate_kind != kGateNone && !aligned_to(gate, el)) ||
        !aligned_to(out, scale ? 1 : el) || !aligned_to(scale, 4))
        return DFLASH2_ERR_MISALIGNED;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    const bool gate_vec = gate_kind == kGateChannel  ? aligned_to(gate, 16)
                          : gate_kind == kGateFull ? vec_rows(gate, gate_row_stride, el) : true;
    const bool vec = hidden % 8 == 0 && vec_rows(residual, residual_row_stride, xe) &&
                     vec_rows(residual_out, residual_out_row_stride, xe) && vec_rows(y, y_row_stride, el) && gate_vec &&
                     aligned_to(post_weight, 16) && aligned_to(next_weight, 16) && (scale || aligned_to(out, 16));
    return dispatch_norm<true>(a, residual_dtype, dtype, vec, static_cast<cudaStream_t>(stream));
}
