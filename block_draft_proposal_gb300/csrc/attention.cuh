// Attention over the paged cache and over packed prompts: what the CUDA-core
// kernel (attention_simt.cu), the tcgen05 kernel (attention_tc.cu), the
// join of split rows and the entry points (attention.cu) share.
//
// Rows.  The T tokens of a request and the G = q_heads / kv_heads query heads
// of one key/value head are packed into T * G rows, row r = token r / G, head
// r % G of the group, so that a pass over the keys serves them all; rows go in
// blocks of 2^row_shift.  An item is one (request, key/value head, row block).
//
// Split of the cache (paged mode).  Requests are ragged and few rows may face
// many keys, so the keys are split by work, not by item: an item is worth its key
// tiles (kKeyTile keys each, at least one) and item_units more for its start and
// end; these units are numbered through, request by request, head by head, row
// block by row block, an item's extra ones first, and CTA c of C (at most W) takes
// the units [c W / C, (c + 1) W / C) of all W.  A CTA that holds all tiles of an
// item writes its rows; an item whose tiles span CTAs leaves unnormalised partial
// rows in the workspace, joined by combine_kernel in CTA order.
#pragma once

#include "kernels.h"

namespace dflash2 {
namespace attn {

constexpr int kKeyTile = 128;
constexpr int kMaxBatch = 65536;
constexpr int kMaxGroup = 128;
// Keys of a paged request.  Kernels count positions in 32 bits up to some tiles past the last key
// (its tile's end, and page numbers fetched fifteen tiles ahead).
constexpr int64_t kMaxKeys = (1ll << 31) - 4096;

struct Params {
    const void *q;
    int64_t q_stride;              // elements from token to token
    const void *k, *v;             // packed rows (prompt) or cache arrays (paged)
    int64_t k_stride, v_stride;    // prompt: elements from token to token
    const uint8_t *k_exp, *v_exp;  // E4M3 cache
    const int32_t *page_table;     // paged: [batch, max_pages]
    int32_t max_pages;
    int32_t page_size;
    int64_t num_pages;
    const int32_t *cu_q;
    const int32_t *kv_lens;        // paged
    const int64_t *tree_mask;      // paged: [total_q, mask_words] or NULL (chain)
    int32_t mask_words;
    int32_t batch, total_q, q_heads, kv_heads, group, head_dim;
    float scale_log2;              // scale * log2(e)
    void *out;
    float *lse;
    struct Join *join;             // paged: one per CTA, then
    float *part;                   // the partial rows' slots
    int32_t part_rows;             // rows of a slot
    int32_t row_shift;             // log2 of the rows of a block
    int32_t tile_units[4];         // units of a key tile, by quarters of a full row block
    int32_t item_units[4];         // units of an item beside its key tiles
    int32_t most_units;            // the largest of those that a request may have
    int32_t n_cta;                 // CTAs the work is split over
    int32_t *err;
};

// Partial slot s of the workspace: fp32 sums [ceil(head_dim / 4)][part_rows][4] (a
// warp writes and reads neighbouring rows), then part_rows maxima (log2 domain),
// then part_rows sums.  CTA c owns slots 2c
// (an item it did not start) and 2c + 1 (an item it started and did not end).
__host__ __device__ inline int64_t part_slot_floats(int32_t part_rows, int32_t head_dim) {
    return (int64_t)part_rows * ((head_dim + 3) / 4 * 4 + 2);
}
// Offset of a slot's maxima; the sums of weights follow.
__host__ __device__ inline int64_t part_stats(int32_t part_rows, int32_t head_dim) {
    return (int64_t)part_rows * ((head_dim + 3) / 4 * 4);
}

// The item that CTA c starts and does not end, for combine_kernel; every CTA
// writes its own.
struct alignas(16) Join {
    int32_t rows;  // live rows, or 0: there is none
    int32_t last;  // the CTA that ends it
    int32_t row0;  // its first row
    int32_t t0;    // the request's first packed token
    int32_t h;     // key/value head
    int32_t pad[3];
};

struct Request {
    int32_t t0, t;    // first packed token, tokens
    int32_t len, ctx; // keys, keys before the first token; len < 0: sees nothing
};

// cu_q and kv_lens of request b, clamped to what the arrays hold.  `bad` is
// raised for values that had to be.
template <bool kPaged>
__device__ __forceinline__ Request load_request(const Params &p, int32_t b, bool *bad) {
    Request r;
    const int32_t a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
    const int32_t lo = min(max(a, 0), p.total_q), hi = min(max(e, lo), p.total_q);
    *bad = a != lo || e != hi;
    r.t0 = lo;
    r.t = hi - lo;
    if (kPaged) {
        r.len = __ldg(p.kv_lens + b);
        r.ctx = r.len - r.t;
        if (r.len < r.t || (int64_t)r.len > (int64_t)p.max_pages * p.page_size) {
            *bad = true;
            r.len = 0;
            r.ctx = 0;
        }
        if (p.tree_mask && r.t > 64 * (int64_t)p.mask_words) *bad = true;
    } else {
        r.len = r.t;
        r.ctx = 0;
    }
    return r;
}

__device__ __forceinline__ int32_t row_blocks(const Params &p, const Request &r) {
    const uint32_t rows = (uint32_t)r.t * (uint32_t)p.group;  // below 2^31
    return (int32_t)((rows + (1u << p.row_shift) - 1u) >> p.row_shift);
}
__device__ __forceinline__ int32_t key_tiles(const Request &r) {
    return max(1, (r.len + kKeyTile - 1) / kKeyTile);
}
// Which of tile_units and item_units holds: that of the request's first row block.
__device__ __forceinline__ int32_t units_class(const Params &p, const Request &r) {
    const uint32_t rows = min((uint32_t)r.t * (uint32_t)p.group, 1u << p.row_shift);
    return (max(rows, 1u) - 1u) >> (p.row_shift - 2);
}
// Units of one item (a head and row block) of the request, and of all of them; 0 when it
// has no rows.
__device__ __forceinline__ int64_t units_of_item(const Params &p, const Request &r) {
    const int32_t c = units_class(p, r);
    return (int64_t)key_tiles(r) * p.tile_units[c] + p.item_units[c];
}
__device__ __forceinline__ int64_t request_units(const Params &p, const Request &r) {
    return (int64_t)p.kv_heads * row_blocks(p, r) * units_of_item(p, r);
}

// First unit of CTA c's range, and the CTA that holds unit u.  A key tile is the
// CTA's that holds its first unit; split_ctas leaves every range as many units as any
// tile has, so that no CTA between two others of an item has no tile.
__device__ __forceinline__ int64_t split_ctas(const Params &p, int64_t units) {
    if (units >= p.n_cta * (int64_t)p.most_units) return p.n_cta;
    return units < p.most_units ? min(units, (int64_t)1) : units / p.most_units;
}
__device__ __forceinline__ int64_t range_start(int64_t c, int64_t units, int64_t n_cta) {
    return c * units / n_cta;
}
__device__ __forceinline__ int32_t cta_of(int64_t u, int64_t units, int64_t n_cta) {
    return (int32_t)(((u + 1) * n_cta - 1) / units);
}

// Sum of a 64-bit value over the block; every thread gets it.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t s = (threadIdx.x & 31) < blockDim.x / 32 ? red[threadIdx.x & 31] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}

// Where CTA `cta` of the split begins: all units, its range [u, end), and the request
// that holds u with the units before that request.  Every thread of the block
// calls it; block sums and one scan per blockDim requests.
struct Start {
    int64_t u, end, before, units;
    int32_t b;
};
struct StartScratch {
    int64_t red[32];
    int64_t before;
    int32_t b;
};
__device__ __forceinline__ Start find_start(const Params &p, int64_t cta, StartScratch *s, bool *any_bad) {
    bool bad;
    int64_t mine = 0, n = 0;
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
        n = request_units(p, load_request<true>(p, b, &bad));
        *any_bad |= bad;
        mine += n;
    }
    const int64_t units = block_sum(mine, s->red);
    Start o;
    const int64_t n_cta = split_ctas(p, units);
    o.u = o.end = o.before = 0;
    o.b = 0;
    o.units = units;
    if (cta >= n_cta) return o;
    o.u = range_start(cta, units, n_cta);
    o.end = range_start(cta + 1, units, n_cta);
    int64_t passed = 0;
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        if (p.batch > (int)blockDim.x)
            n = b < p.batch ? request_units(p, load_request<true>(p, b, &bad)) : 0;
        else if (b >= p.batch)
            n = 0;
        int64_t incl = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, k);
            if ((threadIdx.x & 31) >= (unsigned)k) incl += up;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 31) s->red[threadIdx.x >> 5] = incl;
        __syncthreads();
        int64_t total = 0, warps_before = 0;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) {
            if (w == (int)threadIdx.x / 32) warps_before = total;
            total += s->red[w];
        }
        const int64_t pre = passed + warps_before + incl - n;
        if (n > 0 && o.u >= pre && o.u < pre + n) {
            s->before = pre;
            s->b = b;
        }
        passed += total;
        if (o.u < passed) break;
    }
    __syncthreads();
    o.before = s->before;
    o.b = s->b;
    return o;
}

// Is key position l of a paged request seen by token i (absolute index row)?
__device__ __forceinline__ bool sees(const Params &p, const Request &r, int32_t i, int32_t l) {
    if (l >= r.len) return false;
    const int32_t j = l - r.ctx;
    if (j < 0) return true;
    if (!p.tree_mask) return j <= i;
    if (j >= 64 * p.mask_words) return false;
    return (__ldg(p.tree_mask + (int64_t)(r.t0 + i) * p.mask_words + (j >> 6)) >> (j & 63)) & 1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e of an exponent byte: a normal number.
__device__ __forceinline__ float pow2_byte(uint8_t b) {
    return __uint_as_float((uint32_t)(kv_exponent(b) + 127) << 23);
}

// Element loads as fp32.
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
    return __half2float(__half(h));
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

dflash2_status launch_simt(const DeviceInfo &di, Params p, bool paged, int32_t dtype,
                           int32_t kv_format, cudaStream_t st);
// attention_tc.cu: whether the tcgen05 kernel takes the call, and the call.
bool tc_takes(const Params &p, bool paged, int32_t dtype);
dflash2_status launch_tc(const DeviceInfo &di, const Params &p, bool paged, int32_t kv_format,
                         cudaStream_t st);
// attention_few.cu: the same call over an E4M3 cache, where few rows share the keys.
dflash2_status launch_few(const DeviceInfo &di, const Params &p, cudaStream_t st);
dflash2_status launch_combine(const DeviceInfo &di, const Params &p, int32_t dtype, cudaStream_t st);

}  // namespace attn
}  // namespace dflash2
