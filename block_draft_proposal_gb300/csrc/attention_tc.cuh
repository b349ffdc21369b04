// What the tcgen05 attention kernels share: inline PTX, the pieces of work that a
// CTA walks, and the values the guard took out.
#pragma once
#include "attention.cuh"
#include "tcgen05.cuh"

namespace dflash2 {
namespace attn {
namespace {

using dflash2::bar_wait;  // the wait of every role here

constexpr int kTile = 128;  // keys per tile

// ---- tensor-core helpers -----------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// D (+)= A[tmem] * B[smem], 16-bit inputs.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f16 instruction descriptor: bf16 or fp16 operands, fp32 accumulator,
// M = 128; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc16(bool f16, int n, bool b_mn) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// Shared-memory matrix descriptors with 128-byte swizzle: the low word holds the
// start address (and the leading offset), the high word is a constant.
//   K-major (Q, K): 8-row groups 1024 bytes apart.
//   MN-major (V [keys x kD], kD contiguous): column blocks of 64 are 128 keys x
//   128 bytes apart (leading offset), groups of 8 keys 1024 bytes.
constexpr uint32_t kKMajorHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kKMajorLo = 1u << 16;  // leading offset, unused with a swizzle
constexpr uint32_t kMnMajorHi = kKMajorHi;
// K-major codes: rows of 128 bytes as above, or of 64 bytes with the 64-byte swizzle
// (8-row groups 512 bytes apart).
template <int kD>
constexpr uint32_t kCodesHi = kD == 128 ? kKMajorHi : (512u >> 4) | (1u << 14) | (4u << 29);
constexpr uint32_t kMnMajorLo = (uint32_t)((kTile * 128) >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) { return (smem_addr & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) {
    return ((uint64_t)hi << 32) | lo;
}
// ---- pieces --------------------------------------------------------------------
// The key tiles [t0, t1) of one item, as the producer warp hands it to the other
// roles through a ring in shared memory.
constexpr int kPieces = 4, kPieceBytes = 64;  // the ring
struct alignas(16) Piece {
    Request rq;
    int32_t b, h;
    int32_t row0, n_rows;   // first row of the block, live rows (0: no more pieces)
    int32_t t0, t1;         // key tiles
    int32_t t1a;            // shared: the end of slot 0's tiles (prompt rows see fewer)
    int32_t guard_from;     // first tile with positions some row does not see
    int32_t slot;           // workspace slot, or -1: the whole item
    int32_t tok0, rem0;     // row0 / group, row0 % group
    int32_t pad;
    __device__ __forceinline__ bool shared() const { return n_rows > kTile; }
};
static_assert(sizeof(Piece) <= kPieceBytes, "piece");

// Paged: walks CTA blockIdx.x's range of units.
struct Walk {
    int64_t u, end, before, n, units;
    int32_t b;
    Request rq;
    Join join;  // the item that the range starts and does not end
    __device__ __forceinline__ void begin(const Params &p, const Start &s) {
        bool bad;
        join = Join{};
        u = s.u, end = s.end, before = s.before, b = s.b, units = s.units;
        n = 0;
        if (u < end) {
            rq = load_request<true>(p, b, &bad);
            n = request_units(p, rq);
        }
    }
    __device__ __forceinline__ void next(const Params &p, Piece *pc) {
        pc->n_rows = 0;
        while (u < end) {
            while (u >= before + n) {
                bool bad;
                before += n;
                ++b;
                rq = load_request<true>(p, b, &bad);
                n = request_units(p, rq);
            }
            const int32_t c = units_class(p, rq), tile = p.tile_units[c], start = p.item_units[c];
            const int32_t tiles = key_tiles(rq);
            const uint32_t worth = tiles * tile + start, nrb = row_blocks(p, rq);
            uint32_t item;
            int32_t o0;
            if (n < (1ll << 31)) {
                const uint32_t off = (uint32_t)(u - before);
                item = off / worth;
                o0 = (int32_t)(off - item * worth);
            } else {
                const int64_t off = u - before;
                item = (uint32_t)(off / worth);  // kv_heads * row blocks: below 2^31
                o0 = (int32_t)(off - (int64_t)item * worth);
            }
            const int32_t o1 = (int32_t)min((int64_t)worth, o0 + (end - u));
            u += o1 - o0;
            pc->t0 = (max(o0 - start, 0) + tile - 1) / tile;
            pc->t1 = (max(o1 - start, 0) + tile - 1) / tile;
            if (pc->t1 <= pc->t0) continue;  // no tile's first unit lies in the range
            pc->t1a = pc->t1;
            pc->rq = rq;
            pc->b = b;
            pc->h = (int32_t)(item / nrb);
            pc->row0 = (int32_t)(item - (uint32_t)pc->h * nrb) << p.row_shift;
            pc->n_rows = min(1 << p.row_shift, rq.t * p.group - pc->row0);
            pc->slot = pc->t0 == 0 && pc->t1 == tiles ? -1 : 2 * (int32_t)blockIdx.x + (pc->t0 == 0);
            pc->guard_from = rq.ctx / kTile;
            if (pc->slot >= 0 && pc->t0 == 0) {
                join.rows = pc->n_rows, join.row0 = pc->row0, join.t0 = rq.t0, join.h = pc->h;
                join.last = cta_of(u - o1 + start + (tiles - 1) * tile, units, split_ctas(p, units));
            }
            return;
        }
    }
};

// Bits j0 .. j0 + 31 of a node's mask words (bit k: it sees node j0 + k); nodes
// before 0 are context and seen.
__device__ __forceinline__ uint32_t tree_bits(const int64_t *words, int32_t n_words, int32_t j0) {
    if (j0 <= -32) return 0xFFFFFFFFu;
    if (j0 < 0) return (uint32_t)((uint64_t)__ldg(words) << -j0) | ((1u << -j0) - 1u);
    const int32_t w = j0 >> 6, s = j0 & 63;
    if (w >= n_words) return 0u;
    uint64_t x = (uint64_t)__ldg(words + w) >> s;
    if (s > 32 && w + 1 < n_words) x |= (uint64_t)__ldg(words + w + 1) << (64 - s);
    return (uint32_t)x;
}
// Bits of the positions first .. first + 31 that lie below `end`.
__device__ __forceinline__ uint32_t below(int32_t first, int32_t end) {
    const int32_t n = end - first;
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The positions first .. first + 31 that token i of the request sees.
template <bool kPaged>
__device__ __forceinline__ uint32_t seen_bits(const Params &p, const Request &rq, int32_t i, int32_t first) {
    const bool tree = kPaged && p.tree_mask;
    uint32_t w = below(first, min(rq.len, tree ? rq.len : rq.ctx + i + 1));
    if (tree && w)
        w &= tree_bits(p.tree_mask + (int64_t)(rq.t0 + i) * p.mask_words, p.mask_words, first - rq.ctx);
    return w;
}

// Values of the keys [l0, l1) that token i of the request sees and that are not
// finite, added to columns [col, col + cols) of a row as it was written (`part`:
// the row's first four sums of a partial slot, or `out`: the output row): what the guard warp took out.
// Rare, so one thread per row.
template <int kD, bool kE4M3, bool kPaged>
__device__ __noinline__ void add_poison(const Params &p, Request rq, int32_t b, int32_t h, int32_t i,
                                        int32_t l0, int32_t l1, int32_t col, int32_t cols,
                                        float *part, __nv_bfloat16 *out) {
    for (int32_t l = l0; l < l1; ++l) {
        if (kPaged ? !sees(p, rq, i, l) : l > i) continue;
        int64_t at;
        if (kPaged) {
            const int32_t pg = __ldg(p.page_table + (int64_t)b * p.max_pages + l / p.page_size);
            if (pg < 0 || pg >= p.num_pages) continue;
            at = (((int64_t)pg * p.kv_heads + h) * p.page_size + l % p.page_size) * kD;
        } else {
            at = (int64_t)(rq.t0 + l) * p.v_stride + (int64_t)h * kD;
        }
        for (int c = col; c < col + cols; ++c) {
            const float v = kE4M3 ? as_f32(__ldg((const uint8_t *)p.v + at + c))
                                  : as_f32(((const __nv_bfloat16 *)p.v)[at + c]);
            if (fabsf(v) <= 3.4e38f) continue;
            if (part)
                part[(int64_t)(c >> 2) * 4 * p.part_rows + (c & 3)] += v;
            else
                out[c] = __float2bfloat16_rn(__bfloat162float(out[c]) + v);
        }
    }
}

}  // namespace
}  // namespace attn
}  // namespace dflash2
