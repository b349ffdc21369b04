// Attention on the 5th-generation tensor cores: bf16 queries, head_dim 64 or
// 128, over a paged cache (bf16 rows or E4M3 codes) or packed bf16 prompts.
//
// One pass over the keys in tiles of 128 with the softmax's running base and
// sum.  A slot is one accumulator pair in TMEM: scores S [128 rows x 128 keys],
// overwritten by the weights P (16 bits), and sums O [128 rows x head_dim].
//
//   S = Q K^T          tcgen05.mma, Q and K from shared memory, K-major
//   P = 2^(z - base)   z = scale log2(e) S, one thread per row (no shuffles)
//   O += P V           tcgen05.mma, P from TMEM, V [keys x head_dim] as the
//                      MN-major B operand, as it lies in memory
//
// base follows the row's maximum lazily: O and the sum are rescaled only when
// the maximum has grown by more than 2^8 (weights stay below 2^8 and the sums
// are fp32, so nothing is lost), which leaves the accumulators alone in most
// tiles.
//
// There are two slots, each with a softmax warpgroup, so that one slot's
// exponentials run beside the other's MMAs:
//   shared:     a row block of up to 256 rows; slot s holds rows 128 s ..; both
//               take every key tile, so a key is loaded once for 256 rows.
//   alternate:  up to 128 rows; both slots hold the same rows and take the key
//               tiles in turn; their sums are joined at the end.
//
// Roles: warps 0-3 and 4-7 softmax of slots 0 and 1 (and the loads of Q and the
// epilogue); warp 8 issues the MMAs; warp 9 the TMA loads (one box per
// page and 64 columns); warps 10-11 guard the values (below); E4M3 adds warps
// 12-15, which widen codes to fp16 (exact) into the operand ring.
//
// What a row does not see must not reach it, but a product 0 * NaN would.  In the
// key tiles that hold masked positions the guard warps zero the rows past the
// end and every value that is not finite, and note that they found one; the
// epilogue then adds such values to the rows that do see them.
//
// E4M3.  S = q' k' with q' = q 2^-a in fp16 (a per row, so that |q'| < 2^8: exact
// for values within 2^-22 of the row's largest) and k' the codes, which fp16
// holds; z = S 2^ke 2^a scale log2(e).  A value row's scale goes into its weight:
// P = 2^(z - base) 2^ve 2^-x, where the row's integer x follows the largest
// 2^(z - base) 2^ve as lazily as base follows z, so that weights fit fp16
// whatever the scales are.  Both factors are powers of two: the sum of the weights
// does not depend on the values.
#include <type_traits>

#include "attention.cuh"

namespace dflash2 {
namespace attn {
namespace {

constexpr int kTile = 128;       // keys per tile, rows per slot
constexpr int kRowBlock = 256;
constexpr float kLazy = 8.0f;    // log2 growth of the maximum that forces a rescale
constexpr int kTopE4M3 = 6;      // fp16 weights: the largest starts in [2^6, 2^7) ...
constexpr int kCapE4M3 = 14;     // ... and x moves once one reaches 2^14 or more
constexpr int kNoShift = -1000;  // no weight yet

// Barriers and small state, behind the operand rings in dynamic shared memory.
struct Shared {
    uint64_t full[8], empty[8];  // operand ring (E4M3: filled by the widening warps)
    uint64_t guard_go, guard_done;  // a value tile handed to the guard warps and back
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t q_full, drain;
    uint32_t tmem;
    int abort_flag;
    int poison;                  // number of the last piece with a value not finite
    StartScratch start;
};
struct SharedE4M3 : Shared {
    uint64_t raw_full[6], raw_empty[6];      // code ring
    uint64_t sc_full[4];                     // scales of a key tile
    float qmul[2][kRowBlock];                // 2^a scale log2(e) of a row, by piece parity
    alignas(16) uint8_t exps[6][2][kTile];   // exponent bytes as copied, by the keys' code-ring slot
    alignas(16) float kmul[4][kTile];        // 2^ke of a key, 4 tiles
    alignas(16) float vmul[4][kTile];        // 2^ve
};

template <int kD, bool kE4M3> struct Cfg {
    using Sh = std::conditional_t<kE4M3, SharedE4M3, Shared>;
    static constexpr int kHalves = kD / 64;            // 128-byte column blocks of a 16-bit tile
    static constexpr int kTileBytes = kTile * kD * 2;  // a 16-bit operand tile
    static constexpr int kRawBytes = kTile * kD;       // E4M3 codes of a tile
    static constexpr int kStages = kE4M3 ? 3 : (kD == 128 ? 5 : 8);
    static constexpr int kRaw = kE4M3 ? (kD == 128 ? 3 : 6) : 0;
    static constexpr int kThreads = kE4M3 ? 512 : 384;
    // registers: softmax warps take what the others give back
    static constexpr int kRegsMany = kE4M3 ? 192 : 216, kRegsFew = kE4M3 ? 64 : 72;
    static constexpr int kSmem =
        2 * kTileBytes + kStages * kTileBytes + kRaw * kRawBytes + (int)sizeof(Sh) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// ---- tensor-core helpers -----------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
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
// B operand [keys x kD], kD contiguous, 128-byte swizzle: column blocks of 64
// are 128 keys x 128 bytes apart, groups of 8 keys 1024 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((kTile * 128) >> 4) << 16;  // leading offset: next 64 columns
    d |= (uint64_t)(1024 >> 4) << 32;           // stride offset: next 8 keys
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// 32 TMEM columns of this warp's lanes; the registers are valid after
// tmem_ld_wait, which takes them so that no use moves ahead of it.
#define DF_R32(r)                                                                                  \
    r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], r[12], r[13], r[14], \
        r[15], r[16], r[17], r[18], r[19], r[20], r[21], r[22], r[23], r[24], r[25], r[26], r[27], \
        r[28], r[29], r[30], r[31]
#define DF_OUT32(c, r)                                                                             \
    c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7]), c(r[8]), c(r[9]),      \
        c(r[10]), c(r[11]), c(r[12]), c(r[13]), c(r[14]), c(r[15]), c(r[16]), c(r[17]), c(r[18]),  \
        c(r[19]), c(r[20]), c(r[21]), c(r[22]), c(r[23]), c(r[24]), c(r[25]), c(r[26]), c(r[27]),  \
        c(r[28]), c(r[29]), c(r[30]), c(r[31])
#define DF_SET(x) "=r"(x)
#define DF_TIE(x) "+r"(x)
#define DF_USE(x) "r"(x)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : DF_OUT32(DF_SET, r)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_tie(uint32_t (&r)[32]) {
    asm volatile("" : DF_OUT32(DF_TIE, r));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::DF_OUT32(
            DF_USE, r),
        "r"(taddr)
        : "memory");
}

// Register split of a warpgroup, inside its branch (ptxas allots a branch what it sees there).
template <int kN> __device__ __forceinline__ void regs_give() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN> __device__ __forceinline__ void regs_take() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kId, int kCount> __device__ __forceinline__ void named_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kCount) : "memory");
}

template <bool kF16> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// ---- pieces --------------------------------------------------------------------
// The key tiles [t0, t1) of one item.
struct Piece {
    Request rq;
    int32_t b, h;
    int32_t row0, n_rows;  // first row of the block, live rows
    int32_t t0, t1;        // key tiles
    int32_t t1a;           // shared: the end of slot 0's tiles (prompt rows see fewer)
    int32_t guard_from;    // first tile with positions some row does not see
    bool shared;
    int64_t slot;          // workspace slot, or -1: the whole item
};

__device__ __forceinline__ void finish_piece(const Params &p, Piece *pc, int32_t first_masked) {
    pc->shared = pc->n_rows > kTile;
    pc->guard_from = first_masked / kTile;  // tile [128 g, 128 g + 128) reaches past first_masked - 1
}

// Paged: walks CTA blockIdx.x's range of units.
struct Walk {
    int64_t u, end, before, n;
    int32_t b;
    Request rq;
    __device__ __forceinline__ void begin(const Params &p, const Start &s) {
        bool bad;
        u = s.u, end = s.end, before = s.before, b = s.b;
        n = 0;
        if (u < end) {
            rq = load_request<true>(p, b, &bad);
            n = request_units(p, rq);
        }
    }
    __device__ __forceinline__ bool next(const Params &p, Piece *pc) {
        if (u >= end) return false;
        while (u >= before + n) {
            bool bad;
            before += n;
            ++b;
            rq = load_request<true>(p, b, &bad);
            n = request_units(p, rq);
        }
        const int32_t tiles = key_tiles(rq), nrb = row_blocks(p, rq);
        const int64_t item = (u - before) / tiles;
        pc->t0 = (int32_t)((u - before) % tiles);
        pc->t1 = (int32_t)min((int64_t)tiles, pc->t0 + (end - u));
        pc->t1a = pc->t1;
        pc->rq = rq;
        pc->b = b;
        pc->h = (int32_t)(item / nrb);
        pc->row0 = (int32_t)(item % nrb) * kRowBlock;
        pc->n_rows = min(kRowBlock, rq.t * p.group - pc->row0);
        pc->slot = pc->t0 == 0 && pc->t1 == tiles ? -1 : 2 * (int64_t)blockIdx.x + (pc->t0 == 0);
        finish_piece(p, pc, rq.ctx);
        u += pc->t1 - pc->t0;
        return true;
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

// The positions of key tile `tile` that token i of the request sees.
template <bool kPaged>
__device__ __forceinline__ void seen_bits(const Params &p, const Request &rq, int32_t i,
                                          int32_t tile, uint32_t (&w)[4]) {
    const bool tree = kPaged && p.tree_mask;
    const int32_t end = min(rq.len, tree ? rq.len : rq.ctx + i + 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int32_t first = tile * kTile + 32 * k;
        w[k] = below(first, end);
        if (tree && w[k])
            w[k] &= tree_bits(p.tree_mask + (int64_t)(rq.t0 + i) * p.mask_words, p.mask_words,
                              first - rq.ctx);
    }
}

// Values of the keys [l0, l1) that token i of the request sees and that are not
// finite, added to columns [col, col + cols) of a row as it was written (a
// partial row of fp32 sums, or the output row): what the guard warps took out.
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
                part[c] += v;
            else
                out[c] = __float2bfloat16_rn(__bfloat162float(out[c]) + v);
        }
    }
}

// ---- the kernel ------------------------------------------------------------------
template <int kD, bool kE4M3, bool kPaged>
__global__ void __launch_bounds__(Cfg<kD, kE4M3>::kThreads, 1)
    tc_kernel(const Params p, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<kD, kE4M3>;
    constexpr int kStages = C::kStages;
    constexpr int kRaw = kE4M3 ? C::kRaw : 1;
    extern __shared__ uint8_t dyn[];
    const uint32_t pad = (0u - smem_u32(dyn)) & 1023u;
    const uint32_t sm_q = smem_u32(dyn) + pad;
    const uint32_t sm_ring = sm_q + 2 * C::kTileBytes;
    const uint32_t sm_raw = sm_ring + kStages * C::kTileBytes;
    auto &sh = *reinterpret_cast<typename C::Sh *>(
        dyn + pad + (2 + kStages) * C::kTileBytes + C::kRaw * C::kRawBytes);
    // alternate: each slot's (base, sum, 2^x) per row, in the second query tile, which that mode leaves unused
    float *stat = reinterpret_cast<float *>(dyn + pad + C::kTileBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], kE4M3 ? 128 : 1);
            mbar_init(&sh.empty[i], 1);
        }
        if constexpr (kE4M3) {
            for (int i = 0; i < kRaw; ++i) {
                mbar_init(&sh.raw_full[i], 1);
                mbar_init(&sh.raw_empty[i], 128);
            }
            for (int i = 0; i < 4; ++i) mbar_init(&sh.sc_full[i], 128);
        }
        mbar_init(&sh.guard_go, 1);
        mbar_init(&sh.guard_done, 64);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.q_full, 256);
        mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        sh.poison = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    grid_dep_wait();
    grid_dep_launch();

    // ---- what this CTA does ----
    bool bad = false;
    Start start{};
    Piece only{};
    bool have = false;
    if constexpr (kPaged) {
        start = find_start(p, &sh.start, &bad);
    } else {
        // CTA (x, h): row block number `want` of all requests, the last ones first
        int64_t want = (int64_t)gridDim.x - 1 - blockIdx.x;
        for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
            const int b = b0 + threadIdx.x;
            Request r{};
            bool bd = false;
            if (b < p.batch) r = load_request<false>(p, b, &bd);
            bad |= bd;
            const int64_t n = b < p.batch ? row_blocks(p, r) : 0;
            const int64_t total = block_sum(n, sh.start.red);
            if (want >= total) {
                want -= total;
                continue;
            }
            for (int i = b0; i < min(p.batch, b0 + (int)blockDim.x); ++i) {
                r = load_request<false>(p, i, &bd);
                const int32_t nb = row_blocks(p, r);
                if (want < nb) {
                    only.rq = r;
                    only.b = i;
                    only.h = blockIdx.y;
                    only.row0 = (int32_t)want * kRowBlock;
                    only.n_rows = (int32_t)min((int64_t)kRowBlock, (int64_t)r.t * p.group - only.row0);
                    const int32_t last = (only.row0 + only.n_rows - 1) / p.group;
                    const int32_t last0 = (only.row0 + min(only.n_rows, kTile) - 1) / p.group;
                    only.t0 = 0;
                    only.t1 = last / kTile + 1;
                    only.t1a = last0 / kTile + 1;
                    only.slot = -1;
                    finish_piece(p, &only, only.row0 / p.group);
                    have = true;
                    break;
                }
                want -= nb;
            }
            break;
        }
    }
    if (bad && p.err && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *abort_flag = &sh.abort_flag;

    Walk walk{};
    if constexpr (kPaged) walk.begin(p, start);
    auto next_piece = [&](Piece *pc) -> bool {
        if constexpr (kPaged) return walk.next(p, pc);
        if (!have) return false;
        *pc = only;
        have = false;
        return true;
    };
    Piece pc{};
    if (warp >= 8 && warp < 12) {
        regs_give<C::kRegsFew>();
        if (warp == 9) {
        // ---- TMA producer ----
        uint32_t pos = 0;  // operand tiles issued
        bool ok = true;
        const int32_t rows_box = kPaged ? min(p.page_size, kTile) : kTile;
        const int32_t n_box = kTile / rows_box;
        const int32_t per_page = kPaged ? max(1, p.page_size / kTile) : 1;  // tiles per page
        bool bad_page = false;
        auto full_bar = [&](uint32_t s) -> uint64_t * {
            if constexpr (kE4M3)
                return &sh.raw_full[s];
            else
                return &sh.full[s];
        };
        auto load = [&](int32_t tile, bool values) {
            constexpr uint32_t kSlots = kE4M3 ? kRaw : kStages;
            const uint32_t s = pos % kSlots, ph = (pos / kSlots) & 1u;
            uint64_t *fullb = full_bar(s), *emptyb;
            if constexpr (kE4M3)
                emptyb = &sh.raw_empty[s];
            else
                emptyb = &sh.empty[s];
            int32_t z = -1, y = 0, pg = 0;
            const int32_t l = tile * kTile + lane * rows_box;
            if constexpr (kPaged) {
                if (lane < n_box && l < pc.rq.len) {
                    pg = __ldg(p.page_table + (int64_t)pc.b * p.max_pages + l / p.page_size);
                    if (pg < 0 || pg >= p.num_pages) {
                        bad_page = true;
                        pg = 0;
                    } else {
                        z = pg * p.kv_heads + pc.h;
                    }
                }
                y = per_page > 1 ? (tile % per_page) * kTile : 0;
            }
            if (!mbar_wait(emptyb, ph ^ 1u, abort_flag, p.err)) return false;
            constexpr uint32_t kBytes = kE4M3 ? C::kRawBytes : C::kTileBytes;
            const bool with_exps = kE4M3 && !values;
            if (lane == 0) mbar_arrive_expect_tx(fullb, kBytes + (with_exps ? 2 * kTile : 0));
            __syncwarp();
            const CUtensorMap *map = values ? &vmap : &kmap;
            const int box = lane % n_box, half = lane / n_box;
            const int32_t zz = __shfl_sync(0xFFFFFFFFu, z, box);
            if constexpr (kE4M3) {
                if (lane < n_box) {
                    tma_load_3d(sm_raw + s * C::kRawBytes + lane * rows_box * kD, map, fullb, 0, y, z);
                    if (with_exps) {  // of page 0 where there is no page: any scale serves zero rows
                        const int64_t at = ((int64_t)pg * p.kv_heads + pc.h) * p.page_size + y;
                        bulk_load(smem_u32(&sh.exps[s][0][lane * rows_box]), p.k_exp + at, rows_box, fullb);
                        bulk_load(smem_u32(&sh.exps[s][1][lane * rows_box]), p.v_exp + at, rows_box, fullb);
                    }
                }
            } else if (lane < n_box * C::kHalves) {
                const uint32_t dst = sm_ring + s * C::kTileBytes + half * (kTile * 128) + box * rows_box * 128;
                if constexpr (kPaged)
                    tma_load_3d(dst, map, fullb, 64 * half, y, zz);
                else
                    tma_load_3d(dst, map, fullb, 64 * half, pc.h, pc.rq.t0 + tile * kTile);
            }
            __syncwarp();
            ++pos;
            return true;
        };
        while (ok && next_piece(&pc)) {
            if (pc.shared) {
                for (int32_t t = pc.t0; ok && t < pc.t1; ++t) ok = load(t, false) && load(t, true);
            } else {
                ok = load(pc.t0, false);
                for (int32_t t = pc.t0; ok && t < pc.t1; ++t)
                    ok = (t + 1 >= pc.t1 || load(t + 1, false)) && load(t, true);
            }
        }
        if (bad_page && p.err) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
        if (!ok) {  // wait for the copies in flight before the shared memory goes
            constexpr uint32_t kSlots = kE4M3 ? kRaw : kStages;
            for (uint32_t n = pos > kSlots ? pos - kSlots : 0; n < pos; ++n) {
                uint64_t *fullb = full_bar(n % kSlots);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(fullb, (n / kSlots) & 1u))
                    if (global_timer_ns() - t0 > kWaitLimitNs) break;
            }
        }
    } else if (warp == 8) {
        // ---- MMA issuer: lane 0 issues, the warp waits together ----
        constexpr uint32_t kIdS = idesc16(kE4M3, kTile, false);
        constexpr uint32_t kIdO = idesc16(kE4M3, kD, true);
        uint32_t pos = 0, n_piece = 0, n_guard = 0;
        uint32_t n_p[2] = {0, 0};
        const uint64_t qd[2] = {sw128_desc(sm_q), sw128_desc(sm_q + C::kTileBytes)};
        bool ok = true;
        auto wait_ring = [&](uint32_t n) {
            if (!mbar_wait(&sh.full[n % kStages], (n / kStages) & 1u, abort_flag, p.err)) return false;
            tc_fence_after();
            return true;
        };
        auto release = [&](uint32_t n) {
            if (lane == 0) tc_commit(&sh.empty[n % kStages]);
        };
        auto mma_s = [&](int s, int q, uint32_t n) {
            if (lane == 0) {
                const uint64_t kd = sw128_desc(sm_ring + (n % kStages) * C::kTileBytes);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t off = (k >> 2) * ((kTile * 128) >> 4) + (k & 3) * 2;
                    tc_mma_bf16(tmem + s * kTile, qd[q] + off, kd + off, kIdS, k > 0);
                }
                tc_commit(&sh.s_full[s]);
            }
            __syncwarp();
        };
        auto mma_o = [&](int s, uint32_t n, bool acc) {
            if (!mbar_wait(&sh.p_full[s], n_p[s] & 1u, abort_flag, p.err)) return false;
            ++n_p[s];
            tc_fence_after();
            if (lane == 0) {
                const uint64_t vd = mn_desc(sm_ring + (n % kStages) * C::kTileBytes);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc_mma_ts(tmem + 256 + s * kD, tmem + s * kTile + 8 * k, vd + k * (2048 >> 4), kIdO,
                              acc || k > 0);
            }
            __syncwarp();
            return true;
        };
        auto wait_v = [&](int32_t t, uint32_t n) {
            if (!wait_ring(n)) return false;
            if (!kE4M3 && t >= pc.guard_from) {
                if (lane == 0) mbar_arrive(&sh.guard_go);
                __syncwarp();
                if (!mbar_wait(&sh.guard_done, n_guard & 1u, abort_flag, p.err)) return false;
                ++n_guard;
            }
            return true;
        };
        while (ok && next_piece(&pc)) {
            ok = mbar_wait(&sh.q_full, n_piece & 1u, abort_flag, p.err);
            ++n_piece;
            tc_fence_after();
            if (!ok) break;
            if (pc.shared) {
                ok = wait_ring(pos);
                if (!ok) break;
                mma_s(0, 0, pos);
                mma_s(1, 1, pos);
                release(pos);
                for (int32_t t = pc.t0; ok && t < pc.t1; ++t) {
                    const uint32_t nv = pos + 1, nk = pos + 2;
                    const bool more = t + 1 < pc.t1;
                    ok = wait_v(t, nv);
                    if (!ok) break;
                    if (t < pc.t1a) {
                        ok = mma_o(0, nv, t > pc.t0);
                        if (!ok) break;
                    }
                    if (more) {
                        ok = wait_ring(nk);
                        if (!ok) break;
                    }
                    if (t + 1 < pc.t1a)
                        mma_s(0, 0, nk);
                    else if (t + 1 == pc.t1a && lane == 0)
                        tc_commit(&sh.o_full[0]);
                    ok = mma_o(1, nv, t > pc.t0);
                    if (!ok) break;
                    release(nv);
                    if (more) {
                        mma_s(1, 1, nk);
                        release(nk);
                    } else if (lane == 0) {
                        tc_commit(&sh.o_full[1]);
                    }
                    pos += 2;
                }
            } else {
                // tiles in turn; operand order K0 K1 V0 K2 V1 ...
                const int32_t n = pc.t1 - pc.t0;
                for (int32_t j = 0; ok && j < min(n, 2); ++j) {
                    ok = wait_ring(pos + j);
                    if (!ok) break;
                    mma_s(j, 0, pos + j);
                    release(pos + j);
                }
                for (int32_t j = 0; ok && j < n; ++j) {
                    // V(j) is operand 2 j + 2 of the piece, or the last one
                    const uint32_t nv = pos + (j + 1 < n ? 2 * j + 2 : 2 * n - 1);
                    const uint32_t nk = pos + 2 * j + 3;
                    ok = wait_v(pc.t0 + j, nv) && mma_o(j & 1, nv, j >= 2);
                    if (!ok) break;
                    release(nv);
                    if (j + 2 < n) {
                        ok = wait_ring(nk);
                        if (!ok) break;
                        mma_s(j & 1, 0, nk);
                        release(nk);
                    } else if (lane == 0) {
                        tc_commit(&sh.o_full[j & 1]);
                    }
                }
                pos += 2 * n;
            }
        }
        // nothing of this CTA's is in flight when the accumulators are freed
        if (lane == 0) tc_commit(&sh.drain);
        __syncwarp();
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&sh.drain, 0))
            if (global_timer_ns() - t0 > kWaitLimitNs) break;
    } else if (warp == 10 || warp == 11) {
        // ---- guard: values of tiles with masked positions ----
        if constexpr (!kE4M3) {
            uint32_t pos = 0, n_piece = 0, n_guard = 0;
            bool ok = true;
            const int tid = threadIdx.x - 320;
            while (ok && next_piece(&pc)) {
                ++n_piece;
                const int32_t n = pc.t1 - pc.t0;
                for (int32_t j = max(0, pc.guard_from - pc.t0); ok && j < n; ++j) {
                    const uint32_t nv = pos + (pc.shared ? 2 * j + 1 : j + 1 < n ? 2 * j + 2 : 2 * n - 1);
                    ok = mbar_wait(&sh.guard_go, n_guard & 1u, abort_flag, p.err);
                    if (!ok) break;
                    ++n_guard;
                    const uint32_t base = sm_ring + (nv % kStages) * C::kTileBytes;
                    const int32_t live = pc.rq.len - (pc.t0 + j) * kTile;  // rows of the tile that are keys
                    bool found = false;
                    for (int i = tid; i < C::kTileBytes / 16; i += 64) {
                        const uint32_t addr = base + i * 16;
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(addr));
                        bool change = false;
                        if (((i >> 3) & (kTile - 1)) >= live) {
                            change = true;
                            w[0] = w[1] = w[2] = w[3] = 0u;
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u, change = found = true;
                                if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0xFFFFu, change = found = true;
                            }
                        }
                        if (change)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]),
                                         "r"(w[1]), "r"(w[2]), "r"(w[3])
                                         : "memory");
                    }
                    if (found) *(volatile int *)&sh.poison = (int)n_piece;
                    fence_proxy_async_smem();
                    mbar_arrive(&sh.guard_done);
                }
                pos += 2 * n;
            }
        }
    }
    } else if (warp >= 12) {
        // ---- E4M3: codes to fp16, rows past the end to zero, scales to fp32 ----
        regs_give<C::kRegsFew>();
        if constexpr (kE4M3) {
            uint32_t pos = 0, n_piece = 0, tiles_done = 0;
            bool ok = true;
            const int row = threadIdx.x - 384;
            auto widen = [&](int32_t tile, bool values, uint32_t key_no) {
                const uint32_t rs = pos % kRaw, s = pos % kStages;
                if (!mbar_wait(&sh.raw_full[rs], (pos / kRaw) & 1u, abort_flag, p.err)) return false;
                if (!mbar_wait(&sh.empty[s], ((pos / kStages) & 1u) ^ 1u, abort_flag, p.err)) return false;
                const uint32_t src = sm_raw + rs * C::kRawBytes + row * kD;
                const uint32_t dst = sm_ring + s * C::kTileBytes + row * 128;
                const bool live = tile * kTile + row < pc.rq.len;
                const bool guarded = values && tile >= pc.guard_from;
                if (!values) {
                    // written exponents lie in [-48, 48]; what was never written is masked
                    const int ke = min(max((int)sh.exps[rs][0][row] - 127, -48), 48);
                    const int ve = min(max((int)sh.exps[rs][1][row] - 127, -48), 48);
                    const uint32_t ss = key_no & 3u;
                    sh.kmul[ss][row] = __uint_as_float((uint32_t)(ke + 127) << 23);
                    sh.vmul[ss][row] = __uint_as_float((uint32_t)(ve + 127) << 23);
                    mbar_arrive(&sh.sc_full[ss]);
                }
                bool found = false;
#pragma unroll
                for (int c = 0; c < kD / 16; ++c) {
                    // 16 codes; the copy's swizzle spreads the rows' chunks over the banks
                    const uint32_t a =
                        src + ((kD == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(a));
                    if (values && !live) w[0] = w[1] = w[2] = w[3] = 0u;
                    if (guarded && live) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t nan = __vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            if (nan) found = true, w[k] &= ~nan;
                        }
                    }
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(w[k] & 0xFFFFu), __NV_E4M3);
                        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(w[k] >> 16), __NV_E4M3);
                        o[2 * k] = (uint32_t)lo.x | ((uint32_t)lo.y << 16);
                        o[2 * k + 1] = (uint32_t)hi.x | ((uint32_t)hi.y << 16);
                    }
                    const uint32_t d0 = dst + (c >> 2) * (kTile * 128);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         d0 + (((2 * (c & 3) + k) ^ (row & 7)) << 4)),
                                     "r"(o[4 * k]), "r"(o[4 * k + 1]), "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                                     : "memory");
                }
                if (found) *(volatile int *)&sh.poison = (int)n_piece;
                mbar_arrive(&sh.raw_empty[rs]);
                fence_proxy_async_smem();
                mbar_arrive(&sh.full[s]);
                ++pos;
                return true;
            };
            while (ok && next_piece(&pc)) {
                ++n_piece;
                const int32_t n = pc.t1 - pc.t0;
                if (pc.shared) {
                    for (int32_t j = 0; ok && j < n; ++j)
                        ok = widen(pc.t0 + j, false, tiles_done + j) && widen(pc.t0 + j, true, 0);
                } else {
                    ok = widen(pc.t0, false, tiles_done);
                    for (int32_t j = 0; ok && j < n; ++j)
                        ok = (j + 1 >= n || widen(pc.t0 + j + 1, false, tiles_done + j + 1)) &&
                             widen(pc.t0 + j, true, 0);
                }
                tiles_done += n;
            }
        }
    } else {
        // ---- softmax of slot s, with the loads of Q and the epilogue ----
        regs_take<C::kRegsMany>();
        const int s = warp >> 2;
        const int wq = warp & 3;
        const int my = wq * 32 + lane;  // row within the slot
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + s * kTile + lane_base;
        uint32_t n_piece = 0, n_s = 0, tiles_done = 0;
        uint32_t n_o[2] = {0, 0};
        bool ok = true;
        // a negative scale negates Q; with scale 0 Q counts as zeros (masked scores are
        // -inf and must not meet a factor 0)
        const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
        const uint32_t keep = p.scale_log2 == 0.0f ? 0u : 0xFFFFFFFFu;
        const float mul = p.scale_log2 == 0.0f ? 1.0f : fmaxf(fabsf(p.scale_log2), 1.1754944e-38f);
        while (ok && next_piece(&pc)) {
            ++n_piece;
            // queries: kD / 8 lanes hold a row, 8 values each
            {
                constexpr int kLanes = kD / 8;
                const int l8 = threadIdx.x % kLanes;
                for (int r = threadIdx.x / kLanes; r < pc.n_rows; r += 256 / kLanes) {
                    const int32_t g = pc.row0 + r;
                    const __nv_bfloat16 *src = (const __nv_bfloat16 *)p.q +
                                               (int64_t)(pc.rq.t0 + g / p.group) * p.q_stride +
                                               (int64_t)(pc.h * p.group + g % p.group) * kD + l8 * 8;
                    uint4 v = __ldg(reinterpret_cast<const uint4 *>(src));
                    uint32_t w[4] = {(v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep,
                                     (v.w ^ flip) & keep};
                    if constexpr (kE4M3) {
                        float f[8], amax = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            f[2 * k] = __uint_as_float(w[k] << 16);
                            f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
                            amax = fmaxf(amax, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
                        }
                        const uint32_t group_mask =
                            (kLanes == 32 ? 0xFFFFFFFFu : ((1u << kLanes) - 1u)) << (lane & ~(kLanes - 1));
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o >>= 1)
                            amax = fmaxf(amax, __shfl_xor_sync(group_mask, amax, o));
                        // 2^-a: the largest magnitude's binade becomes 2^7
                        const int a = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -110), 110);
                        const float down = __uint_as_float((uint32_t)(127 - a) << 23);
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = pack16<true>(f[2 * k] * down, f[2 * k + 1] * down);
                        if (l8 == 0)
                            sh.qmul[n_piece & 1u][r] =
                                fmaxf(__uint_as_float((uint32_t)(127 + a) << 23) * mul, 1.1754944e-38f);
                    }
                    const int c = l8 & 7, half = l8 >> 3;
                    const uint32_t dst = sm_q + (r >> 7) * C::kTileBytes + half * (kTile * 128) +
                                         (r & 127) * 128 + ((c ^ (r & 7)) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]),
                                 "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                mbar_arrive(&sh.q_full);
                if constexpr (kE4M3) named_sync<1, 256>();  // the rows' scales
            }
            const int32_t r_blk = (pc.shared ? s * kTile : 0) + my;  // row within the block
            const int32_t r_req = pc.row0 + r_blk;
            const int32_t tok = r_req / p.group;
            const bool live_row = r_blk < pc.n_rows;
            const bool live_warp = (pc.shared ? s * kTile : 0) + wq * 32 < pc.n_rows;
            float qm = mul;
            if constexpr (kE4M3) qm = live_row ? sh.qmul[n_piece & 1u][r_blk] : 0.0f;
            const int32_t first_tok = (pc.row0 + (pc.shared ? s * kTile : 0)) / p.group;
            // positions below this one are seen by every row of the slot
            const int32_t all_seen = kPaged ? pc.rq.ctx : first_tok + 1;
            const int32_t t_end = pc.shared && s == 0 ? pc.t1a : pc.t1;
            const int32_t step = pc.shared ? 1 : 2;
            float base = -INFINITY, sum = 0.0f;
            int shift = kNoShift;  // E4M3: x
            const uint32_t tO = tmem + 256 + s * kD + lane_base;
            bool first = true;
            for (int32_t t = pc.t0 + (pc.shared ? 0 : s); t < t_end; t += step) {
                const uint32_t sc = (tiles_done + (uint32_t)(t - pc.t0));
                if constexpr (kE4M3) {
                    ok = mbar_wait(&sh.sc_full[sc & 3u], (sc >> 2) & 1u, abort_flag, p.err);
                    if (!ok) break;
                }
                ok = mbar_wait(&sh.s_full[s], n_s & 1u, abort_flag, p.err);
                if (!ok) break;
                ++n_s;
                tc_fence_after();
                if (live_warp) {
                    uint32_t x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, x[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_tie(x[c]);
                    if constexpr (kE4M3) {
                        const float *km = sh.kmul[sc & 3u];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(km + 32 * c + k);
                                x[c][k] = __float_as_uint(__uint_as_float(x[c][k]) * f.x);
                                x[c][k + 1] = __float_as_uint(__uint_as_float(x[c][k + 1]) * f.y);
                                x[c][k + 2] = __float_as_uint(__uint_as_float(x[c][k + 2]) * f.z);
                                x[c][k + 3] = __float_as_uint(__uint_as_float(x[c][k + 3]) * f.w);
                            }
                    }
                    if ((t + 1) * kTile > all_seen) {
                        uint32_t w[4] = {0, 0, 0, 0};
                        if (live_row) seen_bits<kPaged>(p, pc.rq, tok, t, w);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((w[c] >> k) & 1u)) x[c][k] = 0xFF800000u;  // -inf
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k) top[k & 3] = fmaxf(top[k & 3], __uint_as_float(x[c][k]));
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * qm;
                    const bool grow = mx > base + kLazy;
                    const float nb = grow ? mx : base;
                    const float safe = nb == -INFINITY ? 0.0f : nb;
                    // grow: base was -inf (fix = 0, nothing summed yet) or finite
                    float fix = grow ? ex2(base - nb) : 1.0f;
                    bool move = grow;
                    base = nb;
                    sum *= fix;
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    float down = 1.0f;  // 2^-x
                    if constexpr (kE4M3) {
                        const float *vm = sh.vmul[sc & 3u];
                        float hi[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(vm + 32 * c + k);
                                const float v4[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float w = ex2(fmaf(__uint_as_float(x[c][k + e]), qm, -safe));
                                    part[e] += w;
                                    const float u = w * v4[e];
                                    hi[e] = fmaxf(hi[e], u);
                                    x[c][k + e] = __float_as_uint(u);
                                }
                            }
                        const float h = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
                        const int e = (int)(__float_as_uint(h) >> 23) - 127;
                        const bool had = shift != kNoShift;
                        if (h > 0.0f && e - shift >= kCapE4M3) {
                            const int ns = max(e - kTopE4M3, -100);
                            fix = had ? fix * ex2((float)(shift - ns)) : 0.0f;
                            shift = ns;
                            move = true;
                        }
                        down = shift == kNoShift ? 1.0f : __uint_as_float((uint32_t)(127 - shift) << 23);
                    }
                    if (!first && __any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
                        for (int c = 0; c < kD / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * c, o);
                            tmem_ld_wait();
                            tmem_tie(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
                            tmem_st32(tO + 32 * c, o);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int c = 2 * h + (k >> 4), e = (2 * k) & 31;
                            if constexpr (kE4M3) {
                                pk[k] = pack16<true>(__uint_as_float(x[c][e]) * down,
                                                     __uint_as_float(x[c][e + 1]) * down);
                            } else {
                                const float a = ex2(fmaf(__uint_as_float(x[c][e]), qm, -safe));
                                const float b = ex2(fmaf(__uint_as_float(x[c][e + 1]), qm, -safe));
                                part[k & 1] += a;
                                part[2 + (k & 1)] += b;
                                pk[k] = pack16<false>(a, b);
                            }
                        }
                        tmem_st32(tS + 32 * h, pk);
                    }
                    sum += (part[0] + part[1]) + (part[2] + part[3]);
                    tmem_st_wait();
                    first = false;
                }
                tc_fence_before();
                mbar_arrive(&sh.p_full[s]);
            }
            if (!ok) break;
            // ---- epilogue ----
            const int32_t n = pc.t1 - pc.t0;
            const bool used0 = true, used1 = pc.shared || n > 1;
            tiles_done += n;
            const float up = !kE4M3 || shift == kNoShift ? 1.0f : __uint_as_float((uint32_t)(127 + shift) << 23);
            float f0, f1 = 0.0f;
            int col0 = 0, cols = kD;
            if (pc.shared) {
                ok = mbar_wait(&sh.o_full[s], n_o[s] & 1u, abort_flag, p.err);
                if (!ok) break;
                f0 = up;
            } else {
                ok = mbar_wait(&sh.o_full[0], n_o[0] & 1u, abort_flag, p.err) &&
                     (!used1 || mbar_wait(&sh.o_full[1], n_o[1] & 1u, abort_flag, p.err));
                if (!ok) break;
                float *mine = stat + 3 * kTile * s + my;
                mine[0] = base;
                mine[kTile] = sum;
                mine[2 * kTile] = up;
                named_sync<1, 256>();
                const float *st0 = stat + my, *st1 = stat + 3 * kTile + my;
                const float b0 = st0[0], b1 = used1 ? st1[0] : -INFINITY;
                const float l0 = st0[kTile], l1 = used1 ? st1[kTile] : 0.0f;
                const float u0 = st0[2 * kTile], u1 = used1 ? st1[2 * kTile] : 0.0f;
                named_sync<1, 256>();  // both have read: the next piece's queries may come
                base = fmaxf(b0, b1);
                const float safe = base == -INFINITY ? 0.0f : base;
                f0 = ex2(b0 - safe);
                f1 = ex2(b1 - safe);
                sum = l0 * f0 + l1 * f1;
                f0 *= u0;
                f1 *= u1;
                cols = kD / 2;
                col0 = s * cols;
            }
            n_o[0] += used0;
            n_o[1] += used1;
            tc_fence_after();
            if (live_warp) {
                const bool poisoned = *(volatile int *)&sh.poison == (int)n_piece;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const int64_t row = (int64_t)(pc.rq.t0 + tok) * p.q_heads + pc.h * p.group + r_req % p.group;
                float *part = pc.slot >= 0 ? p.part + pc.slot * part_slot_floats(p.part_rows, kD) : nullptr;
                float *part_row = part ? part + (int64_t)r_blk * kD : nullptr;
                __nv_bfloat16 *out_row = (__nv_bfloat16 *)p.out + row * kD;
                const bool both = !pc.shared && used1;
                const uint32_t t0 = tmem + 256 + lane_base + (pc.shared && s == 1 ? kD : 0);
#pragma unroll 1
                for (int c0 = col0; c0 < col0 + cols; c0 += 32) {
                    uint32_t a[32];
                    tmem_ld32(t0 + c0, a);
                    tmem_ld_wait();
                    tmem_tie(a);
                    if (both) {
                        uint32_t b[32];
                        tmem_ld32(t0 + kD + c0, b);
                        tmem_ld_wait();
                        tmem_tie(b);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            a[k] = __float_as_uint(__uint_as_float(a[k]) * f0 + __uint_as_float(b[k]) * f1);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * f0);
                    }
                    if (!live_row) continue;
                    if (part) {
                        uint4 *dst = reinterpret_cast<uint4 *>(part_row + c0);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dst[k] = make_uint4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(out_row + c0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack16<false>(__uint_as_float(a[8 * k + 2 * e]) * inv,
                                                     __uint_as_float(a[8 * k + 2 * e + 1]) * inv);
                            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (poisoned && live_row)
                    add_poison<kD, kE4M3, kPaged>(p, pc.rq, pc.b, pc.h, tok,
                                                  max(pc.t0, pc.guard_from) * kTile,
                                                  min(pc.t1 * kTile, pc.rq.len), col0, cols, part_row, out_row);
                if (live_row && col0 == 0) {
                    if (part) {
                        part[(int64_t)p.part_rows * kD + r_blk] = base;
                        part[(int64_t)p.part_rows * (kD + 1) + r_blk] = sum;
                    } else if (p.lse) {
                        p.lse[row] = sum == 0.0f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
                    }
                }
            }
            // the sums are read: the next piece's q_full arrivals say so to the MMAs
            tc_fence_before();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int kD, bool kE4M3, bool kPaged>
dflash2_status launch_one(const DeviceInfo &di, Params p, cudaStream_t st) {
    using C = Cfg<kD, kE4M3>;
    auto fn = tc_kernel<kD, kE4M3, kPaged>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
        cudaGetLastError();
        return DFLASH2_ERR_CUDA;
    }
    CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {
        const void *base = i ? p.v : p.k;
        dflash2_status s;
        if constexpr (kPaged) {
            const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)p.page_size,
                                      (uint64_t)p.num_pages * p.kv_heads};
            const uint64_t el = kE4M3 ? 1 : 2;
            const uint64_t strides[2] = {kD * el, kD * el * p.page_size};
            const uint32_t box[3] = {kE4M3 ? (uint32_t)kD : 64u,
                                     (uint32_t)(p.page_size < kTile ? p.page_size : kTile), 1u};
            s = encode_tmap_3d(&maps[i], base, dims, strides, box, (uint32_t)el);
        } else {
            const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)p.kv_heads, (uint64_t)p.total_q};
            const uint64_t strides[2] = {kD * 2, (uint64_t)(i ? p.v_stride : p.k_stride) * 2};
            const uint32_t box[3] = {64u, 1u, (uint32_t)kTile};
            s = encode_tmap_3d(&maps[i], base, dims, strides, box, 2);
        }
        if (s != DFLASH2_OK) return s;
    }
    p.row_block = kRowBlock;
    p.n_cta = di.sm_count;
    dim3 grid((unsigned)p.n_cta);
    if (!kPaged)
        grid = dim3((unsigned)(((int64_t)p.total_q * p.group + kRowBlock - 1) / kRowBlock + p.batch),
                    (unsigned)p.kv_heads);
    launch_k(fn, grid, dim3(C::kThreads), C::kSmem, st, p, maps[0], maps[1]);
    const dflash2_status s = launch_status();
    if (s != DFLASH2_OK || !kPaged) return s;
    return launch_combine(di, p, DFLASH2_BF16, st);
}

bool rows16(const void *p, int64_t stride, int el) {
    return aligned16(p) && stride * el % 16 == 0;
}

}  // namespace

bool tc_takes(const Params &p, bool paged, int32_t dtype, int32_t kv_format) {
    if (dtype != DFLASH2_BF16 || (p.head_dim != 64 && p.head_dim != 128)) return false;
    if (!rows16(p.q, p.q_stride, 2) || !aligned16(p.out) || !aligned16(p.k) || !aligned16(p.v))
        return false;
    if (!paged) return rows16(p.k, p.k_stride, 2) && rows16(p.v, p.v_stride, 2);
    return p.page_size >= 16 && (p.page_size & (p.page_size - 1)) == 0 &&
           (kv_format == DFLASH2_KV_NATIVE || (aligned16(p.k_exp) && aligned16(p.v_exp)));
}

dflash2_status launch_tc(const DeviceInfo &di, const Params &p, bool paged, int32_t kv_format,
                         cudaStream_t st) {
    if (!paged)
        return p.head_dim == 64 ? launch_one<64, false, false>(di, p, st)
                                : launch_one<128, false, false>(di, p, st);
    if (kv_format == DFLASH2_KV_E4M3)
        return p.head_dim == 64 ? launch_one<64, true, true>(di, p, st)
                                : launch_one<128, true, true>(di, p, st);
    return p.head_dim == 64 ? launch_one<64, false, true>(di, p, st)
                            : launch_one<128, false, true>(di, p, st);
}

}  // namespace attn
}  // namespace dflash2
