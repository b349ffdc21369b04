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
// tiles.  It starts at the first tile's maximum, whose weight of 1 is exact: from a
// fixed base the first tile is not taken twice (255 us in place of 264 for the sixteen
// prompts below), but a row of few keys then carries its only weight's rounding (0.0023
// from 64 bits in place of 0.0020, over all rows).
//
// There are two slots, each with a softmax warpgroup, so that one slot's
// exponentials run beside the other's MMAs:
//   shared:     a row block of up to 256 rows; slot s holds rows 128 s ..; both
//               take every key tile, so a key is loaded once for 256 rows.
//   alternate:  up to 128 rows; both slots hold the same rows and take the key
//               tiles in turn; their sums are joined at the end.  With 64 or 32
//               rows or fewer the accumulator holds 2 or 4 copies of them, and each
//               copy's warps take the weights of their share of a tile's keys (zero
//               elsewhere), so that four warps work however few the rows are.
//
// Roles: warps 0-3 and 4-7 softmax of slots 0 and 1 (and the loads of Q and the
// epilogue); warps 8 and 10 issue the MMAs of slots 0 and 1; warp 9 the TMA loads
// (one box per page and 64 columns); warp 11 guards the values (below).  E4M3: warp 9
// loads the keys, warp 11 the values, and warps 12-19 widen value codes to fp16 into the
// operand ring.
//
// What a row does not see must not reach it, but a product 0 * NaN would.  In the
// key tiles that hold masked positions the guard warp zeroes the rows past the
// end and every value that is not finite, and note that they found one; the
// epilogue then adds such values to the rows that do see them.
//
// E4M3.  S = q' k' on the codes themselves, with q' = q 2^-a as two codes, the nearest
// one and that of the rest (a per row, so that |q'| < 2^8): together they hold the
// eight bits of a bf16 value down to 2^-10 of the row's largest, and 2^-18 of that
// below.  z = S 2^(key scale) 2^a scale log2(e).  Value codes are widened to fp16, which
// holds them, and a value row's scale goes into its weight: P = 2^(z - base)
// 2^(value scale) 2^-x, where the row's integer x follows the largest of them as
// lazily as base follows z, so that weights fit fp16 whatever the scales are.  All of
// these are powers of two: the sum of the weights does not depend on the values.
// (Requests of few rows go to attention_few.cu.)
//
// Measured, 8 key/value heads of 128.  Prompts, bound by the tensor pipe in the tiles (a
// tile for both slots 2500 to 2700 cycles, its MMAs 2048; the softmax's issue slots next)
// and by an item's start and end, some four tiles' time: one of 12001 tokens with 32
// heads 715 to 780 us with the clock under the power cap, 1.52 to 1.65 PFLOP/s; sixteen of
// 100 to 2048 tokens with 40 heads 269 us, the tensor pipe busy for 49 % of it.  Paged, starts,
// ends and joins beside: four trees of 64 tokens over 30011 to 60000 keys 152 to 169 us, 4.4 to
// 4.9 TB/s, bound by the tensor pipe and HBM alike (61 and 67 % busy); 32 blocks of 16 tokens
// over 500 to 8000 keys by HBM, 107 us, 5.3 TB/s.  What paid, in that order: the slots' MMAs in turns (3400 cycles a tile
// without), tiles in registers and the base kept from the tile before (no second pass),
// page numbers eight tiles ahead, queries copied asynchronously, output rows written
// whole.  More polling (test_wait) or less (a suspend hint) both cost.
#include <type_traits>

#include "attention_tc.cuh"

namespace dflash2 {
namespace attn {
namespace {

// A slot has kTile rows, a row block two slots.
constexpr int kRowShift = 8, kRowBlock = 1 << kRowShift;
// The split: units of a key tile, and an item's start and end in tiles.  A tile of more
// than 128 rows of an E4M3 cache counts for more, since the softmax bounds it (32 requests
// of 1 to 64 tokens over 100 to 6000 keys, 4 to 256 rows: 165 us, and 183 with 10 for all);
// over a bf16 cache HBM bounds either (109 us, and 114 with 17).
constexpr int kTileUnits = 10, kSharedUnits = 17, kItemTiles = 4;
constexpr float kLazy = 8.0f;    // log2 growth of the maximum that forces a rescale
constexpr int kTopE4M3 = 6;      // fp16 weights: the largest (or its bound) starts below 2^7 ...
constexpr int kCapE4M3 = 14;     // ... and x moves before one reaches 2^15
// ... and the bound (the tile's largest value scale times the row's largest weight, mostly of
// another key) is at most this many binades above what it stands for: the largest starts at 2^-2
// or more, where fp16's grid ends 2^-22 below it.  Where scales differ more, each weight is looked
// at (the 32 requests above, with values e^(s n) n', n and n' normal, s = 0.3, 1 and 2: 165, 179 and
// 216 us; at 22 binades in place of 8 165, 173 and 173, with the small weights lost).
constexpr int kWideE4M3 = 8;
constexpr int kNoShift = -1000;  // no weight yet

// Barriers and small state, behind the operand rings in dynamic shared memory.
struct TileScale {  // E4M3
    int32_t top;   // largest binary exponent of a tile's value scales
    int32_t wide;  // they span more than kWideE4M3 binades
};
constexpr int kMarks = 2 * kPieces;
__device__ __forceinline__ uint8_t poison_mark(uint32_t piece) { return (uint8_t)(piece / kMarks % 255 + 1); }
struct Shared {
    alignas(16) uint8_t piece[kPieces][kPieceBytes];
    int32_t pages[2][2][kTile / 16 * 8 + 1];  // page numbers of eight key tiles, twice, by producer
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t full[8], empty[8];  // operand ring (E4M3: filled by the widening warps)
    uint64_t guard_go[8], guard_done[8];  // value tiles on their way, for the guard warp, and back, in order
    uint64_t s_full[2], p_full[2][2], o_full[2];  // weights come in halves of 64 keys
    uint64_t turn[2];            // shared: whose sums' and next scores' MMAs come next
    uint64_t q_full, drain[2];
    uint32_t tmem;
    int abort_flag;
    int stop[3][2];              // no more pieces: softmax warps, widening warpgroups; by piece parity
    // The last pieces with a value not finite: entry i % kMarks holds piece i's mark.  Who finds
    // one may be kPieces pieces ahead of the epilogue that looks for its own (no piece is handed
    // out before all roles have taken the one kPieces before it).  An older piece with the same
    // mark is harmless: the epilogue looks for values and finds none.
    uint8_t poison[kMarks];
    StartScratch start;
};
template <int kTiles> struct SharedE4M3 : Shared {
    uint64_t kraw_full[4], kraw_empty[4];    // key codes, as the MMAs read them
    uint64_t vraw_full[4], vraw_empty[4];    // value codes, to be widened
    uint64_t sc_full[kTiles];                // scales of a tile, from the widening warps
    TileScale scale[kTiles];
    int reduce[2][2][4][2];                  // by widening warpgroup and its tile's parity
    float qmul[2][kRowBlock];                // 2^a scale log2(e) of a row, by piece parity
    alignas(16) float kmul[kTiles][kTile];   // 2^ke of the tiles' keys
    alignas(16) float vmul[kTiles][kTile];   // 2^ve
};

template <int kD, bool kE4M3> struct Cfg {
    static constexpr int kTileBytes = kTile * kD * 2;  // a 16-bit operand tile
    static constexpr int kRawBytes = kTile * kD;       // E4M3 codes of a tile
    // operand ring: keys and values in turn, or (E4M3) widened values alone
    static constexpr int kStages = kE4M3 ? (kD == 128 ? 2 : 4) : (kD == 128 ? 5 : 8);
    static constexpr int kKRaw = kE4M3 ? (kD == 128 ? 3 : 4) : 0, kVRaw = kE4M3 ? (kD == 128 ? 2 : 4) : 0;
    static constexpr int kRaw = kKRaw + kVRaw;
    // a tile's scales are written after the same warps' value operand of two tiles before,
    // which waited for the one kStages before that: kStages + 2 tiles at least
    static constexpr int kScales = kStages <= 2 ? 4 : 8;
    using Sh = std::conditional_t<kE4M3, SharedE4M3<kScales>, Shared>;
    static constexpr int kThreads = kE4M3 ? 640 : 384;
    // registers: softmax warps take what the others give back (E4M3: 96 each at launch, else
    // 168; with 72 for the others, the producer spills: 159 us in place of 152 for the four trees)
    static constexpr int kRegsMany = kE4M3 ? 144 : 208, kRegsFew = kE4M3 ? 64 : 88;
    // alternate: (base, sum, 2^x) of 2 x 128 accumulator rows and 128 reciprocal sums; head_dim
    // 128 has room for them in the second query tile, which that mode leaves unused
    static constexpr int kStatBytes = kD == 128 ? 0 : 7 * kTile * 4;
    static constexpr int kSmem =
        2 * kTileBytes + kStages * kTileBytes + kRaw * kRawBytes + (int)sizeof(Sh) + kStatBytes + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Prompts: row blocks with the most keys first.  Level j holds block j of every
// request that has one; the items are numbered level by level from the highest
// down, request by request, head by head, and CTA c takes number c of the first
// n_cta items, number n_cta - 1 - c of the next, and so on in turns, which evens the
// CTAs' key tiles out.  A warp walks; lane i looks at request 32 k + i.
struct Levels {
    int32_t round, level, above, total;  // row blocks in levels > `level`; blocks in all
    __device__ __forceinline__ int32_t blocks_of(const Params &p, int32_t b, Request *r) const {
        bool bad;
        *r = load_request<false>(p, b, &bad);
        return row_blocks(p, *r);
    }
    __device__ __forceinline__ int32_t in_level(const Params &p, int lane) const {
        int32_t n = 0;
        Request r;
        for (int b0 = 0; b0 < p.batch; b0 += 32)
            n += __popc(__ballot_sync(0xFFFFFFFFu,
                                      b0 + lane < p.batch && blocks_of(p, b0 + lane, &r) > level));
        return n;
    }
    __device__ __forceinline__ void begin(const Params &p, int lane, bool *bad) {
        int32_t most = 0, sum = 0;
        for (int b = lane; b < p.batch; b += 32) {
            bool bd;
            const Request r = load_request<false>(p, b, &bd);
            *bad |= bd;
            const int32_t n = row_blocks(p, r);
            most = max(most, n);
            sum += n;
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        total = __reduce_add_sync(0xFFFFFFFFu, sum);
        level = most - 1;
        above = 0;
        round = 0;
    }
    __device__ __forceinline__ void next(const Params &p, int lane, Piece *pc) {
        pc->n_rows = 0;
        const int32_t n_cta = (int32_t)gridDim.x;
        const int32_t c = (round & 1) ? n_cta - 1 - (int32_t)blockIdx.x : (int32_t)blockIdx.x;
        const int64_t item = (int64_t)round * n_cta + c;
        ++round;
        if (item >= (int64_t)total * p.kv_heads) return;
        const int32_t q = (int32_t)(item / p.kv_heads);
        int32_t here = in_level(p, lane);
        while (q >= above + here) {
            above += here;
            --level;
            here = in_level(p, lane);
        }
        int32_t k = q - above;  // the k-th request of the level
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            Request r{};
            const bool has = b0 + lane < p.batch && blocks_of(p, b0 + lane, &r) > level;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
            if (k >= __popc(m)) {
                k -= __popc(m);
                continue;
            }
            const int src = __fns(m, 0, k + 1);
            pc->rq.t0 = __shfl_sync(0xFFFFFFFFu, r.t0, src);
            pc->rq.t = __shfl_sync(0xFFFFFFFFu, r.t, src);
            pc->b = b0 + src;
            break;
        }
        pc->rq.len = pc->rq.t;
        pc->rq.ctx = 0;
        pc->h = (int32_t)(item - (int64_t)q * p.kv_heads);
        pc->row0 = level * kRowBlock;
        pc->n_rows = min(kRowBlock, pc->rq.t * p.group - pc->row0);
        pc->t0 = 0;
        pc->t1 = ((pc->row0 + pc->n_rows - 1) / p.group) / kTile + 1;
        pc->t1a = ((pc->row0 + min(pc->n_rows, kTile) - 1) / p.group) / kTile + 1;
        pc->guard_from = (pc->row0 / p.group) / kTile;
        pc->slot = -1;
    }
};

// ---- the kernel ------------------------------------------------------------------
template <int kD, bool kE4M3, bool kPaged>
__global__ void __launch_bounds__(Cfg<kD, kE4M3>::kThreads, 1)
    tc_kernel(const Params p, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<kD, kE4M3>;
    constexpr int kStages = C::kStages;
    [[maybe_unused]] constexpr int kHalves = kD / 64;  // 128-byte column blocks of a 16-bit tile
    extern __shared__ uint8_t dyn[];
    const uint32_t pad = (0u - smem_u32(dyn)) & 1023u;
    const uint32_t sm_q = smem_u32(dyn) + pad;
    const uint32_t sm_ring = sm_q + 2 * C::kTileBytes;
    const uint32_t sm_kraw = sm_ring + kStages * C::kTileBytes;
    const uint32_t sm_vraw = sm_kraw + C::kKRaw * C::kRawBytes;
    uint8_t *tail = dyn + pad + (2 + kStages) * C::kTileBytes + C::kRaw * C::kRawBytes;
    auto &sh = *reinterpret_cast<typename C::Sh *>(tail);
    float *stat = reinterpret_cast<float *>(C::kStatBytes ? tail + sizeof(typename C::Sh)
                                                          : dyn + pad + C::kTileBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], kE4M3 ? 4 : 1);
            mbar_init(&sh.empty[i], 2);
        }
        if constexpr (kE4M3) {
            for (int i = 0; i < 4; ++i) {
                mbar_init(&sh.kraw_full[i], 1);
                mbar_init(&sh.kraw_empty[i], 2);
                mbar_init(&sh.vraw_full[i], 1);
                mbar_init(&sh.vraw_empty[i], 4);
            }
            for (int i = 0; i < C::kScales; ++i) mbar_init(&sh.sc_full[i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sh.guard_go[i], 1);
            mbar_init(&sh.guard_done[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], kE4M3 ? 19 : 11);  // all but the producer
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.drain[i], 1);
            mbar_init(&sh.turn[i], 1);
        }
        mbar_init(&sh.q_full, 8);
        sh.abort_flag = 0;
        for (int i = 0; i < 3; ++i) sh.stop[i][0] = sh.stop[i][1] = 0;
        for (int i = 0; i < kMarks; ++i) sh.poison[i] = 0;
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

    bool bad = false;
    Start start{};
    if constexpr (kPaged) {
        start = find_start(p, blockIdx.x, &sh.start, &bad);
        if (bad && p.err && blockIdx.x == 0) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the CTA holds all 512 TMEM columns: S of slot s at 128 s, O at 256 + kD s
    volatile int *abort_flag = &sh.abort_flag;
    // Piece number i of the ring, for every role but the producer's; all lanes of a
    // warp (`whole`) or one thread.  Returns false at the end or on an abort.
    auto take_piece = [&](uint32_t i, Piece *pc, bool whole) {
        if (!bar_wait(&sh.piece_full[i % kPieces], (i / kPieces) & 1u, abort_flag, p.err)) return false;
        *pc = *reinterpret_cast<const Piece *>(sh.piece[i % kPieces]);
        if (whole) __syncwarp();
        if (!whole || lane == 0) mbar_arrive(&sh.piece_empty[i % kPieces]);
        return pc->n_rows > 0;
    };

    if (warp >= 8 && warp < 12) {
        regs_give<C::kRegsFew>();
        if (warp == 9 || (kE4M3 && warp == 11)) {
            // ---- producer: the pieces, and the TMA copies by one thread.  E4M3: warp 9 the
            // keys, warp 11 the values ----
            const bool of_keys = !kE4M3 || warp == 9;
            uint32_t pos = 0, n_piece = 0;  // operand tiles issued
            uint32_t n_key = 0, n_value = 0;
            [[maybe_unused]] uint32_t n_guard = 0;
            bool ok = true, bad_page = false;
            const int32_t rows_box = kPaged ? min(p.page_size, kTile) : kTile;
            const int32_t page_shift = kPaged ? 31 - __clz(p.page_size) : 0;
            const int32_t box_shift = kPaged ? 7 - min(page_shift, 7) : 0;  // log2 of the boxes of a tile
            Piece pc{};
            // Page numbers come eight key tiles at a time: the lanes load the next eight's
            // while one thread issues the copies of these.  -1: no page (past the end, or
            // out of range), a box of zeros.
            int32_t ids[2] = {-1, -1};
            auto fetch_pages = [&](int32_t tile) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t e = lane + 32 * k, at = tile + (e >> box_shift);
                    const int32_t l = at * kTile + (e & ((1 << box_shift) - 1)) * rows_box;
                    ids[k] = -1;
                    if (e < (8 << box_shift) && at < pc.t1 && l < pc.rq.len) {
                        ids[k] = __ldg(p.page_table + (int64_t)pc.b * p.max_pages + (l >> page_shift));
                    }
                }
            };
            auto keep_pages = [&](int32_t tile, uint32_t buffer) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t e = lane + 32 * k, at = tile + (e >> box_shift);
                    const int32_t l = at * kTile + (e & ((1 << box_shift) - 1)) * rows_box;
                    const bool good = (uint64_t)(int64_t)ids[k] < (uint64_t)p.num_pages;
                    if (e < (8 << box_shift) && at < pc.t1 && l < pc.rq.len && !good) bad_page = true;
                    if (e < (8 << box_shift)) sh.pages[warp >> 1 & 1][buffer][e] = good ? ids[k] : -1;
                }
                __syncwarp();
            };
            auto load = [&](int32_t j, bool values) {  // key tile t0 + j
                const int32_t tile = pc.t0 + j;
                uint64_t *fullb;
                uint32_t dst;
                if constexpr (kE4M3) {
                    const uint32_t n = values ? n_value : n_key, slots = values ? C::kVRaw : C::kKRaw;
                    const uint32_t s = n % slots, ph = ((n / slots) & 1u) ^ 1u;
                    fullb = values ? &sh.vraw_full[s] : &sh.kraw_full[s];
                    dst = (values ? sm_vraw : sm_kraw) + s * C::kRawBytes;
                    if (!bar_wait(values ? &sh.vraw_empty[s] : &sh.kraw_empty[s], ph, abort_flag, p.err))
                        return false;
                    mbar_arrive_expect_tx(fullb, C::kRawBytes);
                } else {
                    const uint32_t s = pos % kStages;
                    fullb = &sh.full[s];
                    dst = sm_ring + s * C::kTileBytes;
                    if (!bar_wait(&sh.empty[s], ((pos / kStages) & 1u) ^ 1u, abort_flag, p.err)) return false;
                    mbar_arrive_expect_tx(fullb, C::kTileBytes);
                }
                const CUtensorMap *map = values ? &vmap : &kmap;
                if constexpr (!kPaged) {
#pragma unroll
                    for (int half = 0; half < kHalves; ++half)
                        tma_load_3d(dst + half * (kTile * 128), map, fullb, 64 * half, pc.h,
                                    pc.rq.t0 + tile * kTile);
                } else {
                    const int32_t y = (tile * kTile) & (p.page_size - 1) & ~(kTile - 1);
                    const int32_t *page = sh.pages[warp >> 1 & 1][(j >> 3) & 1] + ((j & 7) << box_shift);
                    int32_t id = page[0];
#pragma unroll 1
                    for (int i = 0; i < (1 << box_shift); ++i) {
                        const int32_t z = id >= 0 ? id * p.kv_heads + pc.h : -1;
                        const int32_t next = page[i + 1];  // past the last: unused
                        if constexpr (kE4M3) {
                            tma_load_3d(dst + i * rows_box * kD, map, fullb, 0, y, z);
                        } else {
#pragma unroll
                            for (int half = 0; half < kHalves; ++half)
                                tma_load_3d(dst + half * (kTile * 128) + i * rows_box * 128, map, fullb, 64 * half,
                                            y, z);
                        }
                        id = next;
                    }
                }
                // the guard may wait for the copy now: the operand's barrier is in its phase
                if (!kE4M3 && values && tile >= pc.guard_from) mbar_arrive(&sh.guard_go[n_guard++ & 7u]);
                n_key += !values;
                n_value += values;
                ++pos;
                return true;
            };
            Walk walk{};
            Levels levels{};
            if constexpr (!kPaged)
                levels.begin(p, lane, &bad);
            else if (of_keys)
                walk.begin(p, start);
            for (;;) {
                if (!of_keys) {
                    const bool more = take_piece(n_piece, &pc, true);
                    if (!more) pc.n_rows = 0;
                    if (kPaged && more) fetch_pages(pc.t0);
                } else {
                    if constexpr (kPaged)
                        walk.next(p, &pc);
                    else
                        levels.next(p, lane, &pc);
                    pc.tok0 = pc.row0 / p.group;
                    pc.rem0 = pc.row0 - pc.tok0 * p.group;
                    for (int r = lane; r < pc.n_rows; r += 32) {  // the queries, on their way to L2
                        const int x = pc.rem0 + r, dt = x / p.group;
                        const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.q +
                                                 (int64_t)(pc.rq.t0 + pc.tok0 + dt) * p.q_stride +
                                                 (int64_t)(pc.h * p.group + x - dt * p.group) * kD;
#pragma unroll
                        for (int c = 0; c < kD; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + c));
                    }
                    if (kPaged && pc.n_rows > 0) fetch_pages(pc.t0);
                    if (elect_one()) {
                        ok = bar_wait(&sh.piece_empty[n_piece % kPieces], ((n_piece / kPieces) & 1u) ^ 1u,
                                      abort_flag, p.err);
                        if (ok) {
                            *reinterpret_cast<Piece *>(sh.piece[n_piece % kPieces]) = pc;
                            mbar_arrive(&sh.piece_full[n_piece % kPieces]);
                        }
                    }
                }
                // shared K0 V0 K1 V1 ..., alternate K0 K1 V0 K2 V1 ... V(n-2) V(n-1)
                const int32_t n = pc.n_rows > 0 ? pc.t1 - pc.t0 : 0, lead = pc.shared() ? 0 : 1;
                int32_t jk = 0, jv = 0;
                for (int32_t c = 0; c < n; c += 8) {
                    if constexpr (kPaged) {
                        keep_pages(pc.t0 + c, (c >> 3) & 1);
                        fetch_pages(pc.t0 + c + 8);
                    }
                    if (elect_one()) {
                        if constexpr (kE4M3) {
                            for (; ok && jk < min(n, c + 8); ++jk) ok = load(jk, !of_keys);
                        } else {
                            // the keys of these eight tiles and the values that follow them
                            while (ok && (jk < min(n, c + 8) || (c + 8 >= n && jv < n))) {
                                const bool values = jk == n || jk - jv > lead;
                                ok = load(values ? jv : jk, values);
                                if (values)
                                    ++jv;
                                else
                                    ++jk;
                            }
                        }
                    }
                    __syncwarp();
                }
                ++n_piece;
                if (__any_sync(0xFFFFFFFFu, !ok) || pc.n_rows == 0) break;
            }
            if (kPaged && of_keys && lane == 0) p.join[blockIdx.x] = walk.join;
            if ((bad_page || (!kPaged && bad && blockIdx.x == 0)) && p.err)
                atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
            if (!ok) {  // wait for the copies in flight before the shared memory goes
                auto drain = [&](uint64_t *bars, uint32_t issued, uint32_t slots) {
                    for (uint32_t n = issued > slots ? issued - slots : 0; n < issued; ++n) {
                        const uint64_t t0 = global_timer_ns();
                        while (!mbar_try_wait(bars + n % slots, (n / slots) & 1u))
                            if (global_timer_ns() - t0 > kWaitLimitNs) break;
                    }
                };
                if constexpr (kE4M3) {
                    drain(sh.kraw_full, n_key, C::kKRaw);
                    drain(sh.vraw_full, n_value, C::kVRaw);
                } else {
                    drain(sh.full, pos, kStages);
                }
            }
        } else if (warp == 8 || warp == 10) {
            // ---- MMA issuer of slot s: one thread ----
            // Each slot has its own issuer: an MMA costs the issuing thread about as
            // long as the tensor core takes for it.  Both walk every operand of the
            // ring in order and hand it back (an operand is free when both have).
            if (elect_one()) {
                const int s = warp == 8 ? 0 : 1;
                constexpr uint32_t kIdS = kE4M3 ? idesc_e4m3(kTile, kTile) : idesc16(false, kTile, false);
                constexpr uint32_t kIdO = idesc16(kE4M3, kD, true);
                const uint32_t dS = s * kTile, dO = 256 + s * kD;
                uint32_t pos = 0, tiles_done = 0, n_piece = 0, n_guard = 0, n_p = 0, n_turn = 0;
                bool ok = true;
                Piece pc{};
                // an operand's place: bf16, operand n of the ring; E4M3, by key tile
                struct Place {
                    uint64_t *full, *empty;
                    uint32_t phase, addr;
                };
                auto ring = [&](uint32_t n) {
                    const uint32_t i = n % kStages;
                    return Place{&sh.full[i], &sh.empty[i], (n / kStages) & 1u, sm_ring + i * C::kTileBytes};
                };
                // scores of a key operand (mine), or the other slot's operand handed back
                auto keys = [&](const Place &o, bool mine, bool q1) {
                    if (!bar_wait(o.full, o.phase, abort_flag, p.err)) return false;
                    if (!mine) {
                        mbar_arrive(o.empty);
                        return true;
                    }
                    const uint32_t kd = desc_lo(o.addr) | kKMajorLo;
                    const uint32_t qd = desc_lo(sm_q + (q1 ? C::kTileBytes : 0)) | kKMajorLo;
                    tc_fence_after();
                    if constexpr (kE4M3) {  // both parts of Q, one after the other
#pragma unroll
                        for (int k = 0; k < 2 * (kD / 32); ++k) {
                            const uint32_t off = (k % (kD / 32)) * 2;
                            tc_mma_f8(dS, desc64(qd + (k >= kD / 32 ? C::kRawBytes >> 4 : 0) + off, kCodesHi<kD>),
                                      desc64(kd + off, kCodesHi<kD>), kIdS, k > 0);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kD / 16; ++k) {
                            const uint32_t off = (k >> 2) * ((kTile * 128) >> 4) + (k & 3) * 2;
                            tc_mma_bf16(dS, desc64(qd + off, kKMajorHi), desc64(kd + off, kKMajorHi), kIdS, k > 0);
                        }
                    }
                    tc_commit(&sh.s_full[s]);
                    tc_commit(o.empty);
                    return true;
                };
                // sums over the value operand of key tile t, once the guard is done with it
                auto values = [&](int32_t t, const Place &o, bool mine, bool acc, bool last) {
                    if (!bar_wait(o.full, o.phase, abort_flag, p.err)) return false;
                    if (!kE4M3 && t >= pc.guard_from) {
                        if (mine &&
                            !bar_wait(&sh.guard_done[n_guard & 7u], (n_guard >> 3) & 1u, abort_flag, p.err))
                            return false;
                        ++n_guard;
                    }
                    if (!mine) {
                        mbar_arrive(o.empty);
                        return true;
                    }
                    const uint32_t vd = desc_lo(o.addr) | kMnMajorLo;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!bar_wait(&sh.p_full[s][h], n_p & 1u, abort_flag, p.err)) return false;
                        tc_fence_after();
#pragma unroll
                        for (int k = 4 * h; k < 4 * h + 4; ++k)
                            tc_mma_ts(dO, dS + 8 * k, desc64(vd + k * (2048 >> 4), kMnMajorHi), kIdO,
                                      acc || k > 0);
                    }
                    ++n_p;
                    tc_commit(o.empty);
                    if (last) tc_commit(&sh.o_full[s]);
                    return true;
                };
                while (ok && take_piece(n_piece, &pc, false)) {
                    ok = bar_wait(&sh.q_full, n_piece & 1u, abort_flag, p.err);
                    ++n_piece;
                    const int32_t n = pc.t1 - pc.t0;
                    // shared: K0 V0 K1 V1 ..., every tile mine (slot 0 of a prompt ends earlier)
                    // alternate: K0 K1 V0 K2 V1 ... V(n-2) V(n-1), tile j mine if j % 2 == s
                    const bool both = pc.shared();
                    const int32_t n_mine = both && s == 0 ? pc.t1a - pc.t0 : n;
                    auto key = [&](int32_t j) {
                        Place o;
                        if constexpr (kE4M3) {
                            const uint32_t kt = tiles_done + j, i = kt % C::kKRaw;
                            o = Place{&sh.kraw_full[i], &sh.kraw_empty[i], (kt / C::kKRaw) & 1u,
                                      sm_kraw + i * C::kRawBytes};
                        } else {
                            o = ring(pos + (both ? 2 * j : j == 0 ? 0 : 2 * j - 1));
                        }
                        return keys(o, both ? j < n_mine : (j & 1) == s, both && s == 1);
                    };
                    // the next scores follow the sums that free their place: key j + 1 after
                    // value j of both slots, or key j + 2 after value j of its own
                    if (ok) ok = key(0);
                    if (ok && !both && n > 1) ok = key(1);
#pragma unroll 1
                    for (int32_t j = 0; ok && j < n; ++j) {
                        // shared: the slots' MMAs take turns, a tile's sums and the next scores
                        // together, so that one slot's softmax runs beside the other's MMAs
                        // (issued as they come, both slots fall into step and neither does:
                        // 3400 cycles per tile and pair of slots against 2500)
                        if (both) {
                            ok = bar_wait(&sh.turn[s], (n_turn & 1u) ^ (s == 0 ? 1u : 0u), abort_flag, p.err);
                            if (!ok) break;
                            ++n_turn;
                        }
                        const Place o = ring(kE4M3 ? tiles_done + j
                                                   : pos + (both ? 2 * j + 1 : j + 1 < n ? 2 * j + 2 : 2 * n - 1));
                        const bool mine = both ? j < n_mine : (j & 1) == s;
                        ok = values(pc.t0 + j, o, mine, both ? j > 0 : j >= 2,
                                    both ? j + 1 == n_mine : j + 2 >= n);
                        const int32_t next = both ? j + 1 : j + 2;
                        if (ok && next < n) ok = key(next);
                        if (both) mbar_arrive(&sh.turn[s ^ 1]);
                    }
                    tiles_done += n;
                    pos += 2 * n;
                }
                // nothing of this slot's is in flight when the accumulators are freed
                tc_commit(&sh.drain[s]);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&sh.drain[s], 0))
                    if (global_timer_ns() - t0 > kWaitLimitNs) break;
            }
        } else if constexpr (!kE4M3) {
            // ---- guard: values of tiles with masked positions ----
            uint32_t pos = 0, n_piece = 0, n_guard = 0;
            bool ok = true;
            Piece pc{};
            while (ok && take_piece(n_piece, &pc, true)) {
                const int32_t n = pc.t1 - pc.t0;
                for (int32_t j = max(0, pc.guard_from - pc.t0); ok && j < n; ++j) {
                    const uint32_t nv = pos + (pc.shared() ? 2 * j + 1 : j + 1 < n ? 2 * j + 2 : 2 * n - 1);
                    ok = bar_wait(&sh.guard_go[n_guard & 7u], (n_guard >> 3) & 1u, abort_flag, p.err) &&
                         bar_wait(&sh.full[nv % kStages], (nv / kStages) & 1u, abort_flag, p.err);
                    if (!ok) break;
                    // rows [low, live) of the tile may be masked for some row; from live on
                    // they are no keys.  A 128-byte row of a column block is 8 chunks.
                    const int32_t first = (pc.t0 + j) * kTile;
                    const int32_t live = min(max(pc.rq.len - first, 0), kTile);
                    const int32_t low = min(max((kPaged ? pc.rq.ctx : pc.tok0) - first, 0), live);
                    bool found = false;
#pragma unroll 1
                    for (int half = 0; half < kHalves; ++half) {
                        const uint32_t base = sm_ring + (nv % kStages) * C::kTileBytes + half * (kTile * 128);
#pragma unroll 1
                        for (int i = live * 8 + lane; i < kTile * 8; i += 32)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + i * 16), "r"(0)
                                         : "memory");
#pragma unroll 4
                        for (int i = low * 8 + lane; i < live * 8; i += 32) {
                            uint32_t w[4], odd = 0;
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                         : "r"(base + i * 16));
                            // a 16-bit exponent of all ones: adding 1 to it carries into the sign's place
#pragma unroll
                            for (int k = 0; k < 4; ++k) odd |= ((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                            found |= odd != 0;
                        }
                        if (__any_sync(0xFFFFFFFFu, found)) {
#pragma unroll 1
                            for (int i = low * 32 + lane; i < live * 32; i += 32) {
                                uint32_t w;
                                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(base + i * 4));
                                if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
                                if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + i * 4), "r"(w) : "memory");
                            }
                        }
                    }
                    if (found) *(volatile uint8_t *)&sh.poison[n_piece % kMarks] = poison_mark(n_piece);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.guard_done[n_guard & 7u]);
                    ++n_guard;
                }
                pos += 2 * n;
                ++n_piece;
            }
        }
    } else if (warp >= 12) {
        // ---- E4M3: value codes to fp16 (exact), and the scales of both to fp32; warps 12-15
        // the even key tiles, warps 16-19 the odd ones ----
        regs_give<C::kRegsFew>();
        if constexpr (kE4M3) {
            uint32_t n_piece = 0, tiles_done = 0;
            const int group = warp >= 16, row = (threadIdx.x - 384) & 127;
            Piece pc{};
            // Exponent bytes: this row's key of the group's next tile, and its page of the one
            // after that, so that neither load is waited for.
            const int32_t page_shift = 31 - __clz(p.page_size);
            int32_t page = -1;
            int ke = 0, ve = 0;
            auto fetch_page = [&](int32_t tile) {
                const int32_t l = tile * kTile + row;
                page = -1;
                if (tile < pc.t1 && l < pc.rq.len)
                    page = __ldg(p.page_table + (int64_t)pc.b * p.max_pages + (l >> page_shift));
            };
            auto fetch_exps = [&](int32_t tile) {  // of `page`
                ke = ve = 127;
                if ((uint64_t)(int64_t)page < (uint64_t)p.num_pages) {
                    const int32_t off = (tile * kTile + row) & (p.page_size - 1);
                    const int64_t at = ((int64_t)page * p.kv_heads + pc.h) * p.page_size + off;
                    ke = __ldg(p.k_exp + at);
                    ve = __ldg(p.v_exp + at);
                }
            };
            // the scales of key tile number `no`
            auto scales = [&](int32_t tile, uint32_t no) {
                const uint32_t i = no % C::kScales;
                const bool live = tile * kTile + row < pc.rq.len;
                const int k_exp = kv_exponent((uint8_t)ke), v_exp = kv_exponent((uint8_t)ve);
                fetch_exps(tile + 2);
                fetch_page(tile + 4);
                const int vt = __reduce_max_sync(0xFFFFFFFFu, live ? v_exp : -64);
                const int vb = __reduce_min_sync(0xFFFFFFFFu, live ? v_exp : 64);
                int(*red)[2] = sh.reduce[group][(no >> 1) & 1u];
                if (lane == 0) red[warp & 3][0] = vt, red[warp & 3][1] = vb;
                sh.kmul[i][row] = pow2_int(k_exp);
                sh.vmul[i][row] = pow2_int(v_exp);
                asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");
                int v_top = -64, v_low = 64;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    v_top = max(v_top, red[w][0]);
                    v_low = min(v_low, red[w][1]);
                }
                if (row == 0) {
                    sh.scale[i].top = v_top;
                    sh.scale[i].wide = v_top - v_low > kWideE4M3;  // no live row: -64 and 64
                    mbar_arrive(&sh.sc_full[i]);
                }
            };
            auto widen = [&](int32_t tile, uint32_t no) {
                const uint32_t rs = no % C::kVRaw, s = no % kStages;
                const bool live = tile * kTile + row < pc.rq.len;
                const uint32_t src = sm_vraw + rs * C::kRawBytes + row * kD;
                const uint32_t dst = sm_ring + s * C::kTileBytes + row * 128;
                bar_wait(&sh.vraw_full[rs], (no / C::kVRaw) & 1u, abort_flag, p.err);
                bar_wait(&sh.empty[s], ((no / kStages) & 1u) ^ 1u, abort_flag, p.err);
                const bool fix = tile >= pc.guard_from || !live;
                bool found = false;
                // 16 codes a chunk, two at a time; the copy's swizzle spreads the rows over the banks
#pragma unroll 1
                for (int c0 = 0; c0 < kD / 16; c0 += 2) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = c0 + e;
                        const uint32_t a = src + ((kD == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                                     : "r"(a));
                    }
                    if (fix) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (!live) w[e][k] = 0u;
                                const uint32_t nan = __vcmpeq4(w[e][k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                found |= nan != 0;
                                w[e][k] &= ~nan;
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = c0 + e;
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                                (__nv_fp8x2_storage_t)(w[e][k >> 1] >> (16 * (k & 1))), __NV_E4M3);
                            o[k] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        const uint32_t d0 = dst + (c >> 2) * (kTile * 128);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             d0 + (((2 * (c & 3) + k) ^ (row & 7)) << 4)),
                                         "r"(o[4 * k]), "r"(o[4 * k + 1]), "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                                         : "memory");
                    }
                }
                if (found) *(volatile uint8_t *)&sh.poison[n_piece % kMarks] = poison_mark(n_piece);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.vraw_empty[rs]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.full[s]);
            };
            // (no wait's failure leaves the loop: the barriers want all four warps)
            for (;;) {
                if (!take_piece(n_piece, &pc, true)) sh.stop[1 + group][n_piece & 1u] = 1;
                asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");
                if (*(volatile int *)&sh.stop[1 + group][n_piece & 1u]) break;
                const int32_t n = pc.t1 - pc.t0;
                const int32_t from = (tiles_done & 1u) == (uint32_t)group ? 0 : 1;
                fetch_page(pc.t0 + from);
                fetch_exps(pc.t0 + from);
                fetch_page(pc.t0 + from + 2);
#pragma unroll 1
                for (int32_t j = from; j < n; j += 2) {
                    scales(pc.t0 + j, tiles_done + j);
                    widen(pc.t0 + j, tiles_done + j);
                }
                tiles_done += n;
                ++n_piece;
            }
        }
    } else {
        // ---- softmax of slot s, with the loads of Q and the epilogue ----
        regs_take<C::kRegsMany>();
        const int s = warp >> 2;
        const int wq = warp & 3;
        const int my = wq * 32 + lane;  // accumulator row
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = s * kTile + lane_base;
        const uint32_t tO = 256 + s * kD + lane_base;
        uint32_t n_piece = 0, n_s = 0, tiles_done = 0;
        uint32_t n_o[2] = {0, 0};
        const float mul = p.scale_log2;                                      // > 0
        const uint32_t magic = (65536u + p.group - 1) / (uint32_t)p.group;   // x / group for x < 512
        Piece pc{};
        // (no wait's failure leaves the loop: the barriers below want all warps)
        for (;;) {
            if (!take_piece(n_piece, &pc, true)) sh.stop[0][n_piece & 1u] = 1;
            named_sync<1, 256>();
            if (*(volatile int *)&sh.stop[0][n_piece & 1u]) break;
            const bool both = pc.shared();
            // few rows: `copies` copies of them in the accumulator's rows, one per 128 /
            // copies, each with its share of the tile's keys (log2 of the copies)
            const int split = !kPaged || pc.n_rows > 64 ? 0 : pc.n_rows > 32 ? 1 : 2;
            // queries: kD / 8 lanes hold a row, 8 values each.  bf16: copied as they are, all rows
            // at once; E4M3: eight rows in flight per thread
            {
                constexpr int kLanes = kD / 8, kStep = 256 / kLanes;
                const int l8 = threadIdx.x % kLanes;
                const __nv_bfloat16 *q0 = (const __nv_bfloat16 *)p.q + (int64_t)(pc.rq.t0 + pc.tok0) * p.q_stride +
                                          (int64_t)pc.h * p.group * kD + l8 * 8;
                if constexpr (!kE4M3) {
#pragma unroll 4
                    for (int r = threadIdx.x / kLanes; r < pc.n_rows; r += kStep) {
                        const uint32_t x = pc.rem0 + r, dt = (x * magic) >> 16;
                        const __nv_bfloat16 *src = q0 + (int64_t)dt * p.q_stride + (int)(x - dt * p.group) * kD;
                        for (int k = 0; k < (1 << split); ++k) {
                            const int row = (r & 127) + (k << (7 - split));
                            const uint32_t dst = sm_q + (r >> 7) * C::kTileBytes + (l8 >> 3) * (kTile * 128) +
                                                 row * 128 + (((l8 & 7) ^ (row & 7)) << 4);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                } else {
                    const uint32_t row_lanes = ((1u << kLanes) - 1u) << (lane & ~(kLanes - 1));
#pragma unroll 1
                    for (int rb = threadIdx.x / kLanes; rb < pc.n_rows; rb += 8 * kStep) {
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = rb + i * kStep;
                            const uint32_t x = pc.rem0 + r, dt = (x * magic) >> 16;
                            v[i] = make_uint4(0u, 0u, 0u, 0u);
                            if (r < pc.n_rows)
                                v[i] = __ldg(reinterpret_cast<const uint4 *>(
                                    q0 + (int64_t)dt * p.q_stride + (int)(x - dt * p.group) * kD));
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = rb + i * kStep;
                            if (r >= pc.n_rows) break;
                            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            float f[8], amax = 0.0f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                f[2 * k] = __uint_as_float(w[k] << 16);
                                f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
                                amax = fmaxf(amax, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
                            }
#pragma unroll
                            for (int o = kLanes / 2; o > 0; o >>= 1)
                                amax = fmaxf(amax, __shfl_xor_sync(row_lanes, amax, o));
                            // 2^-a: the largest magnitude's binade becomes 2^7
                            const int a = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -110), 110);
                            // an infinite value makes the row NaN: codes hold no infinity
                            const float down =
                                amax <= 3.4e38f ? __uint_as_float((uint32_t)(127 - a) << 23) : __int_as_float(0x7FC00000);
                            uint32_t hi[2], lo[2];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 y = make_float2(f[2 * k] * down, f[2 * k + 1] * down);
                                const uint32_t ch = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                                const float2 back = __half22float2(
                                    __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)ch, __NV_E4M3)));
                                const uint32_t cl = __nv_cvt_float2_to_fp8x2(
                                    make_float2(y.x - back.x, y.y - back.y), __NV_SATFINITE, __NV_E4M3);
                                hi[k >> 1] = (k & 1) ? hi[k >> 1] | (ch << 16) : ch;
                                lo[k >> 1] = (k & 1) ? lo[k >> 1] | (cl << 16) : cl;
                            }
                            if (l8 == 0)
                                sh.qmul[n_piece & 1u][r] =
                                    fmaxf(__uint_as_float((uint32_t)(127 + a) << 23) * mul, 1.1754944e-38f);
                            for (int k = 0; k < (1 << split); ++k) {
                                const int row = (r & 127) + (k << (7 - split));
                                const int c = kD == 128 ? (l8 >> 1) ^ (row & 7) : (l8 >> 1) ^ ((row >> 1) & 3);
                                const uint32_t dst =
                                    sm_q + (r >> 7) * C::kTileBytes + row * kD + (c << 4) + ((l8 & 1) << 3);
                                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(hi[0]), "r"(hi[1])
                                             : "memory");
                                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + C::kRawBytes), "r"(lo[0]),
                                             "r"(lo[1])
                                             : "memory");
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
                if constexpr (kE4M3) named_sync<1, 256>();  // the rows' scales
            }
            const int copy = my >> (7 - split);
            const int r_blk = (both ? s * kTile : 0) + my - (copy << (7 - split));  // row within the block
            const uint32_t r_off = pc.rem0 + r_blk, r_tok = (r_off * magic) >> 16;
            const int32_t tok = pc.tok0 + (int32_t)r_tok;
            const bool live_row = r_blk < pc.n_rows;
            const bool live_warp = (r_blk & ~31) < pc.n_rows;
            float qm = mul;
            if constexpr (kE4M3) qm = live_row ? sh.qmul[n_piece & 1u][r_blk] : 1.0f;
            // positions below this one are seen by every row of the slot
            const int32_t all_seen =
                kPaged ? pc.rq.ctx : pc.tok0 + (int32_t)(((pc.rem0 + (both ? s * kTile : 0)) * magic) >> 16) + 1;
            const int32_t t_end = both && s == 0 ? pc.t1a : pc.t1;
            float base = -INFINITY, sum = 0.0f;
            int x_shift = kNoShift;  // E4M3: x
            bool first = true;
            // O and x or base move together: O 2^x 2^base stays
            auto rescale = [&](float fix) {
                if (first) return;
#pragma unroll 1
                for (int c = 0; c < kD; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c, o);
                    tmem_ld_wait();
                    tmem_tie(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
                    tmem_st32(tO + c, o);
                }
            };
            auto hand_over = [&](int h) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[s][h]);
            };
            // One key tile: this warp's kC chunks of 32 keys, from chunk c0 on.
            [[maybe_unused]] auto tile = [&](auto chunks, const int c0, const int32_t t) {
                constexpr int kC = decltype(chunks)::value;
                uint32_t x[kC][32];
                const bool masked = (t + 1) * kTile > all_seen;
                auto scores = [&]() {
#pragma unroll
                    for (int c = 0; c < kC; ++c) tmem_ld32(tS + 32 * (c0 + c), x[c]);
                    uint32_t w[kC];
#pragma unroll
                    for (int c = 0; c < kC; ++c)
                        w[c] = masked && live_row ? seen_bits<kPaged>(p, pc.rq, tok, t * kTile + 32 * (c0 + c)) : 0u;
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < kC; ++c) tmem_tie(x[c]);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < kC; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((w[c] >> k) & 1u)) x[c][k] = 0xFF800000u;  // -inf
                    }
                };
                uint64_t part[4];
                const uint64_t qm2 = f2(qm, qm);
                uint32_t pk[32];
                // weights of the chunks [from, to): 2^(z - base)
                auto weights = [&](int from, int to, float safe) {
                    const uint64_t off2 = f2(-safe, -safe);
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        if (c < from || c >= to) continue;
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float a, b;
                            unf2(fma2(f2(x[c][k], x[c][k + 1]), qm2, off2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            part[(k >> 1) & 3] = add2(part[(k >> 1) & 3], f2(a, b));
                            pk[16 * (c & 1) + (k >> 1)] = pack16<false>(a, b);
                        }
                    }
                };
                auto row_top = [&]() {
                    float top[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        top[k] = fmaxf(__uint_as_float(x[0][2 * k]), __uint_as_float(x[0][2 * k + 1]));
#pragma unroll
                    for (int k = 16; k < 32 * kC; k += 2)
                        top[(k >> 1) & 7] =
                            fmaxf(fmaxf(top[(k >> 1) & 7], __uint_as_float(x[k >> 5][k & 31])),
                                  __uint_as_float(x[k >> 5][(k & 31) + 1]));
                    return fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])),
                                 fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7]))) * qm;
                };
                // few rows: this copy's weights, zeros at the other copies' keys
                auto store_split = [&]() {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if constexpr (kC == 2)
                                v[k] = c0 == 2 * h ? pk[k] : 0u;
                            else
                                v[k] = c0 == 2 * h + (k >> 4) ? pk[k & 15] : 0u;
                        }
                        tmem_st32(tS + 32 * h, v);
                    }
                    hand_over(0);
                    if (lane == 0) mbar_arrive(&sh.p_full[s][1]);
                };
                // the first weights against the base so far, beside the maximum; again, from
                // the scores in TMEM, where the maximum moved the base (the first tiles,
                // mostly)
                constexpr int kFirst = kC == 4 ? 2 : kC;
#pragma unroll 1
                for (bool again = false;;) {
                    scores();
                    const float mx = row_top();
                    part[0] = part[1] = part[2] = part[3] = 0ull;
                    weights(0, kFirst, base == -INFINITY ? 0.0f : base);
                    if (again) break;
                    const bool grow = live_row && mx > base + kLazy;
                    if (!__any_sync(0xFFFFFFFFu, grow)) break;
                    // grow: base was -inf (fix = 0, nothing summed yet) or finite
                    const float fix = grow ? ex2(base - mx) : 1.0f;
                    if (grow) base = mx;
                    sum *= fix;
                    rescale(fix);
                    again = true;
                }
                if constexpr (kC == 4) {
                    tmem_st32(tS, pk);
                    hand_over(0);
                    weights(2, 4, base == -INFINITY ? 0.0f : base);
                    tmem_st32(tS + 32, pk);
                    hand_over(1);
                } else {
                    store_split();
                }
                float a, b;
                unf2(add2(add2(part[0], part[1]), add2(part[2], part[3])), a, b);
                sum += a + b;
                first = false;
            };
            // The same with E4M3 scales, chunk by chunk from TMEM, once for the maximum and
            // once for the weights: one short body for every number of chunks, since these
            // warps share the instruction cache with the widening ones (unrolled as above,
            // every second issue slot waited for an instruction).
            [[maybe_unused]] auto tile_e4m3 = [&](const int c0, const int c1, const int32_t t, const uint32_t i4) {
                if constexpr (kE4M3) {
                    const bool masked = (t + 1) * kTile > all_seen;
                    uint32_t x[32];
                    // chunk c's scores times 2^ke, -inf where not seen
                    auto scores = [&](int c) {
                        tmem_ld32(tS + 32 * c, x);
                        const uint32_t w =
                            masked && live_row ? seen_bits<kPaged>(p, pc.rq, tok, t * kTile + 32 * c) : 0u;
                        tmem_ld_wait();
                        tmem_tie(x);
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&sh.kmul[i4][32 * c + k]);
                            float a, b;
                            unf2(mul2(f2(x[k], x[k + 1]), f.x), a, b);
                            x[k] = __float_as_uint(a), x[k + 1] = __float_as_uint(b);
                            unf2(mul2(f2(x[k + 2], x[k + 3]), f.y), a, b);
                            x[k + 2] = __float_as_uint(a), x[k + 3] = __float_as_uint(b);
                        }
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((w >> k) & 1u)) x[k] = 0xFF800000u;  // -inf
                        }
                    };
                    const bool once = c1 - c0 == 1;  // the scores stay in registers
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        scores(c);
                        float top[4] = {mx, mx, mx, mx};
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            top[(k >> 1) & 3] = fmaxf(fmaxf(top[(k >> 1) & 3], __uint_as_float(x[k])),
                                                      __uint_as_float(x[k + 1]));
                        mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    }
                    mx *= qm;
                    const bool grow = live_row && mx > base + kLazy;
                    const float nb = grow ? mx : base;
                    const float safe = nb == -INFINITY ? 0.0f : nb;
                    const float gain = grow ? fminf(nb - base, 1024.0f) : 0.0f;  // 1024: base was -inf
                    float fix = grow ? ex2(base - nb) : 1.0f;
                    base = nb;
                    sum *= fix;
                    // binade of the largest weight with its value's scale: at most the largest
                    // weight's and the largest scale's
                    const TileScale ts = sh.scale[i4];
                    int level = ts.top + (int)floorf(fmaxf(mx - safe, -4096.0f));
                    bool some = mx > -INFINITY;
                    if (ts.wide) {  // the scales differ too much: look at each weight
                        float hi = 0.0f;
#pragma unroll 1
                        for (int c = c0; c < c1; ++c) {
                            if (!once) scores(c);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                hi = fmaxf(hi, ex2(fmaf(__uint_as_float(x[k]), qm, -safe)) * sh.vmul[i4][32 * c + k]);
                        }
                        level = (int)(__float_as_uint(hi) >> 23) - 127;
                        some = hi > 0.0f;
                    }
                    const bool had = x_shift != kNoShift;
                    if (live_row && some && (grow || level - x_shift >= kCapE4M3)) {
                        const int nx = max(had ? x_shift - (int)gain : -100, level - kTopE4M3);
                        if (had) fix *= pow2_int(x_shift - nx);
                        x_shift = nx;
                    }
                    if (__any_sync(0xFFFFFFFFu, fix != 1.0f)) rescale(had ? fix : 0.0f);
                    const float down = had || some ? pow2_int(-x_shift) : 1.0f;
                    const uint64_t down2 = f2(down, down), qm2 = f2(qm, qm), off2 = f2(-safe, -safe);
                    uint64_t part[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        if (!once) scores(c);
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float a, b;
                            unf2(fma2(f2(x[k], x[k + 1]), qm2, off2), a, b);
                            const uint64_t w2 = f2(ex2(a), ex2(b));
                            part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], w2);
                            unf2(mul2(mul2(w2, down2), *reinterpret_cast<const uint64_t *>(&sh.vmul[i4][32 * c + k])), a, b);
                            pk[k >> 1] = pack16<true>(a, b);
                        }
                        tmem_st16(tS + 16 * c, pk);  // over scores of chunk c / 2: done, or in registers
                        if (c == 1 && c1 == 4) hand_over(0);
                    }
                    // few rows: zeros at the other copies' keys
                    const uint32_t zero[16] = {};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c)
                        if (c < c0 || c >= c1) tmem_st16(tS + 16 * c, zero);
                    hand_over(1);
                    if (c1 - c0 < 4 && lane == 0) mbar_arrive(&sh.p_full[s][0]);
                    float a, b;
                    unf2(add2(part[0], part[1]), a, b);
                    sum += a + b;
                    first = false;
                }
            };
            for (int32_t t = pc.t0 + (both ? 0 : s); t < t_end; t += both ? 1 : 2) {
                [[maybe_unused]] const uint32_t tile_no = tiles_done + (uint32_t)(t - pc.t0);
                if constexpr (kE4M3) {
                    bar_wait(&sh.sc_full[tile_no % C::kScales], (tile_no / C::kScales) & 1u, abort_flag, p.err);
                }
                bar_wait(&sh.s_full[s], n_s & 1u, abort_flag, p.err);
                ++n_s;
                tc_fence_after();
                if (!live_warp) {
                    if (lane == 0) {
                        mbar_arrive(&sh.p_full[s][0]);
                        mbar_arrive(&sh.p_full[s][1]);
                    }
                    continue;
                }
                if constexpr (kE4M3) {
                    const int chunks = 4 >> split;
                    tile_e4m3(copy * chunks, (copy + 1) * chunks, t, tile_no % C::kScales);
                } else if (!kPaged || split == 0) {
                    tile(std::integral_constant<int, 4>{}, 0, t);
                } else if (split == 1) {
                    tile(std::integral_constant<int, 2>{}, 2 * copy, t);
                } else {
                    tile(std::integral_constant<int, 1>{}, copy, t);
                }
            }
            // ---- epilogue ----
            const int32_t n = pc.t1 - pc.t0;
            const bool used1 = both || n > 1;
            tiles_done += n;
            const float up = !kE4M3 || x_shift == kNoShift ? 1.0f : pow2_int(x_shift);
            const int64_t row =
                (int64_t)(pc.rq.t0 + tok) * p.q_heads + pc.h * p.group + (int)(r_off - r_tok * p.group);
            float *part = pc.slot >= 0 ? p.part + pc.slot * part_slot_floats(p.part_rows, kD) : nullptr;
            bool owner = live_row;  // this thread writes the row's statistics
            if (both) {
                // each slot's rows are its own: a thread writes its row
                bar_wait(&sh.o_full[s], n_o[s] & 1u, abort_flag, p.err);
                tc_fence_after();
                if (live_warp) {
                    const float g = part ? up : sum == 0.0f ? 0.0f : up / sum;
                    float4 *part_col = reinterpret_cast<float4 *>(part) + r_blk;  // [kD / 4][part_rows] of four
                    // output rows through the slot's query tile, which no product reads any more, so
                    // that a warp writes whole rows (each thread its own: 32 lines a store)
                    constexpr int kRow16 = kD / 8;
                    uint4 *stage = reinterpret_cast<uint4 *>(dyn + pad + s * C::kTileBytes) + wq * 32 * kRow16;
#pragma unroll 1
                    for (int c0 = 0; c0 < kD; c0 += 32) {
                        uint32_t a[32];
                        tmem_ld32(tO + c0, a);
                        tmem_ld_wait();
                        tmem_tie(a);
                        if (!live_row) continue;
#pragma unroll
                        for (int k = 0; k < 32; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * g);
                        if (part) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                part_col[(c0 / 4 + k) * p.part_rows] =
                                    make_float4(__uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1]),
                                                __uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t o[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    o[e] = pack16<false>(__uint_as_float(a[8 * k + 2 * e]),
                                                         __uint_as_float(a[8 * k + 2 * e + 1]));
                                stage[lane * kRow16 + ((c0 / 8 + k) ^ (lane & 7))] = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        }
                    }
                    if (!part) {
                        __syncwarp();
                        const int first_row = r_blk - lane, rows = min(32, pc.n_rows - first_row);
#pragma unroll 4
                        for (int i = lane / kRow16; i < rows; i += 32 / kRow16) {
                            const uint32_t x = pc.rem0 + first_row + i, dt = (x * magic) >> 16;
                            const int64_t at = (int64_t)(pc.rq.t0 + pc.tok0 + (int)dt) * p.q_heads + pc.h * p.group +
                                               (int)(x - dt * p.group);
                            const int c = lane % kRow16;
                            reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.out + at * kD)[c] = stage[i * kRow16 + (c ^ (i & 7))];
                        }
                        __syncwarp();  // other lanes wrote this thread's row, and it may add to it below
                    }
                }
            } else {
                // a row's sums lie in up to two slots and four copies: joined through shared
                // memory, 32 columns at a time (the query tiles are free by now)
                bar_wait(&sh.o_full[0], n_o[0] & 1u, abort_flag, p.err);
                if (used1) bar_wait(&sh.o_full[1], n_o[1] & 1u, abort_flag, p.err);
                tc_fence_after();
                float *mine = stat + 3 * kTile * s + my;
                mine[0] = base;
                mine[kTile] = sum;
                mine[2 * kTile] = up;
                named_sync<1, 256>();
                const int rows = kTile >> split, row_in = my & (rows - 1);
                // source i: slot i >> split, copy i & (copies - 1)
                const int sources = (used1 ? 2 : 1) << split;
                float sb[8], sl[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *st = stat + 3 * kTile * (i >> split) + (i & ((1 << split) - 1)) * rows + row_in;
                    sb[i] = i < sources ? st[0] : -INFINITY;
                    sl[i] = i < sources ? st[kTile] : 0.0f;
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, sb[i]);
                const float safe = top == -INFINITY ? 0.0f : top;
                const float g = ex2(base - safe) * up;
                float all = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) all = fmaf(sl[i], ex2(sb[i] - safe), all);
                base = top;
                sum = all;
                owner = live_row && s == 0 && copy == 0;
                float *inv = stat + 6 * kTile;
                if (s == 0 && copy == 0) inv[row_in] = part ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
                // [source][row][groups of four, swizzled]: rows up to a power of two, and as many
                // columns at a time as 32 KB hold
                const int row_shift = max(0, 32 - __clz(pc.n_rows - 1)), rows_in = 1 << row_shift;
                const int per = (2 << split) * rows_in;  // rows of all sources: 2 .. 256
                const int k_shift = kD == 128 && per <= 64 ? 5 : per <= 128 ? 4 : 3, quads = 1 << k_shift;
                float4 *red = reinterpret_cast<float4 *>(dyn + pad);
#pragma unroll 1
                for (int c0 = 0; c0 < kD; c0 += 4 * quads) {
                    if (live_warp && (s == 0 || used1)) {
                        float4 *dst = red + (((((s << split) + copy) << row_shift) + row_in) << k_shift);
#pragma unroll 1
                        for (int q = 0; q < quads; q += 8) {
                            uint32_t a[32];
                            tmem_ld32(tO + c0 + 4 * q, a);
                            tmem_ld_wait();
                            tmem_tie(a);
                            if (live_row) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    dst[(q + k) ^ (row_in & 7)] =
                                        make_float4(__uint_as_float(a[4 * k]) * g, __uint_as_float(a[4 * k + 1]) * g,
                                                    __uint_as_float(a[4 * k + 2]) * g, __uint_as_float(a[4 * k + 3]) * g);
                            }
                        }
                    }
                    named_sync<1, 256>();
#pragma unroll 1
                    for (int i = threadIdx.x; i < rows_in << k_shift; i += 256) {
                        // partial rows: rows fastest; output rows: columns fastest
                        const int r = part ? i & (rows_in - 1) : i >> k_shift;
                        const int k = part ? i >> row_shift : i & (quads - 1);
                        if (r >= pc.n_rows) continue;
                        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int src = 0; src < 8; ++src) {
                            if (src >= sources) break;
                            const float4 v = red[(((src << row_shift) + r) << k_shift) + (k ^ (r & 7))];
                            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
                        }
                        if (part) {
                            reinterpret_cast<float4 *>(part)[(c0 / 4 + k) * p.part_rows + r] = o;
                        } else {
                            const uint32_t ro = pc.rem0 + r, rt = (ro * magic) >> 16;
                            const int64_t to = ((int64_t)(pc.rq.t0 + pc.tok0 + (int)rt) * p.q_heads +
                                                pc.h * p.group + (int)(ro - rt * p.group)) * kD + c0 + 4 * k;
                            const float f = inv[r];
                            *reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.out + to) =
                                make_uint2(pack16<false>(o.x * f, o.y * f), pack16<false>(o.z * f, o.w * f));
                        }
                    }
                    named_sync<1, 256>();
                }
            }
            n_o[0] += 1;
            n_o[1] += used1;
            if (owner) {
                if (*(volatile uint8_t *)&sh.poison[n_piece % kMarks] == poison_mark(n_piece))
                    add_poison<kD, kE4M3, kPaged>(p, pc.rq, pc.b, pc.h, tok, max(pc.t0, pc.guard_from) * kTile,
                                                  min(pc.t1 * kTile, pc.rq.len), 0, kD, part ? part + 4 * r_blk : nullptr,
                                                  (__nv_bfloat16 *)p.out + row * kD);
                if (part) {
                    part[part_stats(p.part_rows, kD) + r_blk] = base;
                    part[part_stats(p.part_rows, kD) + p.part_rows + r_blk] = sum;
                } else if (p.lse) {
                    p.lse[row] = sum == 0.0f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
                }
            }
            // the sums are read: the next piece's q_full arrivals say so to the MMAs
            tc_fence_before();
            ++n_piece;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

template <int kD, bool kE4M3, bool kPaged>
dflash2_status launch_one(const DeviceInfo &di, Params p, cudaStream_t st) {
    using C = Cfg<kD, kE4M3>;
    auto fn = tc_kernel<kD, kE4M3, kPaged>;
    static std::atomic<uint64_t> done{0};
    const dflash2_status allowed = allow_smem(fn, C::kSmem, di.device, done);
    if (allowed != DFLASH2_OK) return allowed;
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
    p.row_shift = kRowShift;
    const bool shared = (int64_t)p.total_q * p.group > kTile;  // some row block may fill both slots
    for (int i = 0; i < 4; ++i) {
        p.tile_units[i] = kE4M3 && i >= 2 ? kSharedUnits : kTileUnits;
        p.item_units[i] = kItemTiles * p.tile_units[i];
    }
    p.most_units = kE4M3 && shared ? kSharedUnits : kTileUnits;
    // prompts: every row block of every request, at most one short one each
    const int64_t items = ((((int64_t)p.total_q * p.group) >> kRowShift) + p.batch) * p.kv_heads;
    p.n_cta = kPaged || items > di.sm_count ? di.sm_count : (int32_t)items;
    launch_k(fn, dim3((unsigned)p.n_cta), dim3(C::kThreads), C::kSmem, st, p, maps[0], maps[1]);
    const dflash2_status s = launch_status();
    if (s != DFLASH2_OK || !kPaged) return s;
    return launch_combine(di, p, DFLASH2_BF16, st);
}

bool rows16(const void *p, int64_t stride, int el) {
    return aligned16(p) && stride * el % 16 == 0;
}

}  // namespace

bool tc_takes(const Params &p, bool paged, int32_t dtype) {
    if (dtype != DFLASH2_BF16 || (p.head_dim != 64 && p.head_dim != 128)) return false;
    if (!(p.scale_log2 >= 1.1754944e-38f)) return false;  // masked scores are -inf times the scale
    if (!rows16(p.q, p.q_stride, 2) || !aligned16(p.out) || !aligned16(p.k) || !aligned16(p.v))
        return false;
    if (!paged) return rows16(p.k, p.k_stride, 2) && rows16(p.v, p.v_stride, 2);
    return p.page_size >= 16 && (p.page_size & (p.page_size - 1)) == 0;
}

dflash2_status launch_tc(const DeviceInfo &di, const Params &p, bool paged, int32_t kv_format,
                         cudaStream_t st) {
    if (!paged)
        return p.head_dim == 64 ? launch_one<64, false, false>(di, p, st)
                                : launch_one<128, false, false>(di, p, st);
    // Few rows a request on average: the transposed kernel.  64 requests over 0 to 8191 keys,
    // head_dim 128, with 4, 16, 32, 48 and 60 rows take it 97, 100, 127, 165 and 212 us, and
    // this file's 155, 158, 165, 211 and 211 (head_dim 64, 48 and 60 rows: 155 and 196, 177 and 177).
    // Empty requests count, since only the device knows them: beside 48 or 56 empty ones, 16
    // requests of 128 rows over 4000 keys take it 234 us and this file's kernel 95, 8 of 256 rows
    // 230 and 89, 8 of 64 rows 76 and 50.
    if (kv_format == DFLASH2_KV_E4M3 && (int64_t)p.total_q * p.group <= 48 * (int64_t)p.batch)
        return launch_few(di, p, st);
    if (kv_format == DFLASH2_KV_E4M3)
        return p.head_dim == 64 ? launch_one<64, true, true>(di, p, st)
                                : launch_one<128, true, true>(di, p, st);
    return p.head_dim == 64 ? launch_one<64, false, true>(di, p, st)
                            : launch_one<128, false, true>(di, p, st);
}

}  // namespace attn
}  // namespace dflash2
