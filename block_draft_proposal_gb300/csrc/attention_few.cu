// Attention over an E4M3 cache on the 5th-generation tensor cores, for requests of
// few query rows (a row: one token's query head).  head_dim 64 or 128.
//
// One pass over the keys in tiles of 128, transposed, so that an MMA's 128 rows are
// keys and then channels, and its columns only as many as there are query rows:
//
//   S^T = K Q^T        tcgen05.mma kind::f8f6f4 on the codes as they are held
//   P^T = 2^(z - base) one thread per key: its two scales are the thread's own, and
//                      the exponentials of a key's rows need no shuffles
//   O^T += V^T P^T     the same kind, V's codes read as the MN-major A operand
//
// Both products run at the rate of 8-bit operands and no code is widened: the
// operands that carry more than four bits are split into E4M3 parts instead, where
// they are small.  Q is two parts (the nearest code and that of the rest, under a
// power of two per row): the eight bits of a bf16 value down to 2^-10 of the row's
// largest, and 2^-18 of that below.  P is three, in columns of their own that the end
// adds up: fp16's eleven bits, each part's rest scaled by 2^5 for the next, down to
// 2^-20 absolute, where a row's largest P starts at 2^3 and stays below 2^8.  A higher start
// would keep smaller weights and move x more often (2^5: 210 us in place of 171, for the
// trees below).
//
// z = S 2^(key scale) 2^a scale log2(e), and a weight carries its value's scale:
// P = 2^(z - base) 2^(value scale) 2^-x with an integer x per row.  base and x are
// lazy: a tile is computed against the ones so far, and only where some z exceeds
// its base by 8 or some P exceeds 2^8 (the first tile, and few after it) the CTA finds
// the maxima, moves them, rescales its sums and takes the tile again.  base follows z
// alone, so that the sum of the weights does not depend on the values.
//
// Two CTAs share an SM, so that one's softmax runs beside the other's waits, an item's
// start and end among them (one CTA per SM with two accumulators that take the key tiles
// in turns: 105 and 189 us for the 96 and 170 below).  Warps 0-3 softmax, the loads of
// Q and the epilogue; warp 4 issues the MMAs; warp 5 loads the keys, warp 6 the values
// (one TMA box per page).
//
// Measured (128 per head, 8 key/value heads): 64 requests of one token over 0 to 8191
// keys, 4 rows a head, take 96 us, 5.7 TB/s of the cache's bytes; 128 requests of trees of
// up to 12 tokens over 13 to 4096 keys, 5 to 60 rows, 170 us.  Few rows are bound by the
// loads and by an item's start and end (four to five tiles' time); many by the softmax
// warps, whose chains of conversions two warps per scheduler do not fill (56 % of the issue
// slots): 64 requests over 3000 to 4096 keys with 15, 30 and 60 rows take 89, 113 and 178
// us.  Their code is kept short, chunk by chunk of 16 rows: over two chunks at once, 128
// requests take 200 us, and unrolled over 64 rows 309, since the warps wait for
// instructions.  Sums in place of the maxima that tell when to move: no change.
#include <type_traits>

#include "attention_tc.cuh"

namespace dflash2 {
namespace attn {
namespace {

constexpr int kRowShift = 6, kRows = 1 << kRowShift;  // rows of a block
// Units of a key tile with up to 16, 32, 48 and 64 rows, and of an item's start and end.
constexpr int kTileUnits[4] = {10, 13, 18, 23}, kItemUnits[4] = {40, 50, 60, 70};
constexpr int kParts = 3;       // of a weight
constexpr float kPartScale = 32.0f;  // from one part to the next: what is left of 2^8 stays below 2^8
constexpr float kLazy = 8.0f;   // log2 growth of a maximum that moves its base
constexpr float kCap = 256.0f;  // the largest P
constexpr int kTop = 3;         // binade of the largest P where x moves

struct Shared {
    alignas(16) uint8_t piece[kPieces][kPieceBytes];
    alignas(16) float qm[kRows];       // 2^a scale log2(e) of a row
    alignas(16) float off[kRows];      // -base (0: no base yet)
    alignas(16) float xm[kRows];       // 2^-x
    alignas(16) float fix_sum[kRows], fix_o[kRows];
    float top[4][2][kRows];            // a warp's largest z, and z + value scale
    float sums[4][kRows];              // of a tile's weights by warp, then of all
    int32_t pages[2][2][kTile / 16 * 8 + 1];  // page numbers of eight key tiles, twice, by producer
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t raw_full[2][4], raw_empty[2][4];  // codes of keys, values
    uint64_t s_full, s_free, p_full, pv_done, q_full, drain;
    uint32_t tmem;
    int abort_flag;
    int stop[2];  // no more pieces, by piece parity
    int poison;  // number of the last piece with a value not finite
    StartScratch start;
};

template <int kD> struct Few {
    static constexpr int kRawBytes = kTile * kD;           // codes of a tile
    static constexpr int kStages = kD == 128 ? 2 : 4;      // tiles of keys, and of values
    static constexpr int kQBytes = 2 * kRows * kD;         // both parts
    static constexpr int kPBytes = kParts * kTile * 64;    // [column blocks of 64][key][column]
    static constexpr int kThreads = 256;
    // registers: 128 each at launch; with 72 for the producers, they spill (101 us below for 96)
    static constexpr int kRegsMany = 144, kRegsFew = 112;
    static constexpr int kSmem = kQBytes + kPBytes + 2 * kStages * kRawBytes + (int)sizeof(Shared) + 1024;
    static_assert(kSmem <= 113 * 1024, "half of an SM's shared memory");
};

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Does any softmax thread say so?  (a barrier of them)
__device__ __forceinline__ bool group_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync() { named_sync<1, 128>(); }

template <int kD>
__global__ void __launch_bounds__(Few<kD>::kThreads, 2)
    few_kernel(const Params p, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
    using C = Few<kD>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t dyn[];
    const uint32_t pad = (0u - smem_u32(dyn)) & 1023u;
    const uint32_t sm_q = smem_u32(dyn) + pad;
    const uint32_t sm_p = sm_q + C::kQBytes;
    const uint32_t sm_raw[2] = {sm_p + C::kPBytes, sm_p + C::kPBytes + kStages * C::kRawBytes};
    Shared &sh = *reinterpret_cast<Shared *>(dyn + pad + C::kQBytes + C::kPBytes + 2 * kStages * C::kRawBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k)
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&sh.raw_full[k][i], 1);
                mbar_init(&sh.raw_empty[k][i], 1);
            }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], 6);  // all but the producer
        }
        mbar_init(&sh.s_full, 1);
        mbar_init(&sh.s_free, 4);
        mbar_init(&sh.p_full, 4);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.drain, 1);
        mbar_init(&sh.q_full, 4);
        sh.abort_flag = 0;
        sh.stop[0] = sh.stop[1] = 0;
        sh.poison = -1;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(&sh.tmem, 256);
        tmem_relinquish();
    }
    if (warp == 5 && lane == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    grid_dep_wait();
    grid_dep_launch();

    bool bad = false;
    const Start start = find_start(p, blockIdx.x, &sh.start, &bad);
    if (bad && p.err && blockIdx.x == 0) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // two CTAs share the SM's TMEM, 256 columns each: S^T, then O^T
    const uint32_t tmem = sh.tmem;
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

    if (warp >= 4) {
        regs_give<C::kRegsFew>();
        if (warp == 5 || warp == 6) {
            // ---- producers: warp 5 the pieces and the keys, warp 6 the values ----
            const int of = warp - 5;
            uint32_t issued = 0, n_piece = 0;
            bool ok = true, bad_page = false;
            const int32_t rows_box = min(p.page_size, kTile);
            const int32_t page_shift = 31 - __clz(p.page_size);
            const int32_t box_shift = 7 - min(page_shift, 7);  // log2 of the boxes of a tile
            const uint8_t *exps = of ? p.v_exp : p.k_exp;
            Piece pc{};
            // Page numbers come eight key tiles at a time: the lanes load the next eight's
            // while one thread issues the copies of these.  -1: no page (past the end, or
            // out of range), a box of zeros.
            int32_t ids[2] = {-1, -1};
            auto line_of = [&](int32_t tile, int k) {  // first key of box lane + 32 k, or -1
                const int32_t e = lane + 32 * k, at = tile + (e >> box_shift);
                const int32_t l = at * kTile + (e & ((1 << box_shift) - 1)) * rows_box;
                return e < (8 << box_shift) && at < pc.t1 && l < pc.rq.len ? l : -1;
            };
            auto fetch_pages = [&](int32_t tile) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t l = line_of(tile, k);
                    ids[k] = l >= 0 ? __ldg(p.page_table + (int64_t)pc.b * p.max_pages + (l >> page_shift)) : -1;
                }
            };
            auto keep_pages = [&](int32_t tile, uint32_t buffer) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t e = lane + 32 * k;
                    const bool good = (uint64_t)(int64_t)ids[k] < (uint64_t)p.num_pages;
                    if (!good && line_of(tile, k) >= 0) bad_page = true;
                    if (e < (8 << box_shift)) sh.pages[of][buffer][e] = good ? ids[k] : -1;
                    // the box's exponents, on their way to L2
                    if (good)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            exps + ((int64_t)ids[k] * p.kv_heads + pc.h) * p.page_size + (line_of(tile, k) & (p.page_size - 1))));
                }
                __syncwarp();
            };
            auto load = [&](int32_t j) {  // key tile t0 + j
                const int32_t tile = pc.t0 + j;
                const uint32_t s = issued % kStages;
                uint64_t *fullb = &sh.raw_full[of][s];
                if (!bar_wait(&sh.raw_empty[of][s], ((issued / kStages) & 1u) ^ 1u, abort_flag, p.err)) return false;
                mbar_arrive_expect_tx(fullb, C::kRawBytes);
                const uint32_t dst = sm_raw[of] + s * C::kRawBytes;
                const int32_t y = (tile * kTile) & (p.page_size - 1) & ~(kTile - 1);
                const int32_t *page = sh.pages[of][(j >> 3) & 1] + ((j & 7) << box_shift);
                int32_t id = page[0];
#pragma unroll 1
                for (int i = 0; i < (1 << box_shift); ++i) {
                    const int32_t z = id >= 0 ? id * p.kv_heads + pc.h : -1;
                    const int32_t next = page[i + 1];  // past the last: unused
                    tma_load_3d(dst + i * rows_box * kD, of ? &vmap : &kmap, fullb, 0, y, z);
                    id = next;
                }
                ++issued;
                return true;
            };
            Walk walk{};
            if (of == 0) walk.begin(p, start);
            for (;;) {
                if (of == 1) {
                    if (!take_piece(n_piece, &pc, true)) pc.n_rows = 0;
                } else {
                    walk.next(p, &pc);
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
                    if (elect_one()) {
                        ok = bar_wait(&sh.piece_empty[n_piece % kPieces], ((n_piece / kPieces) & 1u) ^ 1u,
                                      abort_flag, p.err);
                        if (ok) {
                            *reinterpret_cast<Piece *>(sh.piece[n_piece % kPieces]) = pc;
                            mbar_arrive(&sh.piece_full[n_piece % kPieces]);
                        }
                    }
                }
                const int32_t n = pc.n_rows > 0 ? pc.t1 - pc.t0 : 0;
                if (n > 0) fetch_pages(pc.t0);
                for (int32_t c = 0; c < n; c += 8) {
                    keep_pages(pc.t0 + c, (c >> 3) & 1);
                    fetch_pages(pc.t0 + c + 8);
                    if (elect_one())
                        for (int32_t j = c; ok && j < min(n, c + 8); ++j) ok = load(j);
                    __syncwarp();
                }
                ++n_piece;
                if (__any_sync(0xFFFFFFFFu, !ok) || pc.n_rows == 0) break;
            }
            if (of == 0 && lane == 0) p.join[blockIdx.x] = walk.join;
            if (bad_page && p.err) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
            if (!ok) {  // wait for the copies in flight before the shared memory goes
                for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(&sh.raw_full[of][i % kStages], (i / kStages) & 1u))
                        if (global_timer_ns() - t0 > kWaitLimitNs) break;
                }
            }
        } else if (warp == 4 && elect_one()) {
            // ---- MMA issuer: one thread ----
            const uint32_t dS = tmem, dO = tmem + kRows;
            uint32_t tiles_done = 0, n_piece = 0, n_s = 0, n_p = 0;
            bool ok = true;
            Piece pc{};
            // descriptors' high words: K-major rows of kD bytes; V [keys][kD] as MN-major with
            // 8-key groups one swizzle atom apart (head_dim 64: M is 128 all the same, and
            // the second 64 repeat the first, a leading offset of zero)
            constexpr uint32_t kVHi = kCodesHi<kD>;
            while (ok && take_piece(n_piece, &pc, false)) {
                ok = bar_wait(&sh.q_full, n_piece & 1u, abort_flag, p.err);
                ++n_piece;
                const int32_t n = pc.t1 - pc.t0, cols = (pc.n_rows + 15) & ~15;
                const uint32_t id_s = idesc_e4m3(128, cols);
                const uint32_t id_o = idesc_e4m3(128, kParts * cols) | (1u << 15) | (1u << 16);  // both MN-major
                auto scores = [&](int32_t j) {
                    const uint32_t kt = tiles_done + j, i = kt % kStages;
                    if (!bar_wait(&sh.raw_full[0][i], (kt / kStages) & 1u, abort_flag, p.err) ||
                        !bar_wait(&sh.s_free, (n_s & 1u) ^ 1u, abort_flag, p.err))
                        return false;
                    ++n_s;
                    tc_fence_after();
                    const uint32_t kd = desc_lo(sm_raw[0] + i * C::kRawBytes) | kKMajorLo;
                    const uint32_t qd = desc_lo(sm_q) | kKMajorLo;
#pragma unroll
                    for (int k = 0; k < 2 * (kD / 32); ++k) {  // both parts of Q, one after the other
                        const uint32_t at = (k % (kD / 32)) * 2, part = k >= kD / 32 ? (kRows * kD) >> 4 : 0;
                        tc_mma_f8(dS, desc64(kd + at, kCodesHi<kD>), desc64(qd + part + at, kCodesHi<kD>), id_s,
                                  k > 0);
                    }
                    tc_commit(&sh.s_full);
                    tc_commit(&sh.raw_empty[0][i]);
                    return true;
                };
                if (ok) ok = scores(0);
#pragma unroll 1
                for (int32_t j = 0; ok && j < n; ++j) {
                    if (j + 1 < n) ok = scores(j + 1);
                    const uint32_t kt = tiles_done + j, i = kt % kStages;
                    ok = ok && bar_wait(&sh.raw_full[1][i], (kt / kStages) & 1u, abort_flag, p.err) &&
                         bar_wait(&sh.p_full, n_p & 1u, abort_flag, p.err);
                    if (!ok) break;
                    ++n_p;
                    tc_fence_after();
                    const uint32_t vd = desc_lo(sm_raw[1] + i * C::kRawBytes);
                    const uint32_t pd = desc_lo(sm_p) | (uint32_t)((kTile * 64) >> 4) << 16;
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        tc_mma_f8(dO, desc64(vd + k * (32 * kD >> 4), kVHi), desc64(pd + k * (32 * 64 >> 4), kCodesHi<64>), id_o,
                                  j > 0 || k > 0);
                    tc_commit(&sh.raw_empty[1][i]);
                    tc_commit(&sh.pv_done);
                }
                tiles_done += n;
            }
            // nothing is in flight when the accumulators are freed
            tc_commit(&sh.drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&sh.drain, 0))
                if (global_timer_ns() - t0 > kWaitLimitNs) break;
        }
    } else {
        // ---- softmax, with the loads of Q and the epilogue ----
        regs_take<C::kRegsMany>();
        const int my = threadIdx.x;  // key of a tile, channel of the sums
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t tS = tmem + lane_base, tO = tS + kRows;
        const uint32_t my_p = sm_p + my * 64;
        const uint32_t magic = (65536u + p.group - 1) / (uint32_t)p.group;  // x / group for x < 512
        const int32_t page_shift = 31 - __clz(p.page_size);
        uint32_t n_piece = 0, n_tile = 0, tiles_done = 0;
        Piece pc{};
        int32_t page = -1;
        int ke = 127, ve = 127;
        // Exponent bytes: this thread's key of the next tile, and its page of the one after
        // that, so that neither load is waited for.
        auto fetch_page = [&](int32_t tile) {
            const int32_t l = tile * kTile + my;
            page = -1;
            if (tile < pc.t1 && l < pc.rq.len)
                page = __ldg(p.page_table + (int64_t)pc.b * p.max_pages + (l >> page_shift));
        };
        auto fetch_exps = [&](int32_t tile) {  // of `page`
            ke = ve = 127;
            if ((uint64_t)(int64_t)page < (uint64_t)p.num_pages) {
                const int32_t at = (tile * kTile + my) & (p.page_size - 1);
                const int64_t i = ((int64_t)page * p.kv_heads + pc.h) * p.page_size + at;
                ke = __ldg(p.k_exp + i);
                ve = __ldg(p.v_exp + i);
            }
        };
        // (no wait's failure leaves the loop: the barriers below want all warps)
        for (;;) {
            if (!take_piece(n_piece, &pc, true)) sh.stop[n_piece & 1u] = 1;
            group_sync();
            if (*(volatile int *)&sh.stop[n_piece & 1u]) break;
            fetch_page(pc.t0);
            // queries: kD / 8 lanes hold a row, 8 values each
            {
                constexpr int kLanes = kD / 8, kStep = 128 / kLanes, kEach = kRows / kStep;
                const uint32_t row_lanes = ((1u << kLanes) - 1u) << (lane & ~(kLanes - 1));
                const int l8 = threadIdx.x % kLanes;
                const __nv_bfloat16 *q0 = (const __nv_bfloat16 *)p.q + (int64_t)(pc.rq.t0 + pc.tok0) * p.q_stride +
                                          (int64_t)pc.h * p.group * kD + l8 * 8;
                uint4 v[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int r = threadIdx.x / kLanes + i * kStep;
                    const uint32_t x = pc.rem0 + r, dt = (x * magic) >> 16;
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < pc.n_rows)
                        v[i] = __ldg(reinterpret_cast<const uint4 *>(q0 + (int64_t)dt * p.q_stride +
                                                                     (int)(x - dt * p.group) * kD));
                }
                fetch_exps(pc.t0);
                fetch_page(pc.t0 + 1);
                if (my < kRows) {
                    sh.off[my] = 0.0f;
                    sh.xm[my] = my < pc.n_rows ? 1.0f : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int r = threadIdx.x / kLanes + i * kStep;
                    if (r >= pc.n_rows) {
                        if (l8 == 0) sh.qm[r] = 0.0f;
                        continue;
                    }
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
                        const uint32_t cl = __nv_cvt_float2_to_fp8x2(make_float2(y.x - back.x, y.y - back.y),
                                                                     __NV_SATFINITE, __NV_E4M3);
                        hi[k >> 1] = (k & 1) ? hi[k >> 1] | (ch << 16) : ch;
                        lo[k >> 1] = (k & 1) ? lo[k >> 1] | (cl << 16) : cl;
                    }
                    if (l8 == 0)
                        sh.qm[r] = fmaxf(__uint_as_float((uint32_t)(127 + a) << 23) * p.scale_log2, 1.1754944e-38f);
                    const int c = kD == 128 ? (l8 >> 1) ^ (r & 7) : (l8 >> 1) ^ ((r >> 1) & 3);
                    const uint32_t dst = sm_q + r * kD + (c << 4) + ((l8 & 1) << 3);
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(hi[0]), "r"(hi[1]) : "memory");
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + kRows * kD), "r"(lo[0]), "r"(lo[1])
                                 : "memory");
                }
                fence_proxy_async_smem();
                // all threads: the rows' factors are there, and the last piece's sums are read
                group_sync();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }
            const int n_chunk = (pc.n_rows + 15) >> 4;  // of 16 rows
            float sum[2] = {0.0f, 0.0f};  // this warp's keys: rows 2 lane and the next
            bool late = false;            // some row may have no base after the first tile
            // row `my`: its base (-inf: none yet), largest z + value scale at the last move, x
            float row_base = -INFINITY, row_top = -INFINITY, row_x = 0.0f;

            for (int32_t t = pc.t0; t < pc.t1; ++t, ++n_tile) {
                const bool first = t == pc.t0;
                const int32_t l = t * kTile + my;
                const float km = pow2_byte((uint8_t)ke), vm = pow2_byte((uint8_t)ve);
                const float vf = (float)kv_exponent((uint8_t)ve);
                fetch_exps(t + 1);
                fetch_page(t + 2);
                const bool masked = (t + 1) * kTile > pc.rq.ctx;
                if (first) late = masked;
                // the rows that see this key: bit r; all of a token's rows do, or none
                uint64_t seen = ~0ull;
                if (masked) {
                    seen = 0;
                    const int n_tok = (pc.rem0 + pc.n_rows + p.group - 1) / p.group;
#pragma unroll 1
                    for (int i0 = 0; i0 < n_tok; i0 += 32) {  // a lane loads a token's bits of this warp's keys
                        uint32_t bits = 0;
                        if (i0 + lane < n_tok)
                            bits = seen_bits<true>(p, pc.rq, pc.tok0 + i0 + lane, t * kTile + warp * 32);
                        const int n_here = min(n_tok - i0, 32);
#pragma unroll 1
                        for (int i = 0; i < n_here; ++i) {
                            const uint32_t w = __shfl_sync(0xFFFFFFFFu, bits, i);
                            // the token's rows in the block: one at least, and they may begin before it
                            const int at = (i0 + i) * p.group - pc.rem0;
                            const int r0 = max(at, 0), n_rows = min(at + p.group, kRows) - r0;
                            if ((w >> lane) & 1u) seen |= (~0ull >> (kRows - n_rows)) << r0;
                        }
                    }
                }
                bar_wait(&sh.s_full, n_tile & 1u, abort_flag, p.err);
                tc_fence_after();
                const uint64_t km2 = f2(km, km), vm2 = f2(vm, vm);
                uint32_t x[16];
                // z of the 16 rows from c on, against the slot's bases
                auto scores = [&](int c) {
                    tmem_ld16(tS + c, x);
                    tmem_ld_wait();
                    tmem_tie16(x);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const ulonglong2 q4 = *reinterpret_cast<const ulonglong2 *>(&sh.qm[c + k]);
                        const ulonglong2 o4 = *reinterpret_cast<const ulonglong2 *>(&sh.off[c + k]);
                        float a, b;
                        unf2(fma2(mul2(f2(x[k], x[k + 1]), km2), q4.x, o4.x), a, b);
                        x[k] = __float_as_uint(a), x[k + 1] = __float_as_uint(b);
                        unf2(fma2(mul2(f2(x[k + 2], x[k + 3]), km2), q4.y, o4.y), a, b);
                        x[k + 2] = __float_as_uint(a), x[k + 3] = __float_as_uint(b);
                    }
                    if (masked) {
                        const uint32_t w = (uint32_t)(seen >> c);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (!((w >> k) & 1u)) x[k] = 0xFF800000u;  // -inf
                    }
                };
                // Weights against the bases and x so far; again where those had to move.  They
                // move first in an item's first tile, and in masked ones where a row may see
                // its first key.
#pragma unroll 1
                for (bool move = first || (masked && late), again = false;; move = again = true) {
                    if (move) {
                        // four rows at a time: this code is rarely in the instruction cache
#pragma unroll 1
                        for (int c = 0; c < pc.n_rows; c += 4) {
                            uint32_t y[4];
                            tmem_ld4(tS + c, y);
                            tmem_ld_wait();
                            tmem_tie4(y);
                            const float4 q4 = *reinterpret_cast<const float4 *>(&sh.qm[c]);
                            const float q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float z = fmaf(__uint_as_float(y[k]) * km, q[k], 0.0f);
                                if (!((seen >> (c + k)) & 1u)) z = -INFINITY;
                                const float top = warp_max(z), top_v = warp_max(z + vf);
                                if (lane == 0) {
                                    sh.top[warp][0][c + k] = top;
                                    sh.top[warp][1][c + k] = top_v;
                                }
                            }
                        }
                        group_sync();
                        if (my < pc.n_rows) {
                            float top = -INFINITY, fix = 1.0f, fix_o = 1.0f;
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                top = fmaxf(top, sh.top[w][0][my]);
                                row_top = fmaxf(row_top, sh.top[w][1][my]);
                            }
                            const bool had = row_base > -INFINITY;
                            if (top > row_base + kLazy) {
                                if (had) fix = ex2(row_base - top);
                                fix_o = fix;
                                row_base = top;
                            }
                            if (row_base > -INFINITY) {
                                const float nx = floorf(fminf(fmaxf(row_top - row_base, -100.0f), 100.0f)) - kTop;
                                if (had) fix_o *= ex2(row_x - nx);
                                row_x = nx;
                                sh.off[my] = -row_base;
                                sh.xm[my] = pow2_int(-(int)nx);
                            }
                            sh.fix_sum[my] = fix;
                            sh.fix_o[my] = fix_o;
                        }
                        group_sync();
                        if (!first) {
                            if (2 * lane < pc.n_rows) sum[0] *= sh.fix_sum[2 * lane];
                            if (2 * lane + 1 < pc.n_rows) sum[1] *= sh.fix_sum[2 * lane + 1];
                            // the products so far, all of them there
                            if (!again) bar_wait(&sh.pv_done, (n_tile - 1u) & 1u, abort_flag, p.err);
                            tc_fence_after();
#pragma unroll 1
                            for (int i = 0; i < kParts * n_chunk; ++i) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * i, o);
                                tmem_ld_wait();
                                tmem_tie16(o);
                                const float4 *f4 = reinterpret_cast<const float4 *>(sh.fix_o + i / kParts * 16);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float4 f = f4[k];
                                    o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * f.x);
                                    o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * f.y);
                                    o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * f.z);
                                    o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * f.w);
                                }
                                tmem_st16(tO + 16 * i, o);
                            }
                            tmem_st_wait();
                        }
                    } else {  // the last weights are read
                        bar_wait(&sh.pv_done, (n_tile - 1u) & 1u, abort_flag, p.err);
                    }
                    float most = -INFINITY;
                    __half2 most_p = __float2half2_rn(0.0f);
                    const __half2 up = __float2half2_rn(kPartScale);
#pragma unroll 1
                    for (int c = 0; c < pc.n_rows; c += 16) {
                        scores(c);
                        uint32_t pk[kParts][4];
                        uint64_t w2[8];
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const ulonglong2 x4 = *reinterpret_cast<const ulonglong2 *>(&sh.xm[c + k]);
                            uint32_t half[kParts][2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float za = __uint_as_float(x[k + 2 * e]), zb = __uint_as_float(x[k + 2 * e + 1]);
                                float a, b;
                                most = fmaxf(fmaxf(most, za), zb);
                                w2[k / 2 + e] = f2(ex2(za), ex2(zb));
                                unf2(mul2(mul2(w2[k / 2 + e], vm2), e ? x4.y : x4.x), a, b);
                                // fp16's eleven bits, as three parts of four: what one
                                // leaves is exact in fp16
                                __half2 rest = __floats2half2_rn(a, b);
                                most_p = __hmax2(most_p, rest);
#pragma unroll
                                for (int part = 0; part < kParts; ++part) {
                                    half[part][e] = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
                                    if (part + 1 == kParts) break;
                                    const __half2 back(__nv_cvt_fp8x2_to_halfraw2(
                                        (__nv_fp8x2_storage_t)half[part][e], __NV_E4M3));
                                    rest = __hmul2(__hsub2(rest, back), up);
                                }
                            }
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                pk[part][k / 4] = half[part][0] | (half[part][1] << 16);
                        }
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            const int at = kParts * (c >> 4) + part;  // block of 16 columns
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             my_p + (at >> 2) * (kTile * 64) + (((at & 3) ^ ((my >> 1) & 3)) << 4)),
                                         "r"(pk[part][0]), "r"(pk[part][1]), "r"(pk[part][2]), "r"(pk[part][3])
                                         : "memory");
                        }
                        // the warp's sums of the rows: half of them go to either half of the lanes
                        float w[16];
#pragma unroll
                        for (int k = 0; k < 8; ++k) unf2(w2[k], w[2 * k], w[2 * k + 1]);
#pragma unroll
                        for (int o = 16; o > 1; o >>= 1) {
                            const bool upper = lane & o;
#pragma unroll
                            for (int k = 0; k < o / 2; ++k) {
                                const float keep = upper ? w[k + o / 2] : w[k], give = upper ? w[k] : w[k + o / 2];
                                w[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                            }
                        }
                        w[0] += __shfl_xor_sync(0xFFFFFFFFu, w[0], 1);
                        if (!(lane & 1)) sh.sums[warp][c + (lane >> 1)] = w[0];
                    }
                    if (again ||
                        !group_any(most > kLazy || fmaxf(__low2float(most_p), __high2float(most_p)) > kCap))
                        break;
                }
                // the scores are read: the next tile's may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_free);
                sum[0] += sh.sums[warp][2 * lane];  // (of rows that are not there: unused)
                sum[1] += sh.sums[warp][2 * lane + 1];
                // What a row does not see must not reach it, but a product 0 * NaN would: the
                // values past the end, and NaN codes where some row may be masked, become
                // zero; the epilogue adds the NaN to the rows that do see it.
                if (t >= pc.guard_from) {
                    const uint32_t kt = tiles_done + (uint32_t)(t - pc.t0), i = kt % kStages;
                    bar_wait(&sh.raw_full[1][i], (kt / kStages) & 1u, abort_flag, p.err);
                    const uint32_t src = sm_raw[1] + i * C::kRawBytes + my * kD;
                    const bool live = l < pc.rq.len;
                    bool found = false;
#pragma unroll 2
                    for (int c = 0; c < kD / 16; ++c) {
                        const uint32_t a = src + ((kD == 128 ? c ^ (my & 7) : c ^ ((my >> 1) & 3)) << 4);
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(a));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (!live) w[k] = 0u;
                            const uint32_t nan = __vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            found |= nan != 0;
                            w[k] &= ~nan;
                        }
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]),
                                     "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                    if (found) *(volatile int *)&sh.poison = (int)n_piece;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full);
            }
            // ---- epilogue ----
            const int32_t n = pc.t1 - pc.t0;
            tiles_done += n;
            __syncwarp();
            sh.sums[warp][2 * lane] = sum[0];
            sh.sums[warp][2 * lane + 1] = sum[1];
            bar_wait(&sh.pv_done, (n_tile - 1u) & 1u, abort_flag, p.err);
            group_sync();
            tc_fence_after();
            float *part = pc.slot >= 0 ? p.part + pc.slot * part_slot_floats(p.part_rows, kD) : nullptr;
            auto out_row = [&](int r) {
                const uint32_t x = pc.rem0 + r, dt = (x * magic) >> 16;
                return (int64_t)(pc.rq.t0 + pc.tok0 + (int)dt) * p.q_heads + pc.h * p.group + (int)(x - dt * p.group);
            };
            if (my < pc.n_rows) {  // a row's statistics, and the factor of its sums
                float all = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; ++w) all += sh.sums[w][my];
                sh.fix_o[my] = pow2_int((int)row_x) * (part ? 1.0f : all == 0.0f ? 0.0f : 1.0f / all);
                if (part) {
                    part[part_stats(p.part_rows, kD) + my] = row_base;
                    part[part_stats(p.part_rows, kD) + p.part_rows + my] = all;
                } else if (p.lse) {
                    p.lse[out_row(my)] = all == 0.0f ? -INFINITY : (row_base + log2f(all)) * 0.6931471805599453f;
                }
            }
            group_sync();
            // eight rows at a time; this thread has channel `my`
#pragma unroll 1
            for (int r0 = 0; r0 < pc.n_rows; r0 += 8) {
                float o[8];
                uint32_t a[kParts][8];
#pragma unroll
                for (int q = 0; q < kParts; ++q)
                    tmem_ld8(tO + (r0 >> 4) * (16 * kParts) + 16 * q + (r0 & 15), a[q]);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < kParts; ++q) tmem_tie8(a[q]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    o[k] = fmaf(fmaf(__uint_as_float(a[2][k]), 1.0f / kPartScale, __uint_as_float(a[1][k])),
                                1.0f / kPartScale, __uint_as_float(a[0][k])) * sh.fix_o[r0 + k];
                if (kD == 64 && my >= kD) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (r0 + k >= pc.n_rows) break;
                    if (part)
                        part[((int64_t)(my >> 2) * p.part_rows + r0 + k) * 4 + (my & 3)] = o[k];
                    else
                        ((__nv_bfloat16 *)p.out)[out_row(r0 + k) * kD + my] = __float2bfloat16_rn(o[k]);
                }
            }
            if (*(volatile int *)&sh.poison == (int)n_piece) {
                __threadfence_block();
                group_sync();
                if (my < pc.n_rows) {
                    const int r = my;
                    add_poison<kD, true, true>(p, pc.rq, pc.b, pc.h, pc.tok0 + (int)(((pc.rem0 + r) * magic) >> 16),
                                               max(pc.t0, pc.guard_from) * kTile, min(pc.t1 * kTile, pc.rq.len), 0, kD,
                                               part ? part + 4 * r : nullptr,
                                               (__nv_bfloat16 *)p.out + out_row(r) * kD);
                }
            }
            // the sums are read: the next piece's first barrier says so
            tc_fence_before();
            ++n_piece;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int kD> dflash2_status launch_one(const DeviceInfo &di, Params p, cudaStream_t st) {
    using C = Few<kD>;
    auto fn = few_kernel<kD>;
    static std::atomic<uint64_t> done{0};
    const dflash2_status allowed = allow_smem(fn, C::kSmem, di.device, done);
    if (allowed != DFLASH2_OK) return allowed;
    CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {
        const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)p.page_size, (uint64_t)p.num_pages * p.kv_heads};
        const uint64_t strides[2] = {kD, (uint64_t)kD * p.page_size};
        const uint32_t box[3] = {(uint32_t)kD, (uint32_t)(p.page_size < kTile ? p.page_size : kTile), 1u};
        const dflash2_status s = encode_tmap_3d(&maps[i], i ? p.v : p.k, dims, strides, box, 1);
        if (s != DFLASH2_OK) return s;
    }
    p.row_shift = kRowShift;
    const int64_t rows = (int64_t)p.total_q * p.group;
    for (int i = 0; i < 4; ++i) {
        p.tile_units[i] = kTileUnits[i];
        p.item_units[i] = kItemUnits[i];
        if (i == 0 || rows > kRows / 4 * i) p.most_units = kTileUnits[i];
    }
    p.n_cta = 2 * di.sm_count;
    p.part_rows = kRows;
    launch_k(fn, dim3((unsigned)p.n_cta), dim3(C::kThreads), C::kSmem, st, p, maps[0], maps[1]);
    const dflash2_status s = launch_status();
    if (s != DFLASH2_OK) return s;
    return launch_combine(di, p, DFLASH2_BF16, st);
}

}  // namespace

dflash2_status launch_few(const DeviceInfo &di, const Params &p, cudaStream_t st) {
    return p.head_dim == 64 ? launch_one<64>(di, p, st) : launch_one<128>(di, p, st);
}

}  // namespace attn
}  // namespace dflash2
