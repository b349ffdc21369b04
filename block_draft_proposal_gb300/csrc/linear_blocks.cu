// Matrix product of E4M3 codes with a scale per block of 128:
//
//   y[m, n] = sum_b xs[m, b] * ws[n / 128, b] * sum_{k in b} dec(xq[m, k]) * dec(wq[n, k])
//
// The tensor cores multiply and add one block of 128 at a time (four MMAs of K = 32 into a
// fresh TMEM accumulator); the epilogue warps read it, scale it and add it to sums that
// they keep in registers in fp32, while the MMAs of the next block fill the other
// accumulator.  Every scale is an fp32 number, so the scaling cannot be left to block-scaled
// MMAs, whose scales are powers of two.
//
// Two kernels, by the rows (launch_linear):
//   linear_pair_kernel  65 rows and more: CTA pairs (M = 256 rows of x, kCols outputs).
//   linear_few_kernel   fewer: the weights are the MMA's M side, 128 a CTA, and the rows of
//                       x its N side; the blocks are split over a cluster's CTAs, which
//                       send one another their sums through distributed shared memory.
// (64 rows on codes, few-row kernel and pairs: x 4096 x 1024 5.7 and 7.9 us, x 5120 x 7168 11.7 and 12.3, x 7168 x
// 7168 14.1 and 15.6, x 4096 x 28672 25.1 and 26.7; x 4096 x 6144, whose tiles fill the pairs to two
// thirds, 11.4 and 10.6.  40 rows x 4096 x 6144 10.0 and 10.4.)
//
// Few rows are bound by the weights' bytes and the latencies around them, many by the
// accumulators' round trip: a block's MMAs take a pair 512 cycles at 256 columns, and from
// their issue to the accumulator's return some 1500 pass for two accumulators (last MMA to
// the waiting warps 200, two TMEM loads and half the sums 370 to 440, the slowest of
// sixteen warps 250 more), so a block takes about 750.
// Measured on codes (graph replays): one row x 4096 x 6144 7.7 us, 3.3 TB/s; x 4096 x 28672
// 20 us, 5.8 TB/s; 256 rows x 4096 x 6144 11.5 us; 512 16.6; 1536 x 5120 x 7168 48 us, 2.4
// PFLOP/s; 8192 x 7168 x 7168 259 to 270 us, 3.1 to 3.2 PFLOP/s, and 311, 2.7, once the power cap
// holds the SMs at 1.5 GHz (some 0.2 s of such calls).
#include <type_traits>

#include "rows.cuh"
#include "stage_ring.h"
#include "tcgen05.cuh"

namespace dflash2 {
namespace {

struct LinearArgs {
    const float *xs, *ws;
    const void *x;  // rows that the kernel quantises itself (linear_few_kernel with a type X)
    int64_t x_stride;
    int32_t n_in;
    int32_t rows, n_out, blocks;  // blocks of 128 along in_features
    void *y;
    int32_t *err;
    int32_t m_tiles, n_tiles, stages;
    bool vec;    // results go out by TMA (rows of y are 16-byte aligned)
    bool early;  // the weights may be read before the kernel before this one is done
};

constexpr uint32_t kBoxBytes = 128 * 128;  // 128 rows of one block
constexpr int kMaxStages = 8;

__device__ __forceinline__ bool wait_drain(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kWaitLimitCycles) return false;
    return true;
}
// What a producer waits for before its CTA may leave: the last use of each stage, of its blocks
// first, first + step, ... below `end`.  A commit arrives on `empty` in the shared memory of
// every CTA that loads the stage whenever its MMAs are done, and only a producer that takes the
// stage again has waited for it; a CTA that left before would have it arrive on whatever lies
// there next.  Once it is there, the copies have landed and the MMAs have read them.  Where a role has
// given up, the copies alone (`landed`: the CTA whose barriers count them).  All waits are bounded.
__device__ __forceinline__ void drain_stages(uint64_t *full, uint64_t *empty, uint32_t first, uint32_t step,
                                             uint32_t end, uint32_t stages, bool landed, volatile int *abort_flag,
                                             int32_t *err) {
    for (uint32_t k = ring_last_uses(first, step, end, stages); k < end; k += step)
        if (!bar_wait(&empty[k % stages], ring_parity(k, stages), abort_flag, err) && landed)
            wait_drain(&full[k % stages], ring_parity(k, stages));
}

// ---- many rows -----------------------------------------------------------------
// Roles (384 threads, one CTA per SM, persistent over tiles): warps 0 and 3 load, warps 1
// and 2 of the leader issue the MMAs (two of each, for the even and the odd blocks: one
// thread's waits, copies and commits take longer than a block's MMAs), warps 4 to 11 scale
// and add: four lane quarters, each with two warps that take half of the tile's columns,
// kCols / 2 sums a thread.  As many accumulators as TMEM holds, 2 at 256 columns.
constexpr int kPairThreads = 384;
constexpr int kPairEpiWarps = 8;
constexpr int kIssuers = 2;

template <int kCols> constexpr uint32_t kPairStage = kBoxBytes + kCols / 2 * 128;
constexpr uint32_t kOutBytes = 4096;  // an epilogue warp's results on their way out

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, 0}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 results of the lane's row, in 16-byte units of T; into row `lane` of a [32][32] tile
// with the store's swizzle (rows of 64 bytes: unit ^ (row / 2) % 4; of 128: unit ^ row % 8).
__device__ __forceinline__ void stage32(uint8_t *tile, int lane, const uint64_t *v, __nv_bfloat16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unf2(v[4 * i + j], lo, hi);
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
            w[j] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(tile + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void stage32(uint8_t *tile, int lane, const uint64_t *v, float) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float4 f;
        unf2(v[2 * i], f.x, f.y);
        unf2(v[2 * i + 1], f.z, f.w);
        *reinterpret_cast<float4 *>(tile + lane * 128 + ((i ^ (lane & 7)) << 4)) = f;
    }
}

template <typename T, int kCols>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_y, const LinearArgs a) {
    constexpr int kHalf = kCols / 2, kChunks = kHalf / 32;
    static_assert(128 % kHalf == 0, "a thread's columns lie in one block of the weights");
    constexpr uint32_t kAccCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256, kBufs = 512 / kAccCols;
    constexpr uint32_t kStage = kPairStage<kCols>;
    extern __shared__ uint8_t dsmem[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kBufs], acc_empty[kBufs], drain[kIssuers];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~(uintptr_t)1023);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (uint32_t i = 0; i < kBufs; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 2 * kPairEpiWarps);
        for (int i = 0; i < kIssuers; ++i) mbar_init(&drain[i], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(&tmem_slot, 512);
        tmem_relinquish_pair();
    }
    if (warp == 1 && lane == 0) prefetch_tmap(&tm_x), prefetch_tmap(&tm_w), prefetch_tmap(&tm_y);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t tmem = tmem_slot;
    const int total = a.m_tiles * a.n_tiles, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    // Tiles in groups of kGroup row tiles, row tiles fastest: the tiles at work together
    // share x and weight rows in L2.
    constexpr int kGroup = 8;
    const auto tile_of = [&](int w, int *m, int *n) {
        const int g = w / (kGroup * a.n_tiles), r = w - g * kGroup * a.n_tiles;
        const int rows = min(kGroup, a.m_tiles - g * kGroup);
        *n = r / rows;
        *m = g * kGroup + r - *n * rows;
    };

    if (warp < 4) {
        regs_give<56>();
        // of the pair's blocks, tile after tile, every other one
        const uint32_t all = (uint32_t)((int64_t)((total - pair + pairs - 1) / pairs) * a.blocks);
        // (whole warps run the loops, so that what a copy or an MMA takes stays in uniform
        // registers, and one lane issues)
        if (warp == 0 || warp == 3) {
            const uint32_t first = warp == 0 ? 0 : 1;
            uint32_t it = first, s = first, ph = 1;  // the first pass finds every stage free
            int w = pair, b = (int)first, m, n;
            tile_of(w, &m, &n);
            for (; it < all; it += 2, b += 2) {
                while (b >= a.blocks) {
                    b -= a.blocks, w += pairs;
                    tile_of(w, &m, &n);
                }
                if (!bar_wait(&empty[s], ph, &abort_flag, a.err)) break;
                if (elect_one()) {
                    const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStage);
                    uint8_t *st = smem + s * kStage;
                    tma_load_2d_pair(st, &tm_x, bar, b * 128, m * 256 + (int)rank * 128);
                    tma_load_2d_pair(st + kBoxBytes, &tm_w, bar, b * 128, n * kCols + (int)rank * kHalf);
                }
                __syncwarp();
                s += 2;
                if (s >= (uint32_t)a.stages) s -= (uint32_t)a.stages, ph ^= 1u;
            }
            // the leader's barriers count the copies of both CTAs
            drain_stages(full, empty, first, 2, min(it, all), (uint32_t)a.stages, rank == 0, &abort_flag, a.err);
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            const uint32_t idesc = idesc_e4m3(256, kCols), first = (uint32_t)warp - 1;
            const uint64_t xd = sw128_desc(smem_u32(smem)), wd = sw128_desc(smem_u32(smem + kBoxBytes));
            uint32_t s = first, ph = 0;
            bool ok = true;
            for (uint32_t it = first; it < all; it += 2) {
                const uint32_t i = it % kBufs, d = tmem + i * kAccCols;
                // the operands first: they are there long before the accumulator is free
                if (!bar_wait(&full[s], ph, &abort_flag, a.err) ||
                    !bar_wait(&acc_empty[i], ((it / kBufs) & 1u) ^ 1u, &abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t x0 = xd + s * (kStage >> 4), w0 = wd + s * (kStage >> 4);
                    tc_mma_f8_pair(d, x0, w0, idesc, 0u);
                    tc_mma_f8_pair(d, x0 + 2, w0 + 2, idesc, 1u);
                    tc_mma_f8_pair(d, x0 + 4, w0 + 4, idesc, 1u);
                    tc_mma_f8_pair(d, x0 + 6, w0 + 6, idesc, 1u);
                    tc_commit_pair_mc(&acc_full[i], 0x3);
                    tc_commit_pair_mc(&empty[s], 0x3);
                }
                __syncwarp();
                s += 2;
                if (s >= (uint32_t)a.stages) s -= (uint32_t)a.stages, ph ^= 1u;
            }
            if (!ok && elect_one()) {  // the MMAs already issued finish before TMEM is released
                tc_commit_pair(&drain[first]);
                wait_drain(&drain[first], 0);
            }
        }
    } else {
        regs_take<224>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t empty_leader = mapa_shared(smem_u32(acc_empty), 0);
        const uint32_t tbase = tmem + (uint32_t)(half * kHalf) + ((uint32_t)(quarter * 32) << 16);
        uint8_t *out = smem + (uint32_t)a.stages * kStage + (uint32_t)(warp - 4) * kOutBytes;
        uint32_t it = 0, stored = 0;
        bool ok = true;
        for (int w = pair; w < total && ok; w += pairs) {
            int mt, nt;
            tile_of(w, &mt, &nt);
            const int64_t m0 = (int64_t)mt * 256 + (int)rank * 128 + quarter * 32, m = m0 + lane;
            const int n0 = nt * kCols + half * kHalf;
            const float *xs = a.xs + min(m, (int64_t)a.rows - 1) * a.blocks;
            // columns past the end take the last block's scales
            const float *ws = a.ws + (int64_t)(min(n0, a.n_out - 1) / 128) * a.blocks;
            uint64_t sum[kHalf / 2];
#pragma unroll
            for (int i = 0; i < kHalf / 2; ++i) sum[i] = 0;
            float x_next = __ldg(xs), w_next = __ldg(ws);
            for (int b = 0; b < a.blocks; ++b, ++it) {
                const float v = x_next * w_next;
                const uint64_t f = f2(v, v);
                if (b + 1 < a.blocks) {  // the next block's scales, ahead of the wait
                    x_next = __ldg(xs + b + 1);
                    w_next = __ldg(ws + b + 1);
                }
                const uint32_t i = it % kBufs;
                if (!bar_wait(&acc_full[i], (it / kBufs) & 1u, &abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t = tbase + i * kAccCols;
                // two loads of 32 columns in flight; the next two are issued between the
                // sums, so that a block waits for TMEM twice
                uint32_t r[2][32];
                tmem_ld32(t, r[0]);
                if (kChunks > 1) tmem_ld32(t + 32, r[1]);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    if (c % 2 == 0) {
                        tmem_ld_wait();
                        tmem_tie(r[0]);
                        if (c + 1 < kChunks) tmem_tie(r[1]);
                        if (c + 2 >= kChunks) {  // all read: the accumulator goes back
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster_relaxed(empty_leader + 8 * i);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum[16 * c + j] = fma2(f, f2(r[c & 1][2 * j], r[c & 1][2 * j + 1]), sum[16 * c + j]);
                    if (c + 2 < kChunks) tmem_ld32(t + 32 * (c + 2), r[c & 1]);
                }
            }
            if (!ok) break;
            if (a.vec) {
                // 32 columns at a time through shared memory and out by TMA, which writes
                // whole lines while the next tile begins (stores of 16 bytes a lane held the
                // warps up: 349 us in place of 306) and leaves out what is past the end
                constexpr int kBufs = (int)(kOutBytes / (1024 * sizeof(T)));
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    uint8_t *buf = out + (stored++ % kBufs) * (1024 * sizeof(T));
                    if (lane == 0) bulk_wait_read<kBufs - 1>();
                    __syncwarp();
                    stage32(buf, lane, sum + 16 * c, T());
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (m0 < a.rows && n0 + 32 * c < a.n_out)
                            tma_store_3d(&tm_y, smem_u32(buf), (n0 + 32 * c) * (int)sizeof(T), (int)m0);
                        bulk_commit();
                    }
                }
            } else {
                // rows that TMA cannot begin: 32 columns at a time through shared memory
                // (value (r, j) at word r, j ^ r), a lane a column on the way out (a lane a
                // row: 300 x 1936 x 1001 14.5 us, so 7.5)
                float *tile = reinterpret_cast<float *>(out);
                const int left = (int)min((int64_t)32, (int64_t)a.rows - m0);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float lo, hi;
                        unf2(sum[16 * c + j], lo, hi);
                        tile[lane * 32 + ((2 * j) ^ lane)] = lo;
                        tile[lane * 32 + ((2 * j + 1) ^ lane)] = hi;
                    }
                    __syncwarp();
                    const int n = n0 + 32 * c + lane;
                    T *y = (T *)a.y + m0 * a.n_out + n;
                    if (n < a.n_out)
#pragma unroll 8
                        for (int r = 0; r < left; ++r) from_f32(y + (int64_t)r * a.n_out, tile[r * 32 + (lane ^ r)]);
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still touch its shared memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---- few rows --------------------------------------------------------------------
// Roles (192 threads): warp 0 loads, warp 1 issues the MMAs, warps 2 to 5 scale and add:
// a thread owns one output column and kN rows of x.  A block's factors xs * ws lie in a
// table of the warp's own, made from scales loaded two blocks ahead.
//
// With a type X (up to 16 rows, 320 threads) x is not codes yet: warps 6 to 9 take every
// fourth block each, quantise its rows into the stage and leave their factors beside it.
// Every CTA does this for its own blocks, which costs less than the launch of a
// quantisation before (one row x 4096 x 6144: 8.0 us in place of 9.3).
constexpr int kFewThreads = 192, kFewQuantThreads = 320;
constexpr int kFewMaxSplit = 8;

template <int kN> constexpr uint32_t kFewStage = kBoxBytes + kN * 128;
template <typename X> constexpr bool kQuantises = !std::is_same<X, uint8_t>::value;  // uint8_t: codes

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <typename T, int kN, typename X>
__global__ void __launch_bounds__(kQuantises<X> ? kFewQuantThreads : kFewThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const LinearArgs a, const int split) {
    constexpr int kChunk = kN < 32 ? kN : 32, kPer = (kN + 31) / 32;
    constexpr uint32_t kAccCols = kN < 32 ? 32 : kN, kBufs = 256 / kAccCols;
    constexpr uint32_t kStage = kFewStage<kN>;
    extern __shared__ uint8_t dsmem[];
    constexpr bool kQuant = kQuantises<X>;
    static_assert(!kQuant || kN == 16, "a quantising warp takes sixteen rows");
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kBufs], acc_empty[kBufs], drain;
    __shared__ uint64_t factor_full[kBufs];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    // codes: [warp][block & 1]; quantised here: [accumulator], one for all warps
    __shared__ __align__(16) float factor[8][kN];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~(uintptr_t)1023);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % split;  // the CTA's rank in its cluster
    const int nt = blockIdx.x / split;    // its tile of 128 output columns
    const int b0 = (int)((int64_t)a.blocks * rank / split), b1 = (int)((int64_t)a.blocks * (rank + 1) / split);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], kQuant ? 2 : 1), mbar_init(&empty[s], 1);
        for (uint32_t i = 0; i < kBufs; ++i)
            mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 4), mbar_init(&factor_full[i], 1);
        mbar_init(&drain, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, 256);
        tmem_relinquish();
    }
    if (warp == 1 && lane == 0) {
        if (!kQuant) prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // the rows' scales and codes wait for the kernel before; the weights need not where
    // that one is this call's own quantisation
    if (!(a.early && warp == 0)) grid_dep_wait();
    if (warp != 0) grid_dep_launch();

    float sum[kN];
    if (warp == 0) {
        const auto arm = [&](int b, uint32_t s) {
            mbar_arrive_expect_tx(&full[s], kQuant ? kBoxBytes : kStage);
            tma_load_2d(smem + s * kStage, &tm_w, &full[s], b * 128, nt * 128);
        };
        const auto load_x = [&](int b, uint32_t s) {
            if (!kQuant) tma_load_2d(smem + s * kStage + kBoxBytes, &tm_x, &full[s], b * 128, 0);
        };
        const int first = min(b1 - b0, a.stages);  // stages that nothing has used yet
        if (elect_one())
            for (int i = 0; i < first; ++i) arm(b0 + i, (uint32_t)i);
        __syncwarp();
        if (a.early) grid_dep_wait();
        if (elect_one())
            for (int i = 0; i < first; ++i) load_x(b0 + i, (uint32_t)i);
        __syncwarp();
        uint32_t issued = (uint32_t)first, s = 0, ph = 0;
        for (int b = b0 + first; b < b1; ++b) {
            if (!bar_wait(&empty[s], ph, &abort_flag, a.err)) break;
            if (elect_one()) {
                arm(b, s);
                load_x(b, s);
            }
            __syncwarp();
            ++issued;
            if (++s == (uint32_t)a.stages) s = 0, ph ^= 1u;
        }
        drain_stages(full, empty, 0, 1, issued, (uint32_t)a.stages, true, &abort_flag, a.err);
    } else if (warp == 1) {
        const uint32_t idesc = idesc_e4m3(128, kN);
        const uint64_t wd = sw128_desc(smem_u32(smem)), xd = sw128_desc(smem_u32(smem + kBoxBytes));
        uint32_t s = 0, ph = 0;
        for (int b = b0; b < b1; ++b) {
            const uint32_t it = (uint32_t)(b - b0), i = it % kBufs;
            if (!bar_wait(&full[s], ph, &abort_flag, a.err) ||
                !bar_wait(&acc_empty[i], ((it / kBufs) & 1u) ^ 1u, &abort_flag, a.err)) {
                if (elect_one()) {
                    tc_commit(&drain);
                    wait_drain(&drain, 0);
                }
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t w0 = wd + s * (kStage >> 4), x0 = xd + s * (kStage >> 4);
                const uint32_t d = tmem + i * kAccCols;
                tc_mma_f8(d, w0, x0, idesc, 0u);
                tc_mma_f8(d, w0 + 2, x0 + 2, idesc, 1u);
                tc_mma_f8(d, w0 + 4, x0 + 4, idesc, 1u);
                tc_mma_f8(d, w0 + 6, x0 + 6, idesc, 1u);
                tc_commit(&acc_full[i]);
                tc_commit(&empty[s]);
            }
            __syncwarp();
            if (++s == (uint32_t)a.stages) s = 0, ph ^= 1u;
        }
    } else if (warp < 6) {
        const int quarter = warp & 3;
        float(*table)[kN] = kQuant ? factor : factor + 2 * quarter;
        const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16);
        const float *ws = a.ws + (int64_t)nt * a.blocks;
        const float *xs[kPer];
        bool in[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int m = i * 32 + lane;
            in[i] = m < a.rows;
            xs[i] = a.xs + (int64_t)(in[i] ? m : 0) * a.blocks;
        }
        const auto scales = [&](int b, float (&f)[kPer]) {
            const float w = __ldg(ws + b);
#pragma unroll
            for (int i = 0; i < kPer; ++i) f[i] = in[i] ? __ldg(xs[i] + b) * w : 0.0f;
        };
        uint64_t acc[kN / 2];
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) acc[i] = 0;
        float f0[kPer] = {}, f1[kPer] = {};  // of this block and the next
        if (!kQuant && b0 < b1) scales(b0, f0);
        if (!kQuant && b0 + 1 < b1) scales(b0 + 1, f1);
        for (int b = b0; b < b1; ++b) {
            const uint32_t it = (uint32_t)(b - b0), i = it % kBufs, at = kQuant ? i : it & 1u;
            if constexpr (!kQuant) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    if (k * 32 + lane < kN) table[at][k * 32 + lane] = f0[k];
                    f0[k] = f1[k];
                }
                if (b + 2 < b1) scales(b + 2, f1);
                __syncwarp();
            } else if (!bar_wait(&factor_full[i], (it / kBufs) & 1u, &abort_flag, a.err)) {
                break;
            }
            if (!bar_wait(&acc_full[i], (it / kBufs) & 1u, &abort_flag, a.err)) break;
            tc_fence_after();
            const uint32_t t = tbase + i * kAccCols;
#pragma unroll
            for (int c = 0; c < kN / kChunk; ++c) {
                uint32_t r[kChunk];
                if constexpr (kChunk == 32)
                    tmem_ld32(t + 32 * c, r);
                else
                    tmem_ld16(t, r);
                tmem_ld_wait();
                if constexpr (kChunk == 32)
                    tmem_tie(r);
                else
                    tmem_tie16(r);
                float4 fs[kChunk / 4];  // read before they go back with the accumulator
#pragma unroll
                for (int j = 0; j < kChunk / 4; ++j)
                    fs[j] = *reinterpret_cast<const float4 *>(&table[at][kChunk * c + 4 * j]);
                if (c + 1 == kN / kChunk) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[i]);
                }
#pragma unroll
                for (int j = 0; j < kChunk / 4; ++j) {
                    const float4 f = fs[j];
                    uint64_t *s2 = acc + (kChunk * c) / 2 + 2 * j;
                    s2[0] = fma2(f2(f.x, f.y), f2(r[4 * j], r[4 * j + 1]), s2[0]);
                    s2[1] = fma2(f2(f.z, f.w), f2(r[4 * j + 2], r[4 * j + 3]), s2[1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) unf2(acc[i], sum[2 * i], sum[2 * i + 1]);
    } else if constexpr (kQuant) {
        // Sixteen lanes a row, two rows at a time; the codes go where the copy's swizzle
        // would have put them.  Rows past the last are not written: they are columns of the
        // product that nothing reads.
        const int q = warp - 6, l = lane & 15, live = a.rows;
        const X *x = (const X *)a.x;
        for (int b = b0 + q; b < b1; b += 4) {
            const uint32_t it = (uint32_t)(b - b0), i = it % kBufs;
            const uint32_t s = it % (uint32_t)a.stages, ph = (it / (uint32_t)a.stages) & 1u;
            const int col = b * 128 + l * 8;
            Raw8<X> raw[kN / 2];
#pragma unroll
            for (int u = 0; u < kN / 2; ++u) {
                const int r = 2 * u + (lane >> 4);
                raw[u] = Raw8<X>{};
                if (r < live && col < a.n_in) raw[u] = load_raw8(x + r * a.x_stride + col);
            }
            const float w = __ldg(a.ws + (int64_t)nt * a.blocks + b);
            if (!bar_wait(&empty[s], ph ^ 1u, &abort_flag, a.err) ||
                !bar_wait(&acc_empty[i], ((it / kBufs) & 1u) ^ 1u, &abort_flag, a.err))
                break;
            uint8_t *codes = smem + s * kStage + kBoxBytes;
            const auto put = [&](int r, uint2 c) {
                if (r < live)
                    *reinterpret_cast<uint2 *>(codes + r * 128 + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8) = c;
            };
            if (live <= 2) {
                float v[8], scale;
                as_floats(raw[0], v);
                put(lane >> 4, quantise_block(v, &scale));
                if (l == 0) factor[i][lane >> 4] = scale * w;
            } else {
#pragma unroll
                for (int u = 0; u < kN / 2; u += kQuantUnroll) {
                    if (2 * u >= live) break;  // the whole warp
                    float v[kQuantUnroll][8], scale;
                    uint2 c[kQuantUnroll];
#pragma unroll
                    for (int k = 0; k < kQuantUnroll; ++k) as_floats(raw[u + k], v[k]);
                    quantise_blocks(v, &scale, c);
#pragma unroll
                    for (int k = 0; k < kQuantUnroll; ++k) put(2 * (u + k) + (lane >> 4), c[k]);
                    if ((l & 3) == 0) factor[i][2 * (u + quant_lane()) + (lane >> 4)] = scale * w;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]), mbar_arrive(&factor_full[i]);
        }
    }

    // The sums of the cluster's CTAs, added in the order of the blocks: row j of x is CTA j %
    // split's, and every CTA sends it its sums (the stages, done with everywhere, hold
    // them).  Sent sums do not wait for one another; fetched ones did, 6 us for 64 rows.
    const bool scales_and_adds = warp >= 2 && warp < 6;
    const int row = (warp & 3) * 32 + lane;  // their output column in the tile
    const int64_t n = (int64_t)nt * 128 + row;
    const int live = a.rows;
    T *y = (T *)a.y + n;
    tc_fence_before();
    __syncthreads();  // the loads have landed and been read, on the failing path too
    if (split == 1) {
        if (scales_and_adds && n < a.n_out) {
#pragma unroll
            for (int j = 0; j < kN; ++j)
                if (j < live) from_f32(y + (int64_t)j * a.n_out, sum[j]);
        }
    } else {
        float *part = reinterpret_cast<float *>(smem);  // [sender][slot][128]
        const int slots = (kN + split - 1) / split;
        cluster_sync();
        if (scales_and_adds) {
            const uint32_t mine = smem_u32(part) + (uint32_t)((rank * slots * 128 + row) * 4);
            int to = 0, slot = 0;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                if (j < live) st_cluster(mapa_shared(mine + (uint32_t)slot * 512, (uint32_t)to), sum[j]);
                if (++to == split) to = 0, ++slot;
            }
        }
        __syncwarp();
        cluster_sync();
        if (scales_and_adds && n < a.n_out) {
#pragma unroll 4
            for (int s = 0; s < (live - rank + split - 1) / split; ++s) {
                float v = 0.0f;
#pragma unroll
                for (int c = 0; c < kFewMaxSplit; ++c)
                    if (c < split) v += part[(c * slots + s) * 128 + row];
                from_f32(y + (int64_t)(s * split + rank) * a.n_out, v);
            }
        }
    }
    __syncwarp();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---- launches ----------------------------------------------------------------------
constexpr int kSmemMost = 226 * 1024;  // with the barriers and the 1 KB the system takes: 227

template <typename T, int kCols>
dflash2_status launch_pair(const DeviceInfo &di, const uint8_t *xq, const uint8_t *wq, int32_t n_in, LinearArgs a,
                           cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    constexpr uint32_t stage = kPairStage<kCols>;
    constexpr uint32_t outs = 8 * kOutBytes;
    a.stages = min(kMaxStages, (int)((kSmemMost - 1024 - outs) / stage));
    a.m_tiles = (a.rows + 255) / 256, a.n_tiles = (a.n_out + kCols - 1) / kCols;
    const int total = a.m_tiles * a.n_tiles;  // below 2^27 (shape_ok)
    CUtensorMap tm_x, tm_w, tm_y;
    dflash2_status s = encode_tmap_2d(&tm_x, xq, (uint64_t)a.rows, (uint64_t)n_in, 128, 1);
    if (s == DFLASH2_OK) s = encode_tmap_2d(&tm_w, wq, (uint64_t)a.n_out, (uint64_t)n_in, kCols / 2, 1);
    // results as bytes, so that one box serves both types
    const uint64_t bytes = (uint64_t)a.n_out * sizeof(T);
    a.vec = aligned16(a.y) && bytes % 16 == 0 && bytes * a.rows < 1ull << 40;
    tm_y = tm_x;
    if (s == DFLASH2_OK && a.vec)
        s = encode_tmap_3d(&tm_y, a.y, {bytes, (uint64_t)a.rows, 1}, {bytes, bytes * a.rows},
                           {32 * (uint32_t)sizeof(T), 32, 1}, 1);
    if (s == DFLASH2_OK) s = allow_smem(linear_pair_kernel<T, kCols>, kSmemMost, di.device, allowed);
    if (s != DFLASH2_OK) return s;
    const int pairs = min(di.sm_count / 2, total);
    launch_k(linear_pair_kernel<T, kCols>, dim3(2 * pairs), dim3(kPairThreads), a.stages * stage + outs + 1024, st,
             tm_x, tm_w, tm_y, a);
    return launch_status();
}

template <typename T, int kN, typename X>
dflash2_status launch_few(const DeviceInfo &di, const uint8_t *xq, const uint8_t *wq, int32_t n_in, LinearArgs a,
                          cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    constexpr uint32_t stage = kFewStage<kN>;
    constexpr int most = 108 * 1024;  // two CTAs per SM
    a.stages = min(kMaxStages, (int)((most - 1024) / stage));
    const int tiles = (a.n_out + 127) / 128;
    // As many CTAs per tile as run at once for all tiles, with two blocks each.  Two CTAs run per SM,
    // but a cluster stays within a group of SMs, which leaves up to two clusters' worth of them idle.
    // One row of 4096: 75 tiles of 4 (300 CTAs of 304) take a second wave, 13.4 us for 9.9 in clusters of 2, 74 do
    // not (9.3 for 9.8); 59 of 5 12.4 for 8.3 in clusters of 4, 58 not; 37 of 8 10.3 for 7.2 in 5, 36 not (6.7).
    // On codes by the CTAs per tile 1 to 8: 48 tiles (4096 x 6144), one row 11.4, 8.6, 8.1, 7.6, 7.7 us, then a
    // second wave (11.6, 11.7, 11.4); 64 rows 15.5, 13.1, 13.4, 12.5, 11.5, then 17.7, 17.5, 16.3; 8 tiles
    // (4096 x 1024) one row 10.6, 7.2, 5.8, 5.0, 4.7, 4.4, 4.2, 3.9.  3, 6 and 7 are left out: where the larger of
    // these do not run at once and they do, one row is within 5 % of the next smaller's time.
    int split = 1;
    for (const int s : {8, 5, 4, 2})
        if (tiles * s <= 2 * di.sm_count - 2 * s && a.blocks >= 2 * s) {
            split = s;
            break;
        }
    CUtensorMap tm_x, tm_w;
    dflash2_status s = encode_tmap_2d(&tm_w, wq, (uint64_t)a.n_out, (uint64_t)n_in, 128, 1);
    tm_x = tm_w;
    if (s == DFLASH2_OK && !kQuantises<X>) s = encode_tmap_2d(&tm_x, xq, (uint64_t)a.rows, (uint64_t)n_in, kN, 1);
    if (s == DFLASH2_OK) s = allow_smem(linear_few_kernel<T, kN, X>, most, di.device, allowed);
    if (s != DFLASH2_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(kQuantises<X> ? kFewQuantThreads : kFewThreads);
    cfg.dynamicSmemBytes = a.stages * stage + 1024;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, linear_few_kernel<T, kN, X>, tm_x, tm_w, a, split);
    return launch_status();
}

template <typename T>
dflash2_status launch_linear(const DeviceInfo &di, const uint8_t *xq, const uint8_t *wq, int32_t n_in,
                             const LinearArgs &a, int32_t x_dtype, cudaStream_t st) {
    if (a.x && x_dtype == DFLASH2_F32) return launch_few<T, 16, float>(di, xq, wq, n_in, a, st);
    if (a.x) return launch_few<T, 16, __nv_bfloat16>(di, xq, wq, n_in, a, st);
    if (a.rows <= 16) return launch_few<T, 16, uint8_t>(di, xq, wq, n_in, a, st);
    if (a.rows <= 32) return launch_few<T, 32, uint8_t>(di, xq, wq, n_in, a, st);
    if (a.rows <= 64) return launch_few<T, 64, uint8_t>(di, xq, wq, n_in, a, st);
    // The tile's width by the time of its waves, one of 64 or 128 columns taken as 0.48 or 0.6 of one
    // of 256.  Measured at 256, 128 and 64 columns (us, and waves): 512 x 4096 x 6144
    // 17.1 (1), 19.2 (2), 22.6 (3); 768 x 7168 x 7168 44.2 (2), 40.2 (3), 49.9 (5); 1024 x 4096 x 6144 29.4 (2), 26.7
    // (3), 41.5 (6); 2048 x 5120 x 7168 49.4 (3), 56.8 (6), 79.7 (12); 8192 x 7168 x 7168 262 (12), 319 (24), 433
    // (48): 0.56 to 0.61 at 128 columns, 0.40 to 0.47 at 64, which are thus taken where they win clearly.
    const int64_t m_tiles = (a.rows + 255) / 256, pairs = di.sm_count / 2;
    const auto waves = [&](int cols) { return (m_tiles * ((a.n_out + cols - 1) / cols) + pairs - 1) / pairs; };
    const double t64 = 0.48 * (double)waves(64), t128 = 0.6 * (double)waves(128), t256 = (double)waves(256);
    if (t64 < t128 && t64 < t256) return launch_pair<T, 64>(di, xq, wq, n_in, a, st);
    if (t128 < t256) return launch_pair<T, 128>(di, xq, wq, n_in, a, st);
    return launch_pair<T, 256>(di, xq, wq, n_in, a, st);
}

bool shape_ok(int64_t rows, int32_t n_in, int32_t n_out) {
    return rows >= 0 && rows <= 1 << 20 && n_in >= 1 && n_in <= 1 << 20 && n_out >= 1 && n_out <= 1 << 24 &&
           rows * n_in < 1ll << 40 && (int64_t)n_out * n_in < 1ll << 40 && rows * n_out < 1ll << 40;
}
size_t codes_bytes(int64_t rows, int32_t n_in) { return ((size_t)rows * n_in + 255) / 256 * 256; }

}  // namespace
}  // namespace dflash2

using namespace dflash2;

extern "C" size_t dflash2_linear_fp8_blocks_workspace_size(int64_t rows, int32_t in_features, int32_t out_features) {
    if (!shape_ok(rows, in_features, out_features)) return 0;
    return codes_bytes(rows, in_features) + (size_t)rows * ((in_features + 127) / 128) * sizeof(float);
}

extern "C" dflash2_status dflash2_linear_fp8_blocks(const void *x, int64_t x_row_stride, int32_t x_dtype,
                                                    const uint8_t *x_q, const float *x_scale, const uint8_t *w_q,
                                                    const float *w_scale, int64_t rows, int32_t in_features,
                                                    int32_t out_features, int32_t out_dtype, void *out, void *workspace,
                                                    size_t ws_bytes, int32_t *err_word, void *stream) {
    if (out_dtype != DFLASH2_F32 && out_dtype != DFLASH2_BF16) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (!shape_ok(rows, in_features, out_features)) return DFLASH2_ERR_INVALID_ARG;
    if ((x != nullptr) == (x_q != nullptr) && rows > 0) return DFLASH2_ERR_INVALID_ARG;
    dflash2_status st;
    if (!x_q) {
        st = check_quant_blocks(x, x_row_stride, x_dtype, rows, in_features);
        if (st != DFLASH2_OK) return st;
    }
    if (in_features % 16 != 0) return DFLASH2_ERR_MISALIGNED;
    if (rows == 0) return DFLASH2_OK;
    if ((x_q && !x_scale) || !w_q || !w_scale || !out) return DFLASH2_ERR_INVALID_ARG;
    if ((x_q && (!aligned16(x_q) || !aligned_to(x_scale, 4))) || !aligned16(w_q) || !aligned_to(w_scale, 4) ||
        !aligned_to(out, out_dtype == DFLASH2_F32 ? 4 : 2) || !aligned_to(err_word, 4))
        return DFLASH2_ERR_MISALIGNED;
    if (!x_q && (!workspace || !aligned_to(workspace, 256) ||
                 ws_bytes < dflash2_linear_fp8_blocks_workspace_size(rows, in_features, out_features)))
        return DFLASH2_ERR_WORKSPACE;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LinearArgs a{};
    const int64_t el = x_dtype == DFLASH2_F32 ? 4 : 2;
    if (!x_q && rows <= 16 && aligned16(x) && (rows == 1 || x_row_stride * el % 16 == 0)) {
        a.x = x, a.x_stride = x_row_stride, a.n_in = in_features;  // quantised as it is multiplied
    } else if (!x_q) {
        uint8_t *q = static_cast<uint8_t *>(workspace);
        float *scale = reinterpret_cast<float *>(q + codes_bytes(rows, in_features));
        st = launch_quant_blocks_e4m3(x, x_row_stride, x_dtype, rows, in_features, q, scale, s);
        if (st != DFLASH2_OK) return st;
        x_q = q, x_scale = scale;
        a.early = true;
    }
    a.xs = x_scale, a.ws = w_scale;
    a.rows = (int32_t)rows, a.n_out = out_features, a.blocks = (in_features + 127) / 128;
    a.y = out, a.err = err_word;
    return out_dtype == DFLASH2_F32 ? launch_linear<float>(di, x_q, w_q, in_features, a, x_dtype, s)
                                    : launch_linear<__nv_bfloat16>(di, x_q, w_q, in_features, a, x_dtype, s);
}
