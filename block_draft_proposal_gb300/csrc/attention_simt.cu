// Attention on CUDA cores: fp32 inputs, and every head_dim, page size and
// alignment the tensor-core kernel does not take.
//
// One pass over the keys in tiles of 64 with the running maximum m and sum l
// of the softmax (log2 domain): S = scale log2(e) Q K^T, m' = max(m, max S),
// P = 2^(S - m'), O = O 2^(m - m') + P V, l = l 2^(m - m') + sum P.  256
// threads as 16 x 16: thread (ty, tx) has kRows / 16 rows and the keys tx + 16 j
// of S, and the same rows with four of every 64 values of O, so a row's
// statistics are 16-lane shuffles and every shared-memory read is a broadcast or
// 16 bytes per lane without conflicts (K rows are padded by four floats).
//
// Bound by fp32 FMAs once rows fill the tile (kRows = 64) and by HBM for few
// rows (kRows = 16: 32 FMA cycles per key against 45 cycles of HBM time for an
// fp32 key and value of head_dim 128).  Short calls are bound by one tile after the
// other: 64 keys of head_dim 64 take 11400 cycles, 2100 for the loads (four in flight per
// thread), 4200 for S and 3700 for O, and blocks of 16 rows no less, since every warp
// reads the whole tile from shared memory.  Three fp32 prompts of up to 301 tokens with 8
// heads of 64 take 34 us; one of 1500 tokens with 8 heads of 128 265 us, 17 TFLOP/s.
#include "attention.cuh"

namespace dflash2 {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr int kItemUnits = 1;  // units of an item's start and end, beside its key tiles

__host__ __device__ constexpr int simt_smem_floats(int rows, int dmax) {
    return rows * dmax + kKeys * (dmax + 4) + kKeys * dmax + rows * kKeys;
}

// Rows of a tile into shared memory as fp32, `width` of kDMax columns live and
// the rest zero.  row_ptr(r) gives the row's elements or NULL for a zero row;
// row_mul(r) scales it.
template <typename T, int kDMax, typename PtrF, typename MulF>
__device__ __forceinline__ void stage_rows(float *dst, int pitch, int n, int width, bool vec,
                                           PtrF row_ptr, MulF row_mul) {
    constexpr int kChunks = kDMax / 4, kFly = 4;  // loads in flight per thread
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < n * kChunks; i0 += kFly * kThreads) {
        float x[kFly][4];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int i = i0 + f * kThreads, r = i / kChunks, c = (i % kChunks) * 4;
            const T *src = i < n * kChunks ? row_ptr(r) : nullptr;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[f][k] = 0.0f;
            if (!src || c >= width) continue;
            if (vec) {  // width % 4 == 0 and four elements aligned
                if constexpr (sizeof(T) == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(src + c);
                    x[f][0] = q.x, x[f][1] = q.y, x[f][2] = q.z, x[f][3] = q.w;
                } else {
                    T e[4];
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(src + c);
                    else
                        *reinterpret_cast<uint32_t *>(e) =
                            *reinterpret_cast<const uint32_t *>(src + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[f][k] = as_f32(e[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k < width) x[f][k] = as_f32(src[c + k]);
            }
            const float mul = row_mul(r);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[f][k] *= mul;
        }
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int i = i0 + f * kThreads;
            if (i < n * kChunks)
                *reinterpret_cast<float4 *>(dst + i / kChunks * pitch + i % kChunks * 4) =
                    make_float4(x[f][0], x[f][1], x[f][2], x[f][3]);
        }
    }
}

// The keys [k0, k1) of one item, added up in registers and written as final
// rows (slot < 0) or as partial rows of workspace slot `slot`.
template <typename T, typename C, bool kPaged, int kRows, int kDMax>
__device__ void run_piece(const Params &p, const Request &rq, int32_t b, int32_t h, int32_t rb,
                          int32_t k0, int32_t k1, int64_t slot, float *smem, bool vec_q, bool vec_k,
                          bool *bad_page) {
    constexpr int kPer = kRows / 16;   // rows per thread
    constexpr int kQuads = kDMax / 64; // groups of four output values per thread
    constexpr bool kE4M3 = sizeof(C) == 1;
    float *sq = smem;
    float *sk = sq + kRows * kDMax;
    float *sv = sk + kKeys * (kDMax + 4);
    float *sp = sv + kKeys * kDMax;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int32_t row0 = rb * kRows;
    const int32_t n_rows = (int32_t)min((int64_t)kRows, (int64_t)rq.t * p.group - row0);
    const int d = p.head_dim;

    __syncthreads();  // the previous piece's reads of the shared tiles are over
    stage_rows<T, kDMax>(
        sq, kDMax, kRows, d, vec_q,
        [&](int r) -> const T * {
            if (r >= n_rows) return nullptr;
            const int32_t g = row0 + r;
            return (const T *)p.q + (int64_t)(rq.t0 + g / p.group) * p.q_stride +
                   (int64_t)(h * p.group + g % p.group) * d;
        },
        [&](int) { return p.scale_log2; });

    float o[kPer][kQuads][4];
    float m[kPer], l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][q][e] = 0.0f;
    }

    for (int32_t kt = k0; kt < k1; kt += kKeys) {
        const int nk = min(kKeys, k1 - kt);
        // cache row of key r of the tile, or -1
        auto cache_row = [&](int r) -> int64_t {
            const int32_t l_ = kt + r;
            if (r >= nk || l_ >= rq.len) return -1;
            const int32_t pg = __ldg(p.page_table + (int64_t)b * p.max_pages + l_ / p.page_size);
            if (pg < 0 || pg >= p.num_pages) {
                *bad_page = true;
                return -1;
            }
            return ((int64_t)pg * p.kv_heads + h) * p.page_size + l_ % p.page_size;
        };
        auto key_ptr = [&](int r, const void *base, int64_t stride) -> const C * {
            if constexpr (kPaged) {
                const int64_t at = cache_row(r);
                return at < 0 ? nullptr : (const C *)base + at * d;
            } else {
                if (r >= nk || kt + r >= rq.len) return nullptr;
                return (const C *)base + (int64_t)(rq.t0 + kt + r) * stride + (int64_t)h * d;
            }
        };
        __syncthreads();  // the previous tile's products are over
        stage_rows<C, kDMax>(
            sk, kDMax + 4, kKeys, d, vec_k, [&](int r) { return key_ptr(r, p.k, p.k_stride); },
            [&](int r) { return kE4M3 ? pow2_byte(__ldg(p.k_exp + cache_row(r))) : 1.0f; });
        stage_rows<C, kDMax>(
            sv, kDMax, kKeys, d, vec_k, [&](int r) { return key_ptr(r, p.v, p.v_stride); },
            [&](int r) { return kE4M3 ? pow2_byte(__ldg(p.v_exp + cache_row(r))) : 1.0f; });
        __syncthreads();

        float s[kPer][4];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
        for (int c = 0; c < kDMax; c += 4) {
            float4 kq[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kq[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * (kDMax + 4) + c);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float4 qq = *reinterpret_cast<const float4 *>(sq + (ty * kPer + i) * kDMax + c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(qq.x, kq[j].x, s[i][j]);
                    s[i][j] = fmaf(qq.y, kq[j].y, s[i][j]);
                    s[i][j] = fmaf(qq.z, kq[j].z, s[i][j]);
                    s[i][j] = fmaf(qq.w, kq[j].w, s[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int32_t r = row0 + ty * kPer + i;
            const int32_t tok = r / p.group;
            float top = -INFINITY;
            bool seen[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t pos = kt + tx + 16 * j;
                seen[j] = ty * kPer + i < n_rows && tx + 16 * j < nk &&
                          (kPaged ? sees(p, rq, tok, pos) : pos <= tok);
                if (!seen[j]) s[i][j] = -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float mn = fmaxf(m[i], top);
            // no finite key yet: a base of 0 keeps -inf - base at -inf
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float fix = ex2(m[i] - base);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = seen[j] ? ex2(s[i][j] - base) : 0.0f;
                sp[(ty * kPer + i) * kKeys + tx + 16 * j] = w;
                sum += w;
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
            l[i] = l[i] * fix + sum;
            m[i] = mn;
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][q][e] *= fix;
        }
        __syncwarp();  // a row's 16 threads are in one warp: its weights are written
        // four keys at a time (past nk: weights of zero, and rows of zeros)
        for (int key = 0; key < nk; key += 4) {
            float w[kPer][4];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float4 w4 = *reinterpret_cast<const float4 *>(sp + (ty * kPer + i) * kKeys + key);
                w[i][0] = w4.x, w[i][1] = w4.y, w[i][2] = w4.z, w[i][3] = w4.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 vq[kQuads];
#pragma unroll
                for (int q = 0; q < kQuads; ++q)
                    vq[q] = *reinterpret_cast<const float4 *>(sv + (key + j) * kDMax + 64 * q + 4 * tx);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (w[i][j] != 0.0f) {  // what a row does not see never reaches it, NaN included
#pragma unroll
                        for (int q = 0; q < kQuads; ++q) {
                            o[i][q][0] = fmaf(w[i][j], vq[q].x, o[i][q][0]);
                            o[i][q][1] = fmaf(w[i][j], vq[q].y, o[i][q][1]);
                            o[i][q][2] = fmaf(w[i][j], vq[q].z, o[i][q][2]);
                            o[i][q][3] = fmaf(w[i][j], vq[q].w, o[i][q][3]);
                        }
                    }
                }
            }
        }
        __syncwarp();
    }

#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = ty * kPer + i;
        if (r >= n_rows) continue;
        if (slot >= 0) {
            float *base = p.part + slot * part_slot_floats(p.part_rows, d);
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
                if (64 * q + 4 * tx < d)  // past head_dim the sums are zeros
                    reinterpret_cast<float4 *>(base)[(int64_t)(16 * q + tx) * p.part_rows + r] =
                        make_float4(o[i][q][0], o[i][q][1], o[i][q][2], o[i][q][3]);
            if (tx == 0) {
                base[part_stats(p.part_rows, d) + r] = m[i];
                base[part_stats(p.part_rows, d) + p.part_rows + r] = l[i];
            }
        } else {
            const int32_t g = row0 + r;
            const int64_t row = (int64_t)(rq.t0 + g / p.group) * p.q_heads + h * p.group + g % p.group;
            const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 64 * q + 4 * tx + e;
                    if (c < d) put((T *)p.out + row * d + c, o[i][q][e] * inv);
                }
            if (tx == 0 && p.lse)
                p.lse[row] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
        }
    }
}

// Prompts: row block number `want` of all requests, request by request, with every key that its
// rows may see; `*see` is set where cu_q falls in a chunk of 256 requests that is looked at on the
// way.  The CTAs that hold the blocks from such a chunk on all find it, and are so many: the grid has
// a CTA for every block of the requests before the chunk, and one more for each of the others.
// False: there is no such block.
template <typename T, int kRows, int kDMax>
__device__ __forceinline__ bool run_block(const Params &p, int64_t want, StartScratch *scratch, int32_t *see,
                                          float *smem, bool vec_q, bool vec_k) {
    constexpr int kBad = 48;  // a chunk's blocks are fewer than 2^48; above that, its clamped requests
    bool bad = false;
    const int64_t first = want;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        Request r{};
        int64_t n = 0;
        if (b < p.batch) {
            r = load_request<false>(p, b, &bad);
            n = row_blocks(p, r) + ((int64_t)bad << kBad);
        }
        int64_t total = block_sum(n, scratch->red);
        if (total >> kBad) {
            total &= (1ll << kBad) - 1;
            if (threadIdx.x == 0) {
                if (*see == 0) *see = (int32_t)(gridDim.x - (first - want));
                if (p.err) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
            }
        }
        if (want >= total) {
            want -= total;
            continue;
        }
        // walk this chunk: few requests hold most of the blocks
        for (int i = b0; i < min(p.batch, b0 + kThreads); ++i) {
            r = load_request<false>(p, i, &bad);
            n = row_blocks(p, r);
            if (want < n) {
                const int64_t last = min((int64_t)r.t * p.group, (want + 1) * kRows) - 1;
                run_piece<T, T, false, kRows, kDMax>(p, r, i, blockIdx.y, (int32_t)want, 0,
                                                     (int32_t)(last / p.group) + 1, -1, smem, vec_q,
                                                     vec_k, &bad);
                break;
            }
            want -= n;
        }
        return true;
    }
    return false;
}

// CTAs per SM that the registers leave room for.  Prompts of head_dim 64: what shared memory holds
// (600 fp32 prompts of up to 40 tokens 114 us, and 141 with two in place of three).
constexpr int min_ctas(bool paged, int rows, int dmax) { return paged || dmax > 64 ? 1 : rows == 16 ? 4 : 3; }

template <typename T, typename C, bool kPaged, int kRows, int kDMax>
__global__ void __launch_bounds__(kThreads, min_ctas(kPaged, kRows, kDMax))
    simt_kernel(const Params p, bool vec_q, bool vec_k) {
    extern __shared__ __align__(16) float smem[];
    __shared__ StartScratch scratch;
    grid_dep_wait();
    grid_dep_launch();
    bool bad = false, any_bad = false;
    if constexpr (kPaged) {
        const Start s = find_start(p, blockIdx.x, &scratch, &any_bad);
        int64_t u = s.u, before = s.before;  // units before request b
        const int64_t end = s.end;
        Join join{};
        for (int b = s.b; b < p.batch && u < end; ++b) {
            const Request r = load_request<true>(p, b, &bad);
            const int64_t n = request_units(p, r);
            while (u < end && u < before + n) {
                const int32_t tiles = key_tiles(r), worth = tiles + kItemUnits;
                const int64_t item = (u - before) / worth;
                const int32_t o0 = (int32_t)((u - before) % worth);
                const int32_t o1 = (int32_t)min((int64_t)worth, o0 + (end - u));
                const int32_t t0 = max(o0 - kItemUnits, 0), t1 = o1 - kItemUnits;
                const int32_t nrb = row_blocks(p, r);
                const bool whole = t0 == 0 && t1 == tiles;
                if (t1 > t0)
                    run_piece<T, C, true, kRows, kDMax>(
                        p, r, b, (int32_t)(item / nrb), (int32_t)(item % nrb), t0 * kKeyTile,
                        min(t1 * kKeyTile, r.len), whole ? -1 : 2 * (int64_t)blockIdx.x + (t0 == 0),
                        smem, vec_q, vec_k, &any_bad);
                if (t0 == 0 && t1 > 0 && !whole) {
                    const int32_t row0 = (int32_t)(item % nrb) * kRows;
                    join.rows = min(kRows, r.t * p.group - row0);
                    join.last = cta_of(u - o0 + worth - 1, s.units, split_ctas(p, s.units));
                    join.row0 = row0, join.t0 = r.t0, join.h = (int32_t)(item / nrb);
                }
                u += o1 - o0;
            }
            before += n;
        }
        if (threadIdx.x == 0) p.join[blockIdx.x] = join;
    } else {
        // CTA (x, h): a row block, the last blocks (which see the most keys) first.  The grid has
        // a CTA for every one, unless cu_q falls and requests overlap: the CTAs that find this go
        // on.  (What the loop keeps is in shared memory: run_piece has no registers to spare.)
        __shared__ int32_t see;
        __shared__ int64_t want;
        if (threadIdx.x == 0) {
            see = 0;
            want = (int64_t)gridDim.x - 1 - blockIdx.x;
        }
        __syncthreads();
#pragma unroll 1
        while (run_block<T, kRows, kDMax>(p, want, &scratch, &see, smem, vec_q, vec_k)) {
            __syncthreads();
            if (see == 0) break;
            if (threadIdx.x == 0) want += see;
            __syncthreads();
        }
    }
    if (any_bad && p.err) atomicOr(p.err, DFLASH2_DEVERR_ID_RANGE);
}

// Joins the partial rows of items whose tiles span CTAs, in CTA order.  CTA (x, y)
// takes rows 8 y .. of the item that attention CTA x starts and does not end, a
// thread four values of a row (neighbouring threads neighbouring rows, which
// neighbour in a slot): one read of the partials, four at a time.
constexpr int kJoinRows = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_kernel(const Params p) {
    grid_dep_wait();
    const int32_t rr = blockIdx.y * kJoinRows + (threadIdx.x & (kJoinRows - 1));
    const int4 j = __ldcg(reinterpret_cast<const int4 *>(p.join + blockIdx.x));  // rows, last, row0, t0
    const int32_t h = __ldcg(&p.join[blockIdx.x].h);
    if (rr >= j.x) return;
    const int32_t c0 = blockIdx.x, c1 = j.y, row = j.z + rr;
    const int d = p.head_dim, quads = (d + 3) / 4;
    const int64_t slot_floats = part_slot_floats(p.part_rows, d), stats = part_stats(p.part_rows, d);
    const float *first = p.part + (2 * (int64_t)c0 + 1) * slot_floats;  // the item's start
    const float *rest = p.part + 2 * (int64_t)(c0 + 1) * slot_floats;
    const int64_t at = (int64_t)(j.w + row / p.group) * p.q_heads + h * p.group + row % p.group;
    for (int c = threadIdx.x / kJoinRows; c < quads; c += kThreads / kJoinRows) {
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int32_t k = c0; k <= c1; k += 4) {
            float mk[4], lk[4];
            float4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float *part = k + e == c0 ? first : rest + (int64_t)(k + e - c0 - 1) * 2 * slot_floats;
                mk[e] = -INFINITY, lk[e] = 0.0f, v[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (k + e <= c1) {
                    mk[e] = __ldcg(part + stats + rr);
                    lk[e] = __ldcg(part + stats + p.part_rows + rr);
                    v[e] = __ldcg(reinterpret_cast<const float4 *>(part) + (int64_t)c * p.part_rows + rr);
                }
            }
            const float top = fmaxf(m, fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])));
            const float base = top == -INFINITY ? 0.0f : top;
            const float fix = ex2(m - base);
            l *= fix, o.x *= fix, o.y *= fix, o.z *= fix, o.w *= fix;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w = ex2(mk[e] - base);
                l = fmaf(w, lk[e], l);
                if (w != 0.0f) {
                    o.x = fmaf(w, v[e].x, o.x), o.y = fmaf(w, v[e].y, o.y);
                    o.z = fmaf(w, v[e].z, o.z), o.w = fmaf(w, v[e].w, o.w);
                }
            }
            m = top;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T *dst = (T *)p.out + at * d + 4 * c;
        const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * c + e < d) put(dst + e, v[e]);
        if (c == 0 && p.lse)
            p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <typename T, typename C, bool kPaged, int kRows, int kDMax>
dflash2_status launch_one(Params p, int device, bool vec_q, bool vec_k, cudaStream_t st) {
    constexpr int kSmem = simt_smem_floats(kRows, kDMax) * 4;
    auto fn = simt_kernel<T, C, kPaged, kRows, kDMax>;
    static std::atomic<uint64_t> done{0};
    const dflash2_status allowed = allow_smem(fn, kSmem, device, done);
    if (allowed != DFLASH2_OK) return allowed;
    p.row_shift = kRows == 16 ? 4 : 6;
    dim3 grid((unsigned)p.n_cta);
    if (!kPaged)  // every row block of every request, and at most one short one each
        grid = dim3((unsigned)(((int64_t)p.total_q * p.group + kRows - 1) / kRows + p.batch),
                    (unsigned)p.kv_heads);
    launch_k(fn, grid, dim3(kThreads), kSmem, st, p, vec_q, vec_k);
    return launch_status();
}

template <typename T, typename C, bool kPaged>
dflash2_status launch_typed(const Params &p, int device, bool vec_q, bool vec_k, cudaStream_t st) {
    // few rows per (request, head) on average: the 16-row tile
    const bool few = (int64_t)p.total_q * p.group <= 16ll * p.batch;
    if (p.head_dim <= 64)
        return few ? launch_one<T, C, kPaged, 16, 64>(p, device, vec_q, vec_k, st)
                   : launch_one<T, C, kPaged, 64, 64>(p, device, vec_q, vec_k, st);
    if (p.head_dim <= 128)
        return few ? launch_one<T, C, kPaged, 16, 128>(p, device, vec_q, vec_k, st)
                   : launch_one<T, C, kPaged, 64, 128>(p, device, vec_q, vec_k, st);
    return few ? launch_one<T, C, kPaged, 16, 256>(p, device, vec_q, vec_k, st)
               : launch_one<T, C, kPaged, 64, 256>(p, device, vec_q, vec_k, st);
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

dflash2_status launch_simt(const DeviceInfo &di, Params p, bool paged, int32_t dtype,
                           int32_t kv_format, cudaStream_t st) {
    const int el = dtype == DFLASH2_F32 ? 4 : 2;
    const int kel = kv_format == DFLASH2_KV_E4M3 ? 1 : el;
    const bool four = p.head_dim % 4 == 0;
    const bool vec_q = four && aligned_to(p.q, 4 * el) && p.q_stride % 4 == 0;
    const bool vec_k = four && aligned_to(p.k, 4 * kel) && aligned_to(p.v, 4 * kel) &&
                       (paged || (p.k_stride % 4 == 0 && p.v_stride % 4 == 0));
    p.n_cta = di.sm_count;
    for (int i = 0; i < 4; ++i) p.tile_units[i] = 1, p.item_units[i] = kItemUnits;
    p.most_units = 1;
    dflash2_status s;
    if (dtype == DFLASH2_F32) {
        if (!paged)
            s = launch_typed<float, float, false>(p, di.device, vec_q, vec_k, st);
        else if (kv_format == DFLASH2_KV_E4M3)
            s = launch_typed<float, uint8_t, true>(p, di.device, vec_q, vec_k, st);
        else
            s = launch_typed<float, float, true>(p, di.device, vec_q, vec_k, st);
    } else {
        if (!paged)
            s = launch_typed<__nv_bfloat16, __nv_bfloat16, false>(p, di.device, vec_q, vec_k, st);
        else if (kv_format == DFLASH2_KV_E4M3)
            s = launch_typed<__nv_bfloat16, uint8_t, true>(p, di.device, vec_q, vec_k, st);
        else
            s = launch_typed<__nv_bfloat16, __nv_bfloat16, true>(p, di.device, vec_q, vec_k, st);
    }
    if (s != DFLASH2_OK || !paged) return s;
    p.row_shift = (int64_t)p.total_q * p.group <= 16ll * p.batch ? 4 : 6;
    return launch_combine(di, p, dtype, st);
}

dflash2_status launch_combine(const DeviceInfo &, const Params &p, int32_t dtype, cudaStream_t st) {
    if (p.n_cta < 2) return DFLASH2_OK;
    // no row block is longer than its size or than all rows
    const int64_t all = (int64_t)p.total_q * p.group, most = all < (1 << p.row_shift) ? all : 1 << p.row_shift;
    const dim3 grid((unsigned)(p.n_cta - 1), (unsigned)((most + kJoinRows - 1) / kJoinRows));
    if (dtype == DFLASH2_F32)
        launch_k(combine_kernel<float>, grid, dim3(kThreads), 0, st, p);
    else
        launch_k(combine_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, p);
    return launch_status();
}

}  // namespace attn
}  // namespace dflash2
