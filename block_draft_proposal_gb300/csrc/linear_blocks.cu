// Matrix product of E4M3 codes with a scale per block of 128:
//
//   y[m, n] = sum_b xs[m, b] * ws[n / 128, b] * sum_{k in b} dec(xq[m, k]) * dec(wq[n, k])
//
// the products of a block in fp32, scaled and added in fp32.
#include "rows.cuh"

namespace dflash2 {
namespace {

struct LinearArgs {
    const uint8_t *xq, *wq;
    const float *xs, *ws;
    int32_t rows, n_in, n_out, blocks;  // blocks of 128 along n_in
    void *y;
    int32_t *err;
};

constexpr int kTile = 64, kStep = 32;

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 each, on CUDA cores.
template <typename T>
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearArgs a) {
    __shared__ float xt[kStep][kTile + 1], wt[kStep][kTile + 1];
    grid_dep_wait();
    const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float y[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < a.n_in; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int r = i / kStep, k = i % kStep;
            const bool in = k0 + k < a.n_in;
            xt[k][r] = in && m0 + r < a.rows ? decode1(a.xq[(m0 + r) * a.n_in + k0 + k]) : 0.0f;
            wt[k][r] = in && n0 + r < a.n_out ? decode1(a.wq[(n0 + r) * a.n_in + k0 + k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) part[i][j] += xt[k][ty + 16 * i] * wt[k][tx + 16 * j];
        __syncthreads();
        if ((k0 + kStep) % 128 == 0 || k0 + kStep >= a.n_in) {
            const int b = k0 / 128;
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                    if (m < a.rows && n < a.n_out)
                        y[i][j] += part[i][j] * (a.xs[m * a.blocks + b] * a.ws[n / 128 * a.blocks + b]);
                    part[i][j] = 0.0f;
                }
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < a.rows && n < a.n_out) from_f32((T *)a.y + m * a.n_out + n, y[i][j]);
        }
}

template <typename T> dflash2_status launch_linear(const LinearArgs &a, cudaStream_t st) {
    launch_k(linear_simple_kernel<T>, dim3((a.n_out + kTile - 1) / kTile, (a.rows + kTile - 1) / kTile), dim3(256), 0,
             st, a);
    return launch_status();
}

bool shape_ok(int64_t rows, int32_t n_in, int32_t n_out) {
    return rows >= 0 && rows <= 1 << 20 && n_in >= 1 && n_in <= 1 << 20 && n_out >= 1 && n_out <= 1 << 24 &&
           rows * n_in < 1ll << 40 && (int64_t)n_out * n_in < 1ll << 40;
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
    if (!x_q) {
        uint8_t *q = static_cast<uint8_t *>(workspace);
        float *scale = reinterpret_cast<float *>(q + codes_bytes(rows, in_features));
        st = launch_quant_blocks_e4m3(x, x_row_stride, x_dtype, rows, in_features, q, scale, s);
        if (st != DFLASH2_OK) return st;
        x_q = q, x_scale = scale;
    }
    LinearArgs a{};
    a.xq = x_q, a.wq = w_q, a.xs = x_scale, a.ws = w_scale;
    a.rows = (int32_t)rows, a.n_in = in_features, a.n_out = out_features, a.blocks = (in_features + 127) / 128;
    a.y = out, a.err = err_word;
    return out_dtype == DFLASH2_F32 ? launch_linear<float>(a, s) : launch_linear<__nv_bfloat16>(a, s);
}
