// Entry points of the attention over the paged cache and over packed prompts:
// host checks, then the kernel that takes the call.
#include <math.h>

#include "attention.cuh"

using namespace dflash2;

namespace {

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs the workspace has slots for, one per SM (152 on GB300); or twice as many with
// slots of half of the rows (attention_few.cu), 64 of them.
constexpr int kWorkspaceCtas = 160;

// Rows of a partial slot: no row block is longer than 256 rows or than all rows.
int32_t slot_rows(int32_t total_q, int32_t group) {
    const int64_t rows = ((int64_t)total_q * group + 15) / 16 * 16;
    return (int32_t)(rows < 128 ? 128 : rows > 256 ? 256 : rows);
}

dflash2_status check_shape(int32_t batch, int32_t total_q, int32_t q_heads, int32_t kv_heads,
                           int32_t head_dim, float scale, int32_t dtype) {
    if (dtype != DFLASH2_F32 && dtype != DFLASH2_BF16) return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (batch < 0 || batch > attn::kMaxBatch || total_q < 0 || kv_heads < 1 || kv_heads > 65535 ||
        q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > attn::kMaxGroup ||
        head_dim < 1 || head_dim > 256 || (int64_t)total_q * q_heads >= (1ll << 31) ||
        !isfinite(scale * 1.4426950408889634f))
        return DFLASH2_ERR_INVALID_ARG;
    return DFLASH2_OK;
}

}  // namespace

extern "C" size_t dflash2_tree_attention_workspace_size(int32_t total_q, int32_t batch,
                                                        int32_t q_heads, int32_t kv_heads,
                                                        int32_t head_dim) {
    if (check_shape(batch, total_q, q_heads, kv_heads, head_dim, 1.0f, DFLASH2_BF16) != DFLASH2_OK)
        return 0;
    return sizeof(attn::Join) * 2 * kWorkspaceCtas +
           (size_t)(2 * kWorkspaceCtas *
                    attn::part_slot_floats(slot_rows(total_q, q_heads / kv_heads), head_dim)) * 4;
}

extern "C" dflash2_status dflash2_tree_attention(
    const void *q, int64_t q_row_stride, const void *k_cache, const void *v_cache,
    const uint8_t *k_exp, const uint8_t *v_exp, const int32_t *page_table, int32_t max_pages,
    int64_t num_pages, int32_t page_size, const int32_t *cu_q, const int32_t *kv_lens,
    const int64_t *tree_mask, int32_t mask_words, int32_t batch, int32_t total_q, int32_t q_heads,
    int32_t kv_heads, int32_t head_dim, float scale, int32_t dtype, int32_t kv_format, void *out,
    float *lse, void *workspace, size_t ws_bytes, int32_t *err_word, void *stream) {
    dflash2_status st = check_shape(batch, total_q, q_heads, kv_heads, head_dim, scale, dtype);
    if (st != DFLASH2_OK) return st;
    if (kv_format != DFLASH2_KV_NATIVE && kv_format != DFLASH2_KV_E4M3)
        return DFLASH2_ERR_UNSUPPORTED_DTYPE;
    if (page_size < 1 || max_pages < 1 || num_pages < 1 ||
        (int64_t)max_pages * page_size > attn::kMaxKeys || num_pages >= (1ll << 31) / kv_heads ||
        q_row_stride < (int64_t)q_heads * head_dim || (tree_mask && (mask_words < 1 || mask_words > (1 << 20))))
        return DFLASH2_ERR_INVALID_ARG;
    if (total_q == 0 || batch == 0) return DFLASH2_OK;
    const bool q8 = kv_format == DFLASH2_KV_E4M3;
    if (!q || !k_cache || !v_cache || (q8 && (!k_exp || !v_exp)) || !page_table || !cu_q ||
        !kv_lens || !out)
        return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == DFLASH2_F32 ? 4 : 2, kel = q8 ? 1 : el;
    if (!aligned_to(q, el) || !aligned_to(k_cache, kel) || !aligned_to(v_cache, kel) ||
        !aligned_to(page_table, 4) || !aligned_to(cu_q, 4) || !aligned_to(kv_lens, 4) ||
        !aligned_to(tree_mask, 8) || !aligned_to(out, el) || !aligned_to(lse, 4) ||
        !aligned_to(err_word, 4))
        return DFLASH2_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        ws_bytes < dflash2_tree_attention_workspace_size(total_q, batch, q_heads, kv_heads, head_dim))
        return DFLASH2_ERR_WORKSPACE;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    if (di.sm_count > kWorkspaceCtas) di.sm_count = kWorkspaceCtas;
    attn::Params p{};
    p.q = q, p.q_stride = q_row_stride, p.k = k_cache, p.v = v_cache, p.k_exp = k_exp;
    p.v_exp = v_exp, p.page_table = page_table, p.max_pages = max_pages, p.page_size = page_size;
    p.num_pages = num_pages, p.cu_q = cu_q, p.kv_lens = kv_lens, p.tree_mask = tree_mask;
    p.mask_words = mask_words, p.batch = batch, p.total_q = total_q, p.q_heads = q_heads;
    p.kv_heads = kv_heads, p.group = q_heads / kv_heads, p.head_dim = head_dim;
    p.scale_log2 = scale * 1.4426950408889634f, p.out = out, p.lse = lse;
    p.join = static_cast<attn::Join *>(workspace);
    p.part = reinterpret_cast<float *>(p.join + 2 * kWorkspaceCtas), p.part_rows = slot_rows(total_q, p.group), p.err = err_word;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (attn::tc_takes(p, true, dtype)) return attn::launch_tc(di, p, true, kv_format, s);
    return attn::launch_simt(di, p, true, dtype, kv_format, s);
}

extern "C" size_t dflash2_prompt_attention_workspace_size(int32_t total_q, int32_t batch,
                                                          int32_t q_heads, int32_t kv_heads,
                                                          int32_t head_dim) {
    if (check_shape(batch, total_q, q_heads, kv_heads, head_dim, 1.0f, DFLASH2_BF16) != DFLASH2_OK)
        return 0;
    return 16;
}

extern "C" dflash2_status dflash2_prompt_attention(
    const void *q, const void *k, const void *v, int64_t q_row_stride, int64_t k_row_stride,
    int64_t v_row_stride, const int32_t *cu_q, int32_t batch, int32_t total_q, int32_t q_heads,
    int32_t kv_heads, int32_t head_dim, float scale, int32_t dtype, void *out, float *lse,
    void *workspace, size_t ws_bytes, int32_t *err_word, void *stream) {
    dflash2_status st = check_shape(batch, total_q, q_heads, kv_heads, head_dim, scale, dtype);
    if (st != DFLASH2_OK) return st;
    if (q_row_stride < (int64_t)q_heads * head_dim || k_row_stride < (int64_t)kv_heads * head_dim ||
        v_row_stride < (int64_t)kv_heads * head_dim)
        return DFLASH2_ERR_INVALID_ARG;
    if (total_q == 0 || batch == 0) return DFLASH2_OK;
    if (!q || !k || !v || !cu_q || !out) return DFLASH2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == DFLASH2_F32 ? 4 : 2;
    if (!aligned_to(q, el) || !aligned_to(k, el) || !aligned_to(v, el) || !aligned_to(cu_q, 4) ||
        !aligned_to(out, el) || !aligned_to(lse, 4) || !aligned_to(err_word, 4))
        return DFLASH2_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        ws_bytes < dflash2_prompt_attention_workspace_size(total_q, batch, q_heads, kv_heads, head_dim))
        return DFLASH2_ERR_WORKSPACE;
    DeviceInfo di;
    st = current_device(&di);
    if (st != DFLASH2_OK) return st;
    attn::Params p{};
    p.q = q, p.q_stride = q_row_stride, p.k = k, p.k_stride = k_row_stride, p.v = v;
    p.v_stride = v_row_stride, p.cu_q = cu_q, p.batch = batch, p.total_q = total_q;
    p.q_heads = q_heads, p.kv_heads = kv_heads, p.group = q_heads / kv_heads, p.head_dim = head_dim;
    p.scale_log2 = scale * 1.4426950408889634f, p.out = out, p.lse = lse, p.err = err_word;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (attn::tc_takes(p, false, dtype))
        return attn::launch_tc(di, p, false, DFLASH2_KV_NATIVE, s);
    return attn::launch_simt(di, p, false, dtype, DFLASH2_KV_NATIVE, s);
}
