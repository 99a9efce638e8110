// attention_abi.hip -- the C entry points of include/ops/moe_attention.h:
// argument checks (before anything is enqueued) and the launches.
#include <math.h>
#include <stdint.h>

#include "attention_internal.h"

namespace {

using moe::hip_fail;

constexpr int64_t kMaxStride = 1ll << 40, kMaxPageStride = 1ll << 31, kMaxTokenStride = 1ll << 31, kMaxTokens = 1ll << 20, kMaxSeqs = 1ll << 16;
constexpr int64_t kMaxPositions = 1ll << 30, kMaxUnits = 1ll << 30;
constexpr int kMaxHeads = 1024, kMaxMaskWords = 64;

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int fill_stride(int64_t* stride, int64_t row) {  // 0: the row's length
    if (*stride == 0) *stride = row;
    return *stride < row || *stride > kMaxStride ? MOE_E_SHAPE : MOE_OK;
}

int done(hipError_t err, const char* what) { return err == hipSuccess ? MOE_OK : hip_fail(err, what); }

int check_cache_sizes(moe_kv_cache* c) {
    if (c->reserved) return MOE_E_OPTION;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX) return MOE_E_SHAPE;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return MOE_E_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads) return MOE_E_SHAPE;
    if (c->head_dim < 32 || c->head_dim > 512 || c->head_dim % 32) return MOE_E_SHAPE;
    const int64_t page = (int64_t)c->kv_heads * c->page_size * c->head_dim;
    if (fill_stride(&c->codes_page_stride, page) || fill_stride(&c->scales_page_stride, page / 32)) return MOE_E_SHAPE;
    return c->codes_page_stride > kMaxPageStride || c->scales_page_stride > kMaxPageStride ? MOE_E_SHAPE : MOE_OK;
}

int check_cache_memory(const moe_kv_cache& c) {
    if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return MOE_E_NULL;
    if (misaligned(c.k_codes, 16) || misaligned(c.k_scales, 16) || misaligned(c.v_codes, 16) ||
        misaligned(c.v_scales, 16) || c.codes_page_stride % 16 || c.scales_page_stride % 16)
        return MOE_E_ALIGN;
    return MOE_OK;
}

int check_rows(moe_kv_rows_args* a) {
    if (a->num_tokens < 0 || a->num_tokens > kMaxTokens) return MOE_E_SHAPE;
    int rc = check_cache_sizes(&a->cache);
    if (rc != MOE_OK) return rc;
    if (a->reserved) return MOE_E_OPTION;
    if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F32) return MOE_E_DTYPE;
    const int64_t row = (int64_t)a->cache.kv_heads * a->cache.head_dim, size = a->dtype == MOE_DT_BF16 ? 2 : 4;
    if (fill_stride(&a->k_stride, row) || fill_stride(&a->v_stride, row)) return MOE_E_SHAPE;
    if (a->num_tokens == 0) return MOE_OK;
    if (!a->k || !a->v || !a->slots) return MOE_E_NULL;
    if ((rc = check_cache_memory(a->cache)) != MOE_OK) return rc;
    if (misaligned(a->k, 16) || misaligned(a->v, 16) || misaligned(a->slots, 8) || a->k_stride * size % 16 ||
        a->v_stride * size % 16)
        return MOE_E_ALIGN;
    return MOE_OK;
}

int check_attention_sizes(int64_t T, int64_t B, int32_t heads, int32_t kv_heads, int32_t D) {
    if (T < 0 || T > kMaxTokens || B < 0 || B > kMaxSeqs) return MOE_E_SHAPE;
    if (kv_heads < 1 || kv_heads > kMaxHeads || heads < 1 || heads > kMaxHeads || heads % kv_heads) return MOE_E_SHAPE;
    return D == 64 || D == 128 || D == 256 ? MOE_OK : MOE_E_SHAPE;
}

int check_attention(moe_tree_attention_args* a) {
    int rc = check_cache_sizes(&a->cache);
    if (rc != MOE_OK) return rc;
    const int64_t T = a->num_tokens, B = a->num_seqs;
    if ((rc = check_attention_sizes(T, B, a->num_heads, a->cache.kv_heads, a->cache.head_dim)) != MOE_OK) return rc;
    // what a score is multiplied by, in powers of two, is a normal number too
    if (!(a->scale > 0.f) || !isnormal(a->scale) || !isnormal(a->scale * 1.4426950408889634f)) return MOE_E_OPTION;
    if (a->mask_words < 0 || a->mask_words > kMaxMaskWords) return MOE_E_SHAPE;
    const int64_t row = (int64_t)a->num_heads * a->cache.head_dim;
    if (fill_stride(&a->q_stride, row) || fill_stride(&a->out_stride, row)) return MOE_E_SHAPE;
    if (a->q_stride > kMaxTokenStride || a->out_stride > kMaxTokenStride) return MOE_E_SHAPE;
    if (T == 0 || B == 0) return MOE_OK;
    if ((a->mask != nullptr) != (a->mask_words != 0)) return MOE_E_SHAPE;  // (an empty mask has no address)
    if (a->max_pages < 1 || a->max_pages > kMaxPositions / a->cache.page_size) return MOE_E_SHAPE;
    if (fill_stride(&a->block_table_stride, a->max_pages)) return MOE_E_SHAPE;
    if (!a->q || !a->out || !a->block_table || !a->context_lens || !a->token_offsets) return MOE_E_NULL;
    if ((rc = check_cache_memory(a->cache)) != MOE_OK) return rc;
    if (misaligned(a->q, 16) || misaligned(a->out, 16) || misaligned(a->block_table, 4) ||
        misaligned(a->context_lens, 4) || misaligned(a->token_offsets, 4) || misaligned(a->mask, 8) ||
        misaligned(a->workspace, 16) || a->q_stride % 8 || a->out_stride % 8)
        return MOE_E_ALIGN;
    const moe::AttentionPlan plan = moe::attention_plan(T, B, a->num_heads, a->cache.kv_heads, a->cache.head_dim);
    if (moe::attention_most_units(T, B, a->num_heads, a->cache.kv_heads, plan.rows,
                                  a->max_pages * a->cache.page_size) > kMaxUnits)
        return MOE_E_LIMIT;
    if (!a->workspace) return MOE_E_NULL;
    return plan.bytes > a->workspace_bytes ? MOE_E_LIMIT : MOE_OK;
}

}  // namespace

extern "C" {

int moe_kv_write(const moe_kv_rows_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_kv_rows_args a = *args;
    const int rc = check_rows(&a);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_kv_write(a, (hipStream_t)stream), "kv write");
}

int moe_kv_read(const moe_kv_rows_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_kv_rows_args a = *args;
    const int rc = check_rows(&a);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_kv_read(a, (hipStream_t)stream), "kv read");
}

int64_t moe_tree_attention_workspace(int64_t num_tokens, int64_t num_seqs, int32_t num_heads, int32_t kv_heads,
                                     int32_t head_dim) {
    const int rc = check_attention_sizes(num_tokens, num_seqs, num_heads, kv_heads, head_dim);
    return rc != MOE_OK ? rc : moe::attention_plan(num_tokens, num_seqs, num_heads, kv_heads, head_dim).bytes;
}

int moe_tree_attention(const moe_tree_attention_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_tree_attention_args a = *args;
    const int rc = check_attention(&a);
    if (rc != MOE_OK || a.num_tokens == 0 || a.num_seqs == 0) return rc;
    return done(moe::launch_tree_attention(a, (hipStream_t)stream), "tree attention");
}

}  // extern "C"
