// ops_abi.hip -- the C entry points of include/ops/moe_ops.h: argument checks
// (before anything is enqueued) and the launches.
#include <math.h>
#include <stdint.h>

#include "ops_internal.h"

namespace {

using moe::hip_fail;

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }
int64_t size_of(int32_t dtype) { return dtype == MOE_DT_BF16 ? 2 : dtype == MOE_DT_F32 ? 4 : 1; }
bool is_float(int32_t dtype) { return dtype == MOE_DT_BF16 || dtype == MOE_DT_F32; }

// 0 -> the row length; a stride below it: MOE_E_SHAPE
int fill_stride(int64_t* stride, int64_t row) {
    if (*stride == 0) *stride = row;
    return *stride < row || *stride > (1ll << 40) ? MOE_E_SHAPE : MOE_OK;
}

int done(hipError_t err, const char* what) { return err == hipSuccess ? MOE_OK : hip_fail(err, what); }

constexpr int64_t kMaxSlots = 1ll << 25;

int check_norm(moe_rmsnorm_args* a) {
    if (a->num_tokens < 0 || a->num_tokens > (1ll << 20)) return MOE_E_SHAPE;
    if (a->hidden < 32 || a->hidden > 16384 || a->hidden % 32) return MOE_E_SHAPE;
    if (a->reserved || !(a->eps >= 0.0) || isinf(a->eps)) return MOE_E_OPTION;
    if (!is_float(a->x_dtype) || !is_float(a->weight_dtype)) return MOE_E_DTYPE;
    if ((a->residual || a->residual_out) && !is_float(a->residual_dtype)) return MOE_E_DTYPE;
    if (fill_stride(&a->x_stride, a->hidden) || fill_stride(&a->residual_stride, a->hidden) ||
        fill_stride(&a->residual_out_stride, a->hidden) || fill_stride(&a->y_stride, a->hidden))
        return MOE_E_SHAPE;
    if (a->num_tokens == 0) return MOE_OK;
    if (!a->x || !a->weight || (!a->y && !a->codes) || !a->codes != !a->scales) return MOE_E_NULL;
    if (a->residual_out && !a->residual) return MOE_E_NULL;
    if (a->residual_out == a->residual && a->residual_out && a->residual_out_stride != a->residual_stride)
        return MOE_E_SHAPE;
    if (a->residual_out == a->x && a->residual_out) {
        if (a->residual_dtype != a->x_dtype) return MOE_E_DTYPE;
        if (a->residual_out_stride != a->x_stride) return MOE_E_SHAPE;
    }
    if (a->y && a->y == a->residual_out) return MOE_E_OPTION;
    if (a->y && a->y == a->x) {
        if (a->x_dtype != MOE_DT_BF16) return MOE_E_DTYPE;
        if (a->y_stride != a->x_stride) return MOE_E_SHAPE;
    }
    if (misaligned(a->x, 16) || misaligned(a->residual, 16) || misaligned(a->residual_out, 16) ||
        misaligned(a->weight, 16) || misaligned(a->y, 16) || misaligned(a->codes, 16) || misaligned(a->scales, 4))
        return MOE_E_ALIGN;
    const int64_t rs = size_of(a->residual_dtype);
    if (a->x_stride * size_of(a->x_dtype) % 16 || (a->residual && a->residual_stride * rs % 16) ||
        (a->residual_out && a->residual_out_stride * rs % 16) || (a->y && a->y_stride * 2 % 16))
        return MOE_E_ALIGN;
    return MOE_OK;
}

int check_linear_sizes(int64_t T, int64_t rows, int64_t inner, int32_t activation) {
    if (T < 0 || T > (1ll << 20)) return MOE_E_SHAPE;
    if (rows < 64 || rows > (1ll << 20) || rows % 64) return MOE_E_SHAPE;
    if (inner < 128 || inner > 65536 || inner % 128) return MOE_E_SHAPE;
    if (activation < MOE_EPI_NONE || activation > MOE_EPI_SILU_MUL) return MOE_E_OPTION;
    return MOE_OK;
}

int check_linear(moe_mxfp8_linear_args* a) {
    const int rc = check_linear_sizes(a->num_tokens, a->rows, a->inner, a->activation);
    if (rc != MOE_OK) return rc;
    if (a->reserved) return MOE_E_OPTION;
    const int64_t cols = a->activation == MOE_EPI_SILU_MUL ? a->rows / 2 : a->rows;
    if (fill_stride(&a->residual_stride, cols) || fill_stride(&a->out_stride, cols)) return MOE_E_SHAPE;
    if (a->num_tokens == 0) return MOE_OK;
    if (!a->x_codes || !a->x_scales || !a->w_tiles || !a->w_scales) return MOE_E_NULL;
    if (!a->out_codes != !a->out_scales) return MOE_E_NULL;
    if (!a->out == !a->out_codes) return MOE_E_OPTION;
    if (a->out && a->residual == a->out && a->residual_stride != a->out_stride) return MOE_E_SHAPE;
    if (misaligned(a->x_codes, 16) || misaligned(a->x_scales, 4) || misaligned(a->w_tiles, 16) ||
        misaligned(a->w_scales, 16) || misaligned(a->bias, 16) || misaligned(a->residual, 16) ||
        misaligned(a->out, 16) || misaligned(a->out_codes, 16) || misaligned(a->out_scales, 4) ||
        misaligned(a->workspace, 16))
        return MOE_E_ALIGN;
    if ((a->residual && a->residual_stride % 8) || (a->out && a->out_stride % 8)) return MOE_E_ALIGN;
    const int64_t need = moe::mxfp8_linear_workspace(a->num_tokens, a->rows, a->inner, a->activation);
    if (need > 0 && !a->workspace) return MOE_E_NULL;
    if (need > a->workspace_bytes && need > 0) return MOE_E_LIMIT;
    return MOE_OK;
}

int check_dispatch_sizes(int64_t T, int64_t E, int32_t k) {
    if (T < 0 || T > kMaxSlots || E < 1 || E > moe::kMaxExperts) return MOE_E_SHAPE;
    if (k < 1 || k > moe::kMaxTopK) return MOE_E_TOPK;
    return T * k > kMaxSlots ? MOE_E_SHAPE : MOE_OK;
}

int check_dispatch(moe_dispatch_args* a) {
    const int rc = check_dispatch_sizes(a->num_tokens, a->num_experts, a->top_k);
    if (rc != MOE_OK) return rc;
    if (!a->offsets) return MOE_E_NULL;
    if (misaligned(a->offsets, 4) || misaligned(a->counts, 4)) return MOE_E_ALIGN;
    if (a->num_tokens == 0) return MOE_OK;
    if (!a->ids || !a->pos || !a->x != !a->rows) return MOE_E_NULL;
    if (misaligned(a->ids, 4) || misaligned(a->pos, 4) || misaligned(a->sorted, 4) || misaligned(a->workspace, 4))
        return MOE_E_ALIGN;
    if (a->x) {
        if (!is_float(a->dtype) && a->dtype != MOE_DT_U8) return MOE_E_DTYPE;
        if (a->hidden < 1 || a->hidden > 65536 || (a->dtype == MOE_DT_U8 && a->hidden % 32)) return MOE_E_SHAPE;
        if (fill_stride(&a->x_stride, a->hidden)) return MOE_E_SHAPE;
        const bool mx = a->dtype == MOE_DT_U8;
        if (mx != !!a->x_scales || mx != !!a->row_scales) return MOE_E_NULL;
        const uintptr_t es = (uintptr_t)size_of(a->dtype);
        if (misaligned(a->x, es) || misaligned(a->rows, es)) return MOE_E_ALIGN;
    } else {
        a->x_scales = nullptr;
        a->row_scales = nullptr;
        a->hidden = 0;
    }
    const int64_t need = moe::dispatch_workspace(a->num_tokens, a->num_experts, a->top_k);
    if (need > 0 && !a->workspace) return MOE_E_NULL;
    if (need > 0 && need > a->workspace_bytes) return MOE_E_LIMIT;
    return MOE_OK;
}

// of: 0 combine, 1 backward
int check_combine(moe_combine_args* a, bool backward) {
    if (a->reserved) return MOE_E_OPTION;
    if (a->num_tokens < 0 || a->num_tokens > kMaxSlots || a->num_rows < 0 || a->num_rows > kMaxSlots)
        return MOE_E_SHAPE;
    if (a->hidden < 1 || a->hidden > 65536) return MOE_E_SHAPE;
    if (a->top_k < 1 || a->top_k > moe::kMaxTopK) return MOE_E_TOPK;
    if (a->num_tokens * a->top_k > kMaxSlots) return MOE_E_SHAPE;
    if (!is_float(a->rows_dtype) || !is_float(a->out_dtype)) return MOE_E_DTYPE;
    if (fill_stride(&a->rows_stride, a->hidden) || fill_stride(&a->out_stride, a->hidden) ||
        fill_stride(&a->dout_stride, a->hidden) || fill_stride(&a->drows_stride, a->hidden))
        return MOE_E_SHAPE;
    if (a->num_tokens == 0) return MOE_OK;
    const uintptr_t rs = (uintptr_t)size_of(a->rows_dtype), os = (uintptr_t)size_of(a->out_dtype);
    if (!a->pos) return MOE_E_NULL;
    if (!backward) {
        if (!a->out || (!a->rows && a->num_rows > 0)) return MOE_E_NULL;
    } else {
        // without rows an empty drows may well be null
        if (!a->dout || (!a->drows && !a->dweights && a->num_rows > 0)) return MOE_E_NULL;
        if (a->dweights && !a->rows && a->num_rows > 0) return MOE_E_NULL;
        if (a->drows && a->drows == a->rows && a->drows_stride != a->rows_stride) return MOE_E_SHAPE;
    }
    if (misaligned(a->pos, 4) || misaligned(a->weights, 4) || misaligned(a->dweights, 4) || misaligned(a->rows, rs) ||
        misaligned(a->out, os) || misaligned(a->dout, os) || misaligned(a->drows, rs))
        return MOE_E_ALIGN;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_rmsnorm(const moe_rmsnorm_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_rmsnorm_args a = *args;
    const int rc = check_norm(&a);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_rmsnorm(a, (hipStream_t)stream), "rmsnorm");
}

int64_t moe_mxfp8_linear_workspace(int64_t num_tokens, int64_t rows, int64_t inner, int32_t activation) {
    const int rc = check_linear_sizes(num_tokens, rows, inner, activation);
    return rc != MOE_OK ? rc : moe::mxfp8_linear_workspace(num_tokens, rows, inner, activation);
}

int moe_mxfp8_linear(const moe_mxfp8_linear_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_mxfp8_linear_args a = *args;
    const int rc = check_linear(&a);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_mxfp8_linear(a, (hipStream_t)stream), "linear");
}

int64_t moe_dispatch_workspace(int64_t num_tokens, int64_t num_experts, int32_t top_k) {
    const int rc = check_dispatch_sizes(num_tokens, num_experts, top_k);
    return rc != MOE_OK ? rc : moe::dispatch_workspace(num_tokens, num_experts, top_k);
}

int moe_dispatch(const moe_dispatch_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_dispatch_args a = *args;
    const int rc = check_dispatch(&a);
    if (rc != MOE_OK) return rc;
    return done(moe::launch_dispatch(a, (hipStream_t)stream), "dispatch");
}

int moe_combine(const moe_combine_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_combine_args a = *args;
    const int rc = check_combine(&a, false);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_ops_combine(a, (hipStream_t)stream), "combine");
}

int moe_dispatch_backward(const moe_combine_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    if (args->weights) return MOE_E_OPTION;
    return moe_combine(args, stream);
}

int moe_combine_backward(const moe_combine_args* args, void* stream) {
    if (!args) return MOE_E_NULL;
    moe_combine_args a = *args;
    const int rc = check_combine(&a, true);
    if (rc != MOE_OK || a.num_tokens == 0) return rc;
    return done(moe::launch_ops_combine_backward(a, (hipStream_t)stream), "combine backward");
}

}  // extern "C"
