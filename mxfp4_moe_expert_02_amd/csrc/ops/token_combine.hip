// token_combine.hip -- the experts' rows back in token order, weighted, and
// the gradients of that sum.
//
//   out[t, :] = sum_j w[t, j] * rows[pos[t, j], :]          (combine)
//   dx[t, :]  = sum_j drows[pos[t, j], :]                   (w absent)
//
// One thread owns a piece of 8 (4 for float32 alone) consecutive columns of
// one token: it loads the piece of each of the token's k rows (batches of
// eight, all in flight before the first is used) and adds them in slot
// order in float32.  Threads are numbered over (token, piece), so short rows
// fill their workgroups.  Bound by the rows' bytes, read once: 288 tokens of
// 8 x 7168 bf16 7.9 us, 4.7 TB/s; 1001 of 2 x 7168 float32 13.4 us, 6.4 TB/s
// where the caches still hold part of them.
//
// The backward gives one wave to a slot: it reads the slot's row and its
// token's dout in pieces, writes w * dout, and sums their product; the
// cross-lane sum at the end is the weight's gradient.  A slot's gradient
// needs no other wave, so there are no atomics and no second pass.  4096 x 8
// rows of 7168 bf16: 203 us, 5.2 TB/s over one read and one write of the rows
// (a copy moves 5.0 to 5.5).
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 22;  // beyond it a thread takes several pieces
constexpr int kBatch = 8;  // rows in flight per thread

// N slots [j0, j0 + N) of a token added to v in slot order
template <typename R, int P, int N>
__device__ inline void add_slots(const moe_combine_args& a, int64_t slot0, int col, float (&v)[P]) {
    int p[N];
    float w[N];
#pragma unroll
    for (int u = 0; u < N; u++) {
        p[u] = a.pos[slot0 + u];
        w[u] = a.weights ? a.weights[slot0 + u] : 1.f;
    }
    float y[N][P];
#pragma unroll
    for (int u = 0; u < N; u++) {
#pragma unroll
        for (int i = 0; i < P; i++) y[u][i] = 0.f;
        if (p[u] >= 0 && p[u] < a.num_rows)
            load_piece<P>((const R*)a.rows + (int64_t)p[u] * a.rows_stride + col, y[u]);
        else
            w[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < N; u++)
#pragma unroll
        for (int i = 0; i < P; i++) v[i] = fmaf(w[u], y[u][i], v[i]);
}

template <typename R, typename O, int P>
__global__ void __launch_bounds__(kThreads) token_combine_kernel(moe_combine_args a, int pieces) {
    const int64_t total = a.num_tokens * pieces;
    for (int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * kThreads) {
        const int64_t t = idx / pieces;
        const int col = (int)(idx - t * pieces) * P;
        const int64_t base = t * a.top_k;
        float v[P];
#pragma unroll
        for (int i = 0; i < P; i++) v[i] = 0.f;
        int j = 0;
        for (; j + kBatch <= a.top_k; j += kBatch) add_slots<R, P, kBatch>(a, base + j, col, v);
        if (a.top_k - j >= 4) add_slots<R, P, 4>(a, base + j, col, v), j += 4;
        if (a.top_k - j >= 2) add_slots<R, P, 2>(a, base + j, col, v), j += 2;
        if (a.top_k - j >= 1) add_slots<R, P, 1>(a, base + j, col, v);
        store_piece<P>((O*)a.out + t * a.out_stride + col, v);
    }
}

template <typename R, typename O, int P>
__global__ void __launch_bounds__(kThreads) token_combine_backward_kernel(moe_combine_args a) {
    const int64_t slot = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
    if (slot >= a.num_tokens * a.top_k) return;
    const int lane = threadIdx.x % kWave;
    const int64_t t = slot / a.top_k;
    const int p = a.pos[slot];
    if (p < 0 || p >= a.num_rows) {
        if (a.dweights && lane == 0) a.dweights[slot] = 0.f;
        return;
    }
    const float w = a.weights ? a.weights[slot] : 1.f;
    const O* g = (const O*)a.dout + t * a.dout_stride;
    const R* y = (const R*)a.rows + (int64_t)p * a.rows_stride;
    R* d = a.drows ? (R*)a.drows + (int64_t)p * a.drows_stride : nullptr;
    const int pieces = (int)a.hidden / P;
    float dot = 0.f;
    // two pieces of each row in flight (drows may be rows: every lane stores
    // where it has loaded, and only after it)
    for (int i = lane; i < pieces; i += 2 * kWave) {
        const int i2 = i + kWave;
        const bool two = i2 < pieces;
        float gv[2][P], yv[2][P];
        load_piece<P>(g + i * P, gv[0]);
        if (two) load_piece<P>(g + i2 * P, gv[1]);
        if (a.dweights) {
            load_piece<P>(y + i * P, yv[0]);
            if (two) load_piece<P>(y + i2 * P, yv[1]);
#pragma unroll
            for (int e = 0; e < P; e++) dot = fmaf(gv[0][e], yv[0][e], dot);
            if (two)
#pragma unroll
                for (int e = 0; e < P; e++) dot = fmaf(gv[1][e], yv[1][e], dot);
        }
        if (d) {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                if (u == 1 && !two) break;
                float o[P];
#pragma unroll
                for (int e = 0; e < P; e++) o[e] = w * gv[u][e];
                store_piece<P>(d + (u ? i2 : i) * P, o);
            }
        }
    }
    if (!a.dweights) return;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) dot += __shfl_xor(dot, m);
    if (lane == 0) a.dweights[slot] = dot;
}

bool whole_pieces(const void* p, int64_t stride, int64_t esize, int64_t hidden, int piece) {
    return !p || (((uintptr_t)p & 15u) == 0 && stride * esize % 16 == 0 && hidden % piece == 0);
}

template <typename R, typename O>
hipError_t combine_typed(const moe_combine_args& a, hipStream_t stream) {
    constexpr int P = sizeof(R) == 4 && sizeof(O) == 4 ? 4 : 8;
    const bool whole = whole_pieces(a.rows, a.rows_stride, sizeof(R), a.hidden, P) &&
                       whole_pieces(a.out, a.out_stride, sizeof(O), a.hidden, P);
    const int pieces = (int)(whole ? a.hidden / P : a.hidden);
    const int64_t blocks = (a.num_tokens * pieces + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
    if (whole) token_combine_kernel<R, O, P><<<grid, kThreads, 0, stream>>>(a, pieces);
    else token_combine_kernel<R, O, 1><<<grid, kThreads, 0, stream>>>(a, pieces);
    return hipGetLastError();
}

template <typename R, typename O>
hipError_t backward_typed(const moe_combine_args& a, hipStream_t stream) {
    constexpr int P = sizeof(R) == 4 && sizeof(O) == 4 ? 4 : 8;
    const bool whole = whole_pieces(a.dweights ? a.rows : nullptr, a.rows_stride, sizeof(R), a.hidden, P) &&
                       whole_pieces(a.dout, a.dout_stride, sizeof(O), a.hidden, P) &&
                       whole_pieces(a.drows, a.drows_stride, sizeof(R), a.hidden, P);
    const int64_t slots = a.num_tokens * a.top_k;
    const unsigned grid = (unsigned)((slots + kThreads / kWave - 1) / (kThreads / kWave));
    if (whole) token_combine_backward_kernel<R, O, P><<<grid, kThreads, 0, stream>>>(a);
    else token_combine_backward_kernel<R, O, 1><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ops_combine(const moe_combine_args& a, hipStream_t stream) {
    const bool rb = a.rows_dtype == MOE_DT_BF16, ob = a.out_dtype == MOE_DT_BF16;
    if (rb) return ob ? combine_typed<uint16_t, uint16_t>(a, stream) : combine_typed<uint16_t, float>(a, stream);
    return ob ? combine_typed<float, uint16_t>(a, stream) : combine_typed<float, float>(a, stream);
}

hipError_t launch_ops_combine_backward(const moe_combine_args& a, hipStream_t stream) {
    const bool rb = a.rows_dtype == MOE_DT_BF16, ob = a.out_dtype == MOE_DT_BF16;
    if (rb) return ob ? backward_typed<uint16_t, uint16_t>(a, stream) : backward_typed<uint16_t, float>(a, stream);
    return ob ? backward_typed<float, uint16_t>(a, stream) : backward_typed<float, float>(a, stream);
}

}  // namespace moe
