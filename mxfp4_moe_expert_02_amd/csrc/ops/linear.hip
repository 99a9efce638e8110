// linear.hip -- out = act(x W^T + bias) + residual with x and W in MXFP8.
//
// The weights come in the MXFP8 tile layout of moe_mxfp8_prepack (prepack.hip):
// per 64-row quad and 128-k chunk 8 KB of codes [group][half][lane][16] and
// 256 scale bytes [lane][group], lane (r, g) = (l % 16, l / 16) holding block
// g (k = 32g .. 32g+31) of row r.  D of a 16x16 product: lane (c, g) holds
// rows 4g .. 4g+3 of token c.
//
// Few tokens (linear_rows_kernel): the weights' bytes bound the call.  Both
// operands are decoded to bf16 (exact: E4M3 has four significant bits, the
// block scale is a power of two) and multiplied on the bf16 matrix cores,
// whose products and sums are exact to float32; the FP8 matrix cores drop
// bits below about 2^-16 of the largest product of a group (measured: 1.4e-5
// of the sum's rms against 4e-8), and at these sizes their rate is not
// needed.
#include "ops_internal.h"

namespace moe {
namespace {

__device__ inline i32x8_t operand(const uint4& lo, const uint4& hi) {
    return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// v / (1 + exp(-v)); the hardware exponential and reciprocal (about 1 ulp each)
__device__ inline float silu(float v) { return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
// erfc keeps the relative precision of the left tail that 1 + erf loses
__device__ inline float gelu(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// What a lane does with the sums of G 16-row groups of one quad and one token:
// acc[i][j] = row 4 g + j of group `group(i)`: the groups are sub * G + i,
// or, with gate/up pairs (groups 0, 1 gate and 2, 3 up rows) and G = 2, gate
// group sub and up group sub + 2.  Every lane of the wave takes part (the
// MXFP8 block scales need the four lanes of a token); `live` lanes store.
// MXFP8 output takes whole blocks of 32 columns: G >= 2, gated G = 4.
template <int G>
__device__ inline void finish(const moe_mxfp8_linear_args& a, int64_t quad, int sub, int64_t t, bool live,
                              f32x4_t (&acc)[G]) {
    const int g = (threadIdx.x % kWave) / 16;
    const bool gated = a.activation == MOE_EPI_SILU_MUL;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < G; i++) {
            const int h = G / 2;  // gated: groups i >= h are up rows
            const int64_t row = gated ? (i < h ? 0 : a.rows / 2) + 32 * quad + 16 * (sub * h + (h ? i % h : 0))
                                      : 64 * quad + 16 * (sub * G + i);
            const float4 b = *reinterpret_cast<const float4*>(a.bias + row + 4 * g);
            acc[i] += f32x4_t{b.x, b.y, b.z, b.w};
        }
    }
    int groups = G;  // 16-column groups of output, from column c0
    int64_t c0 = 64 * quad + 16 * sub * G, cols = a.rows;
    if (gated) {
        groups = G / 2;
        c0 = 32 * quad + 16 * sub * (G / 2);
        cols = a.rows / 2;
#pragma unroll
        for (int i = 0; i < G / 2; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = silu(acc[i][j]) * acc[i + G / 2][j];
    } else if (a.activation == MOE_EPI_SILU) {
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = silu(acc[i][j]);
    } else if (a.activation == MOE_EPI_GELU) {
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = gelu(acc[i][j]);
    }
    if (a.residual && live) {
        const uint16_t* r = (const uint16_t*)a.residual + t * a.residual_stride + c0 + 4 * g;
#pragma unroll
        for (int i = 0; i < G; i++) {
            if (i >= groups) break;
            float v[4];
            load_piece<4>(r + 16 * i, v);
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] += v[j];
        }
    }
    if (a.out) {
        if (!live) return;
        uint16_t* o = (uint16_t*)a.out + t * a.out_stride + c0 + 4 * g;
#pragma unroll
        for (int i = 0; i < G; i++) {
            if (i >= groups) break;
            const float v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
            store_piece<4>(o + 16 * i, v);
        }
        return;
    }
    if constexpr (G >= 2) {
#pragma unroll
        for (int b = 0; b < G / 2; b++) {  // blocks of 32 columns: groups 2b, 2b + 1
            if (2 * b >= groups) break;
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int j = 0; j < 4; j++) top = max(top, __float_as_uint(acc[2 * b + h][j]) & 0x7fffffffu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const bool bad = top >= 0x7f800000u;
            const int se = mxfp8_scale_exp(top);
            if (!live) continue;
            uint8_t* o = a.out_codes + t * cols + c0 + 32 * b + 4 * g;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float q[4];
#pragma unroll
                for (int j = 0; j < 4; j++) q[j] = bad ? 0.f : ldexpf(acc[2 * b + h][j], -se);
                *reinterpret_cast<uint32_t*>(o + 16 * h) = e4m3_pack4(q);
            }
            if (g == 0) a.out_scales[t * (cols / 32) + c0 / 32 + b] = bad ? 255 : (uint8_t)(se + 127);
        }
    }
}

// A split of the inner axis leaves float32 sums in the workspace, one float4
// per lane in the order the lanes hold them: [split][token tile][group][lane].
__device__ inline float4* partial_of(const moe_mxfp8_linear_args& a, int split, int64_t tile, int64_t group) {
    const int64_t tiles = (a.num_tokens + 15) / 16;
    return (float4*)a.workspace + ((split * tiles + tile) * (a.rows / 16) + group) * kWave + threadIdx.x % kWave;
}

// one wave per (quad, 16-token tile): the splits' sums in order, then finish
__global__ void __launch_bounds__(256) linear_finish_kernel(moe_mxfp8_linear_args a, int splits) {
    const int64_t quads = a.rows / 64, unit = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
    const int64_t quad = unit % quads, tile = unit / quads;
    if (16 * tile >= a.num_tokens) return;
    f32x4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; s++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float4 v = *partial_of(a, s, tile, 4 * quad + i);
            acc[i] += f32x4_t{v.x, v.y, v.z, v.w};
        }
    const int64_t t = 16 * tile + threadIdx.x % 16;
    finish<4>(a, quad, 0, t, t < a.num_tokens, acc);
}

// ------------------------------------------------------------ few tokens
// A workgroup of W waves owns G 16-row groups of a quad and NT 16-token
// tiles; its waves take the chunks of its part of the inner axis in turn and
// add their sums in LDS, in wave order.  Weights and tokens go straight from
// global memory to registers (a tile-layout load is a contiguous 1 KB per
// wave), one chunk ahead.
template <int G, int NT>
struct RowsChunk {
    u32x4_t a[G][2], b[NT][2];
    uint32_t sa, sb[NT];
};

struct RowsGrid {
    int units, groups;          // weight units (rows / 16G), token groups of NT tiles
    int splits, split_chunks;   // parts of the inner axis, chunks of one
};

template <int G, int NT, int W>
__global__ void __launch_bounds__(W * kWave) linear_rows_kernel(moe_mxfp8_linear_args a, RowsGrid p) {
    __shared__ f32x4_t red[W][NT * G][kWave];
    constexpr bool kPaired = G == 2;
    const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
    // the token groups of a unit run on one XCD (workgroups go round the
    // eight), where its weights come from HBM once
    const int per_split = 8 * p.groups * ((p.units + 7) / 8);
    const int split = blockIdx.x / per_split, b0 = blockIdx.x % per_split;
    const int unit = b0 / (8 * p.groups) * 8 + b0 % 8, tg = b0 / 8 % p.groups;
    if (unit >= p.units) return;
    const int64_t quad = unit / (4 / G);
    const int sub = unit % (4 / G);
    const int chunks = (int)(a.inner / 128);
    const int k0 = split * p.split_chunks, k1 = min(chunks, k0 + p.split_chunks);
    const bool gated = kPaired && a.activation == MOE_EPI_SILU_MUL;
    int group[G];
#pragma unroll
    for (int i = 0; i < G; i++) group[i] = gated ? sub + 2 * i : sub * G + i;
    const uint8_t* wt = a.w_tiles + quad * chunks * 8192 + lane * 16;
    const uint8_t* ws = a.w_scales + quad * chunks * 256 + lane * 4;
    const uint8_t *xr[NT], *xs[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t tok = min((int64_t)(16 * (tg * NT + t) + c), a.num_tokens - 1);
        xr[t] = a.x_codes + tok * a.inner + 32 * g;
        xs[t] = a.x_scales + tok * (a.inner / 32) + g;
    }
    f32x4_t acc[NT][G];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < G; i++) acc[t][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // loads are unconditional (chunks past the end repeat the last one and
    // are not multiplied): the compiler then waits for exactly what it uses
    auto load = [&](RowsChunk<G, NT>& r, int k) {
        const int ch = min(k, k1 - 1);
        r.sa = *reinterpret_cast<const uint32_t*>(ws + (int64_t)ch * 256);
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                r.a[i][h] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(wt + (int64_t)ch * 8192 + group[i] * 2048 + h * 1024));
#pragma unroll
        for (int t = 0; t < NT; t++) {
            r.sb[t] = xs[t][ch * 4];
#pragma unroll
            for (int h = 0; h < 2; h++)
                r.b[t][h] = *reinterpret_cast<const u32x4_t*>(xr[t] + ch * 128 + 16 * h);
        }
    };
    auto multiply = [&](const RowsChunk<G, NT>& r) {
#pragma unroll
        for (int q = 0; q < 4; q++) {  // k = 32 g + 8 q .. + 7 of each lane group
            bf16x8_t B[NT];
#pragma unroll
            for (int t = 0; t < NT; t++)
                B[t] = decode8_e4m3(r.b[t][q / 2][2 * (q % 2)], r.b[t][q / 2][2 * (q % 2) + 1],
                                    e8m0_as_scale(r.sb[t]));
#pragma unroll
            for (int i = 0; i < G; i++) {
                const bf16x8_t A = decode8_e4m3(r.a[i][q / 2][2 * (q % 2)], r.a[i][q / 2][2 * (q % 2) + 1],
                                                e8m0_as_scale((r.sa >> (8 * group[i])) & 0xffu));
#pragma unroll
                for (int t = 0; t < NT; t++)
                    acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[t], acc[t][i], 0, 0, 0);
            }
        }
    };
    RowsChunk<G, NT> r0, r1;
    load(r0, k0 + w);
    for (int k = k0 + w; k < k1; k += 2 * W) {
        load(r1, k + W);
        multiply(r0);
        load(r0, k + 2 * W);
        if (k + W < k1) multiply(r1);
    }
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < G; i++) red[w][t * G + i][lane] = acc[t][i];
    __syncthreads();
    for (int t = w; t < NT; t += W) {
        const int64_t tile = tg * NT + t;
        if (16 * tile >= a.num_tokens) break;
        f32x4_t v[G];
#pragma unroll
        for (int i = 0; i < G; i++) {
            v[i] = red[0][t * G + i][lane];
#pragma unroll
            for (int u = 1; u < W; u++) v[i] += red[u][t * G + i][lane];
        }
        if (p.splits > 1) {
#pragma unroll
            for (int i = 0; i < G; i++)
                *partial_of(a, split, tile, 4 * quad + group[i]) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        } else {
            const int64_t tok = 16 * tile + c;
            finish<G>(a, quad, sub, tok, tok < a.num_tokens, v);
        }
    }
}

// One wave: one quad x 16 tokens over the whole inner axis, both operands
// straight from global memory.
__global__ void __launch_bounds__(kWave) linear_wave_kernel(moe_mxfp8_linear_args a) {
    const int lane = threadIdx.x, c = lane % 16, g = lane / 16;
    const int64_t quads = a.rows / 64, quad = blockIdx.x % quads, tile = blockIdx.x / quads;
    const int chunks = (int)(a.inner / 128);
    const int64_t t = 16 * tile + c;
    const bool live = t < a.num_tokens;
    const int64_t tt = live ? t : a.num_tokens - 1;
    const uint8_t* x = a.x_codes + tt * a.inner + 16 * g;
    const uint8_t* xs = a.x_scales + tt * (a.inner / 32) + g;
    const uint8_t* w = a.w_tiles + quad * chunks * 8192 + (g & 1) * 1024 + (c + 16 * (g >> 1)) * 16;
    const uint8_t* ws = a.w_scales + quad * chunks * 256 + lane * 4;
    f32x4_t acc[4];
#pragma unroll
    for (int rg = 0; rg < 4; rg++) acc[rg] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int ch = 0; ch < chunks; ch++) {
        const i32x8_t B = operand(*reinterpret_cast<const uint4*>(x + ch * 128),
                                  *reinterpret_cast<const uint4*>(x + ch * 128 + 64));
        const uint32_t sb = xs[ch * 4];
        const uint32_t sa = *reinterpret_cast<const uint32_t*>(ws + (int64_t)ch * 256);
        const uint8_t* wc = w + (int64_t)ch * 8192;
        static_for<4>([&](auto rg) {
            const i32x8_t A = operand(*reinterpret_cast<const uint4*>(wc + rg * 2048),
                                      *reinterpret_cast<const uint4*>(wc + rg * 2048 + 512));
            acc[rg] = mfma_scaled<0, rg, 0>(A, B, acc[rg], sa, sb);
        });
    }
    finish<4>(a, quad, 0, t, live, acc);
}

// ------------------------------------------------------------ the choice
constexpr int kRowsMaxTok = 128;  // tokens of linear_rows_kernel

struct LinearPlan {
    bool rows;       // linear_rows_kernel
    int G, NT, W;
    RowsGrid grid;
};

LinearPlan make_plan(int64_t T, int64_t rows, int64_t inner, int32_t activation, bool mx) {
    LinearPlan p{};
    const int tiles = (int)((T + 15) / 16), chunks = (int)(inner / 128);
    const bool gated = activation == MOE_EPI_SILU_MUL;
    p.rows = T <= kRowsMaxTok;
    if (!p.rows) return p;
    if (tiles <= 2) {
        p.G = mx ? (gated ? 4 : 2) : gated ? 2 : 1;
        p.NT = tiles;
        p.W = 8;
        p.grid.groups = 1;
        p.grid.splits = 1;
    } else {
        p.G = 4;
        p.W = 4;
        p.grid.groups = (tiles + 3) / 4;
        p.NT = (tiles + p.grid.groups - 1) / p.grid.groups;
        // enough workgroups for two per CU, as long as each wave keeps two
        // chunks and the partial sums stay within 32 bytes per product
        int64_t splits = 512 / (rows / 64 * p.grid.groups);
        if (splits > chunks / 8) splits = chunks / 8;
        if (splits > 8 * T / (16 * tiles)) splits = 8 * T / (16 * tiles);
        p.grid.splits = splits < 1 ? 1 : (int)splits;
    }
    p.grid.units = (int)(rows / (16 * p.G));
    p.grid.split_chunks = (chunks + p.grid.splits - 1) / p.grid.splits;
    p.grid.splits = (chunks + p.grid.split_chunks - 1) / p.grid.split_chunks;
    return p;
}

template <int G, int NT, int W>
void launch_rows(const moe_mxfp8_linear_args& a, const RowsGrid& p, hipStream_t stream) {
    const unsigned grid = (unsigned)(p.splits * 8 * p.groups * ((p.units + 7) / 8));
    linear_rows_kernel<G, NT, W><<<grid, W * kWave, 0, stream>>>(a, p);
}

}  // namespace

int64_t mxfp8_linear_workspace(int64_t T, int64_t rows, int64_t inner, int32_t activation) {
    if (T == 0) return 0;
    const LinearPlan p = make_plan(T, rows, inner, activation, false);
    return p.rows && p.grid.splits > 1 ? p.grid.splits * ((T + 15) / 16) * rows * 64 : 0;
}

hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream) {
    const LinearPlan p = make_plan(a.num_tokens, a.rows, a.inner, a.activation, a.out_codes != nullptr);
    if (!p.rows) {
        const int64_t grid = a.rows / 64 * ((a.num_tokens + 15) / 16);
        linear_wave_kernel<<<(unsigned)grid, kWave, 0, stream>>>(a);
        return hipGetLastError();
    }
    const RowsGrid& r = p.grid;
    if (p.W == 8) {
        if (p.G == 1) p.NT == 1 ? launch_rows<1, 1, 8>(a, r, stream) : launch_rows<1, 2, 8>(a, r, stream);
        else if (p.G == 2) p.NT == 1 ? launch_rows<2, 1, 8>(a, r, stream) : launch_rows<2, 2, 8>(a, r, stream);
        else p.NT == 1 ? launch_rows<4, 1, 8>(a, r, stream) : launch_rows<4, 2, 8>(a, r, stream);
    } else {
        if (p.NT <= 3) launch_rows<4, 3, 4>(a, r, stream);
        else launch_rows<4, 4, 4>(a, r, stream);
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || r.splits == 1) return err;
    const int64_t units = a.rows / 64 * ((a.num_tokens + 15) / 16);
    linear_finish_kernel<<<(unsigned)((units + 3) / 4), 256, 0, stream>>>(a, r.splits);
    return hipGetLastError();
}

}  // namespace moe
