// linear.hip -- out = act(x W^T + bias) + residual with x and W in MXFP8, on
// the scaled matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4).
//
// The weights come in the MXFP8 tile layout of moe_mxfp8_prepack (prepack.hip):
// per 64-row quad and 128-k chunk 8 KB of codes [group][half][lane][16] and
// 256 scale bytes [lane][group].  Operands of one 16x16x128 product, lane
// (r, g) = (l % 16, l / 16):
//   A: 16 weight rows; lane (r, g) holds the 16-byte pieces g and g + 4 of
//      row r's 128 bytes, and the scale of block g;
//   B: 16 tokens, the same pieces and scale of token r's row;
//   D: lane (c, g) holds rows 4g .. 4g+3 of token c.
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

// What a lane does with the sums of one quad and token: acc[rg][i] = row
// 16 rg + 4 g + i of the quad (with gate/up pairs: groups 0, 1 gate and 2, 3
// up rows).  Every lane of the wave takes part (the MXFP8 block scales need
// the four lanes of a token); `live` lanes store.
__device__ inline void finish_quad(const moe_mxfp8_linear_args& a, int64_t quad, int64_t t, bool live,
                                   f32x4_t (&acc)[4]) {
    const int g = (threadIdx.x % kWave) / 16;
    const bool gated = a.activation == MOE_EPI_SILU_MUL;
    if (a.bias) {
#pragma unroll
        for (int rg = 0; rg < 4; rg++) {
            const int64_t row = gated ? (rg < 2 ? 0 : a.rows / 2) + 32 * quad + 16 * (rg & 1)
                                      : 64 * quad + 16 * rg;
            const float4 b = *reinterpret_cast<const float4*>(a.bias + row + 4 * g);
            acc[rg] += f32x4_t{b.x, b.y, b.z, b.w};
        }
    }
    int groups = 4;  // 16-column groups of output, from column c0
    int64_t c0 = 64 * quad, cols = a.rows;
    if (gated) {
        groups = 2;
        c0 = 32 * quad;
        cols = a.rows / 2;
#pragma unroll
        for (int rg = 0; rg < 2; rg++)
#pragma unroll
            for (int i = 0; i < 4; i++) acc[rg][i] = silu(acc[rg][i]) * acc[rg + 2][i];
    } else if (a.activation == MOE_EPI_SILU) {
#pragma unroll
        for (int rg = 0; rg < 4; rg++)
#pragma unroll
            for (int i = 0; i < 4; i++) acc[rg][i] = silu(acc[rg][i]);
    } else if (a.activation == MOE_EPI_GELU) {
#pragma unroll
        for (int rg = 0; rg < 4; rg++)
#pragma unroll
            for (int i = 0; i < 4; i++) acc[rg][i] = gelu(acc[rg][i]);
    }
    if (a.residual && live) {
        const uint16_t* r = (const uint16_t*)a.residual + t * a.residual_stride + c0 + 4 * g;
#pragma unroll
        for (int rg = 0; rg < 4; rg++) {
            if (rg >= groups) break;
            float v[4];
            load_piece<4>(r + 16 * rg, v);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[rg][i] += v[i];
        }
    }
    if (a.out) {
        if (!live) return;
        uint16_t* o = (uint16_t*)a.out + t * a.out_stride + c0 + 4 * g;
#pragma unroll
        for (int rg = 0; rg < 4; rg++) {
            if (rg >= groups) break;
            const float v[4] = {acc[rg][0], acc[rg][1], acc[rg][2], acc[rg][3]};
            store_piece<4>(o + 16 * rg, v);
        }
        return;
    }
#pragma unroll
    for (int b = 0; b < 2; b++) {  // blocks of 32 columns: groups 2b, 2b + 1
        if (2 * b >= groups) break;
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 4; i++) top = max(top, __float_as_uint(acc[2 * b + h][i]) & 0x7fffffffu);
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
            for (int i = 0; i < 4; i++) q[i] = bad ? 0.f : ldexpf(acc[2 * b + h][i], -se);
            *reinterpret_cast<uint32_t*>(o + 16 * h) = e4m3_pack4(q);
        }
        if (g == 0) a.out_scales[t * (cols / 32) + c0 / 32 + b] = bad ? 255 : (uint8_t)(se + 127);
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
    finish_quad(a, quad, t, live, acc);
}

}  // namespace

int64_t mxfp8_linear_workspace(int64_t, int64_t, int64_t, int32_t) { return 0; }

hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream) {
    const int64_t grid = a.rows / 64 * ((a.num_tokens + 15) / 16);
    linear_wave_kernel<<<(unsigned)grid, kWave, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
