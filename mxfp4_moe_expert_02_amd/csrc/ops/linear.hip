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
#include "../lds_dma.h"
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

// ----------------------------------------------------------- many tokens
// A workgroup computes RQ quads x TT 16-token tiles; its WR x WT waves own
// RQ / WR quads x TT / WT tiles each.  Per 128-k chunk both operands go from
// global memory straight to LDS: A as the tile layout has it, B as token rows
// of 128 bytes with 16-byte piece p of token c in slot p ^ (c / 2 % 8), so
// that the 16 lanes of an operand read cover all banks.  A load of B takes 8
// whole rows: with the rows' pieces spread over the lanes in operand order
// instead (16 rows x 64 bytes per load) every quarter of a wave touches 16
// cache lines, and the loads alone took 1.55 us a chunk against 0.6.  On the
// FP8 matrix cores
// (v_mfma_scale_f32_16x16x128_f8f6f4): lane (r, g) of an operand holds the
// 16-byte pieces g and g + 4 of row r's 128 bytes and the scale of block g.
template <int RQ, int TT, int STAGES>
struct TileSmem {
    alignas(16) uint8_t a[STAGES][RQ][8192];
    alignas(16) uint8_t b[STAGES][TT][2048];
    alignas(16) uint32_t as[STAGES][RQ][kWave];
    alignas(16) uint32_t bs[STAGES][TT * 16];
};

struct TileGrid {
    int row_blocks, tok_blocks;
    int splits, split_chunks;
};

template <int RQ, int TT, int WR, int WT>
__global__ void __launch_bounds__(WR * WT * kWave) linear_tile_kernel(moe_mxfp8_linear_args a, TileGrid p) {
    constexpr int kStages = 2, kWaves = WR * WT;
    constexpr int Q = RQ / WR, NT = TT / WT;              // a wave's quads and token tiles
    constexpr int kA = RQ * 8 / kWaves, kB = TT * 2 / kWaves;  // 1 KB loads per wave and chunk
    static_assert(RQ * 8 % kWaves == 0 && TT * 2 % kWaves == 0 && RQ + TT / 4 == kWaves, "loads per wave");
    extern __shared__ uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<TileSmem<RQ, TT, kStages>*>(smem_raw);
    const int w = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
    const int per_split = p.row_blocks * p.tok_blocks;
    const int split = blockIdx.x / per_split, blk = blockIdx.x % per_split;
    const int rb = blk % p.row_blocks, tb = blk / p.row_blocks;
    const int chunks = (int)(a.inner / 128), quads = (int)(a.rows / 64);
    const int k0 = split * p.split_chunks, k1 = min(chunks, k0 + p.split_chunks);
    const int q0 = rb * RQ;
    const int64_t t0 = (int64_t)tb * (16 * TT);
    const int last = (int)min((int64_t)(16 * TT), a.num_tokens - t0) - 1;  // rows past it repeat it

    // this wave's loads of chunk k0 (quads past the end repeat the last one)
    const uint8_t* srcA[kA];
    const uint8_t* srcB[kB];
    const uint8_t* srcS;
    int step_s;
#pragma unroll
    for (int i = 0; i < kA; i++) {
        const int piece = w * kA + i;  // quad piece / 8, 1 KB piece % 8
        srcA[i] = a.w_tiles + ((int64_t)min(q0 + piece / 8, quads - 1) * chunks + k0) * 8192 + piece % 8 * 1024 + lane * 16;
    }
#pragma unroll
    for (int i = 0; i < kB; i++) {
        const int row = (w * kB + i) * 8 + lane / 8;  // eight token rows per load
        srcB[i] = a.x_codes + (t0 + min(row, last)) * a.inner + (int64_t)k0 * 128 + ((lane % 8) ^ (row / 2 % 8)) * 16;
    }
    if (w < RQ) {
        srcS = a.w_scales + ((int64_t)min(q0 + w, quads - 1) * chunks + k0) * 256 + lane * 4;
        step_s = 256;
    } else {
        const int64_t tok = t0 + min((w - RQ) * kWave + lane, last);
        srcS = a.x_scales + tok * (a.inner / 32) + (int64_t)k0 * 4;
        step_s = 4;
    }
    auto issue = [&](int k, int buf) {
        const int d = k - k0;
#pragma unroll
        for (int i = 0; i < kA; i++)
            dma16(srcA[i] + (int64_t)d * 8192, lds_addr(&sm.a[buf][0][(w * kA + i) * 1024]));
#pragma unroll
        for (int i = 0; i < kB; i++)
            dma16(srcB[i] + d * 128, lds_addr(&sm.b[buf][0][(w * kB + i) * 1024]));
        dma4(srcS + (int64_t)d * step_s, lds_addr(w < RQ ? (const void*)&sm.as[buf][w][0]
                                                        : (const void*)&sm.bs[buf][(w - RQ) * kWave]));
    };
    const int wr = w % WR, wt = w / WR;
    f32x4_t acc[Q][4][NT];
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int t = 0; t < NT; t++) acc[q][i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    issue(k0, 0);
    int buf = 0;
    const int a_lo = (g & 1) * 1024 + (c + 16 * (g >> 1)) * 16;  // piece g; piece g + 4 is 512 bytes on
    const int b_lo = c * 128 + (g ^ (c / 2)) * 16;               // piece g; piece g + 4 is in slot ^ 4
    for (int k = k0; k < k1; k++) {
        // this wave's loads of chunk k have landed; after the barrier every
        // wave's have, and every wave is done reading the other buffer
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        if (k + 1 < k1) issue(k + 1, buf ^ 1);
        i32x8_t B[NT];
        uint32_t sb[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int tile = wt * NT + t;
            B[t] = operand(*reinterpret_cast<const uint4*>(&sm.b[buf][tile][b_lo]),
                           *reinterpret_cast<const uint4*>(&sm.b[buf][tile][b_lo ^ 64]));
            sb[t] = reinterpret_cast<const uint8_t*>(&sm.bs[buf][tile * 16 + c])[g];
        }
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const uint8_t* qa = &sm.a[buf][wr * Q + q][a_lo];
            const uint32_t sa = sm.as[buf][wr * Q + q][lane];
            static_for<4>([&](auto i) {
                const i32x8_t A = operand(*reinterpret_cast<const uint4*>(qa + i * 2048),
                                          *reinterpret_cast<const uint4*>(qa + i * 2048 + 512));
#pragma unroll
                for (int t = 0; t < NT; t++) acc[q][i][t] = mfma_scaled<0, i, 0>(A, B[t], acc[q][i][t], sa, sb[t]);
            });
        }
        buf ^= 1;
    }
    // The sums leave through this wave's own part of the LDS (one quad x tile
    // a time, in the lanes' own order), so that the epilogue is one piece of
    // code in a loop instead of Q * NT copies of it.
    __syncthreads();
    constexpr int kUnits = Q * NT;
    constexpr int kRound = sizeof(TileSmem<RQ, TT, kStages>) / (kWaves * 4096) < kUnits
                               ? sizeof(TileSmem<RQ, TT, kStages>) / (kWaves * 4096) : kUnits;
    f32x4_t(*mine)[4][kWave] = reinterpret_cast<f32x4_t(*)[4][kWave]>(smem_raw + w * kRound * 4096);
    static_for<(kUnits + kRound - 1) / kRound>([&](auto round) {
        static_for<kRound>([&](auto u) {
            constexpr int n = decltype(round)::value * kRound + decltype(u)::value;
            if constexpr (n < kUnits) {
#pragma unroll
                for (int i = 0; i < 4; i++) mine[u][i][lane] = acc[n / NT][i][n % NT];
            }
        });
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int u = 0; u < kRound; u++) {
            const int n = round * kRound + u;
            const int quad = q0 + wr * Q + n / NT;
            const int64_t tile = (int64_t)tb * TT + wt * NT + n % NT;
            if (n >= kUnits || quad >= quads || 16 * tile >= a.num_tokens) continue;
            f32x4_t v[4];
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = mine[u][i][lane];
            if (p.splits > 1) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    *partial_of(a, split, tile, 4 * quad + i) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            } else {
                const int64_t t = 16 * tile + c;
                finish<4>(a, quad, 0, t, t < a.num_tokens, v);
            }
        }
        __builtin_amdgcn_wave_barrier();
    });
}

// ------------------------------------------------------------ the choice
constexpr int kRowsMaxTok = 128;   // tokens of linear_rows_kernel
constexpr int kSplitMaxTok = 1024;  // most tokens whose inner axis is split

struct LinearPlan {
    bool rows;       // linear_rows_kernel
    int G, NT, W;
    RowsGrid grid;
    bool wide;       // 256 x 256 tiles (else 128 x 128)
    TileGrid tile;
};

LinearPlan make_plan(int64_t T, int64_t rows, int64_t inner, int32_t activation, bool mx) {
    LinearPlan p{};
    const int tiles = (int)((T + 15) / 16), chunks = (int)(inner / 128);
    const bool gated = activation == MOE_EPI_SILU_MUL;
    p.rows = T <= kRowsMaxTok;
    if (!p.rows) {
        const int64_t wide_blocks = (rows + 255) / 256 * ((T + 255) / 256);
        p.wide = wide_blocks >= 192;
        const int n = p.wide ? 256 : 128;
        p.tile.row_blocks = (int)((rows + n - 1) / n);
        p.tile.tok_blocks = (int)((T + n - 1) / n);
        int64_t splits = 1;
        if (!p.wide && T <= kSplitMaxTok) {
            splits = 512 / ((int64_t)p.tile.row_blocks * p.tile.tok_blocks);
            if (splits > chunks / 8) splits = chunks / 8;
            if (splits > 8 * T / (16 * tiles)) splits = 8 * T / (16 * tiles);
        }
        p.tile.splits = splits < 1 ? 1 : (int)splits;
        p.tile.split_chunks = (chunks + p.tile.splits - 1) / p.tile.splits;
        p.tile.splits = (chunks + p.tile.split_chunks - 1) / p.tile.split_chunks;
        return p;
    }
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

template <int RQ, int TT, int WR, int WT>
hipError_t launch_tile(const moe_mxfp8_linear_args& a, const TileGrid& p, hipStream_t stream) {
    constexpr int bytes = sizeof(TileSmem<RQ, TT, 2>);
    const auto kernel = linear_tile_kernel<RQ, TT, WR, WT>;
    if (bytes > 65536) {  // more than 64 KB of LDS has to be asked for
        const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
    }
    const unsigned grid = (unsigned)((int64_t)p.splits * p.row_blocks * p.tok_blocks);
    kernel<<<grid, WR * WT * kWave, bytes, stream>>>(a, p);
    return hipGetLastError();
}

int splits_of(const LinearPlan& p) { return p.rows ? p.grid.splits : p.tile.splits; }

}  // namespace

int64_t mxfp8_linear_workspace(int64_t T, int64_t rows, int64_t inner, int32_t activation) {
    if (T == 0) return 0;
    const int splits = splits_of(make_plan(T, rows, inner, activation, false));
    return splits > 1 ? splits * ((T + 15) / 16) * rows * 64 : 0;
}

hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream) {
    const LinearPlan p = make_plan(a.num_tokens, a.rows, a.inner, a.activation, a.out_codes != nullptr);
    const RowsGrid& r = p.grid;
    hipError_t err = hipSuccess;
    if (!p.rows) {
        err = p.wide ? launch_tile<4, 16, 2, 4>(a, p.tile, stream) : launch_tile<2, 8, 2, 2>(a, p.tile, stream);
    } else if (p.W == 8) {
        if (p.G == 1) p.NT == 1 ? launch_rows<1, 1, 8>(a, r, stream) : launch_rows<1, 2, 8>(a, r, stream);
        else if (p.G == 2) p.NT == 1 ? launch_rows<2, 1, 8>(a, r, stream) : launch_rows<2, 2, 8>(a, r, stream);
        else p.NT == 1 ? launch_rows<4, 1, 8>(a, r, stream) : launch_rows<4, 2, 8>(a, r, stream);
        err = hipGetLastError();
    } else {
        if (p.NT <= 3) launch_rows<4, 3, 4>(a, r, stream);
        else launch_rows<4, 4, 4>(a, r, stream);
        err = hipGetLastError();
    }
    const int splits = splits_of(p);
    if (err != hipSuccess || splits == 1) return err;
    const int64_t units = a.rows / 64 * ((a.num_tokens + 15) / 16);
    linear_finish_kernel<<<(unsigned)((units + 3) / 4), 256, 0, stream>>>(a, splits);
    return hipGetLastError();
}

}  // namespace moe
