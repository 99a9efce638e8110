// linear.hip -- out = act(x W^T + bias) + residual with x and W in MXFP8.
//
// The weights come in the MXFP8 tile layout of moe_mxfp8_prepack (prepack.hip):
// per 64-row quad and 128-k chunk 8 KB of codes [group][half][lane][16] and
// 256 scale bytes [lane][group], lane (r, g) = (l % 16, l / 16) holding block
// g (k = 32g .. 32g+31) of row r.
//
// Both operands are decoded to bf16 (exact: E4M3 has four significant bits, the
// block scale is a power of two) and multiplied on the bf16 matrix cores,
// whose products and sums are exact to float32.  The FP8 matrix cores, twice
// as fast, keep the products of eight consecutive k to 13 bits below the
// largest of them: 1.4e-5 of the sum's rms against 4e-8, and nothing of a
// small product beside two large ones that cancel.  They are not used.
// Few tokens (linear_rows_kernel): the weights' bytes bound the call.
// 9 x 6144 x 6144 10.5 us (39 MB, 3.7 TB/s), 72 x 4096 x 7168 16.9.
// Many tokens (linear_tile_kernel): tiles of up to 256 x 256 staged through LDS
// as they are in memory; each wave decodes what it multiplies, between its
// products.  4096 x 7168 x 7168 with bias and residual 343 us (1.23 PFLOP/s;
// without them and from the caches 318, 1.32; a bf16 product of a library
// reaches 1.26): bound by the matrix cores, at the clock that random operands
// leave them, and the vector instructions beside them, and by the second
// round's 192 tiles on 256 CUs (4096 x 8192 x 8192, two full rounds: 1.42
// PFLOP/s).  288 x 7168 x 7168 54 us, 1001 x 2048 x 6144 37: one wave per SIMD,
// whose products wait for its conversions.
// Either may split the inner axis over workgroups that leave float32 sums in
// the workspace for linear_finish_kernel.
#include "lds_dma.h"
#include "linear_plan.h"
#include "ops_internal.h"

namespace moe {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// v / (1 + exp(-v)), relative error up to (8 + |v|) 2^-23 (the exponential's
// argument is rounded).  Below -64 the 1 does not count, and from -87 on
// exp(-v) and then its reciprocal leave float32's normal range while v exp(v)
// is inside it: taken there in two halves.
__device__ inline float silu(float v) {
    const float h = __expf(0.5f * v);
    return v < -64.f ? v * h * h : v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

// v / 2 * (1 + erf(v / sqrt 2)) = v / 2 * erfc(-v / sqrt 2): erfc keeps the
// relative precision of the left tail that 1 + erf loses.  For a >= 0,
// erfc(a) = t exp(-a^2) f(t) with t = 1 / (1 + 0.4 a); f is a least-squares
// polynomial for f(t) = erfc(a) exp(a^2) / t, weighted towards the smallest
// largest relative error, 3e-8.  The function's own is up to (16 + 2 v^2) 2^-23,
// since a^2 is rounded before the exponential: 4e-7 for |v| <= 1, 1.1e-6 to 3,
// 6e-6 at -9, 1.5e-5 at -13 (emulated in float32 against 64 bits).  Below -13.2,
// where the result is below float32's normal range, it is zero.
__device__ inline float gelu(float v) {
    const float a = fabsf(v) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.4f, a, 1.0f));
    float f = -0.0224578306f;
    f = fmaf(f, t, 0.160047933f);
    f = fmaf(f, t, -0.411607653f);
    f = fmaf(f, t, 0.43421036f);
    f = fmaf(f, t, -0.193026885f);
    f = fmaf(f, t, 0.224716902f);
    f = fmaf(f, t, 0.14541091f);
    f = fmaf(f, t, 0.211696655f);
    f = fmaf(f, t, 0.225320622f);
    f = fmaf(f, t, 0.225688994f);
    const float r = t * f * __expf(-a * a);
    return 0.5f * v * (v > 0.f ? 2.0f - r : r);
}

// ------------------------------------------------------------- the output
// A lane finishes 8 consecutive columns of one token: v holds their sums,
// and with gate/up pairs u those of the up rows.

__device__ inline void add8(float (&v)[8], const float* p) {  // 16-byte aligned
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
}

__device__ inline uint4 residual8(const moe_mxfp8_linear_args& a, int64_t t, int64_t c0) {
    return *reinterpret_cast<const uint4*>((const uint16_t*)a.residual + t * a.residual_stride + c0);
}

// the largest of v over the four lanes of a quad (a block of 32 columns)
__device__ inline uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));  // lanes 1, 0, 3, 2
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));  // lanes 2, 3, 0, 1
}

// columns c0 .. c0+7 of token t (live lanes store; whole quads of lanes take
// part).  act and mx are constants where the caller's are.
__device__ inline void finish8(const moe_mxfp8_linear_args& a, int act, bool mx, int64_t cols, int64_t t, int64_t c0,
                               bool live, float (&v)[8], const float (&u)[8], const uint4& res) {
    if (act == MOE_EPI_SILU_MUL) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = silu(v[i]) * u[i];
    } else if (act == MOE_EPI_SILU) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = silu(v[i]);
    } else if (act == MOE_EPI_GELU) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = gelu(v[i]);
    }
    if (a.residual) {
        const uint32_t w[4] = {res.x, res.y, res.z, res.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] += __uint_as_float(w[i] << 16);
            v[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    if (!mx) {
        if (live) store_piece<8>((uint16_t*)a.out + t * a.out_stride + c0, v);
        return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = quad_max(top);
    const bool bad = top >= 0x7f800000u;
    const int se = mxfp8_scale_exp(top);
    if (!live) return;
    uint32_t code[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; i++) q[i] = bad ? 0.f : ldexpf(v[4 * h + i], -se);
        code[h] = e4m3_pack4(q);
    }
    *reinterpret_cast<uint2*>(a.out_codes + t * cols + c0) = make_uint2(code[0], code[1]);
    if (c0 % 32 == 0) a.out_scales[t * (cols / 32) + c0 / 32] = bad ? 255 : (uint8_t)(se + 127);
}

// A split of the inner axis leaves float32 sums in the workspace,
// [split][token][row], rows in the tile layout's order (with gate/up pairs:
// 32 gate, then 32 up rows per quad).
__device__ inline float* partial_of(const moe_mxfp8_linear_args& a, int split, int64_t t, int64_t row) {
    return (float*)a.workspace + (split * a.num_tokens + t) * a.rows + row;
}

// one lane per (token, 8 columns): the splits' sums in order, then finish8
__global__ void __launch_bounds__(256) linear_finish_kernel(moe_mxfp8_linear_args a, int splits) {
    const bool gated = a.activation == MOE_EPI_SILU_MUL;
    const int64_t cols = gated ? a.rows / 2 : a.rows, octs = cols / 8;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool live = idx < a.num_tokens * octs;
    const int64_t t = live ? idx / octs : a.num_tokens - 1, o = live ? idx % octs : octs - 1;
    const int64_t row = gated ? o / 4 * 64 + o % 4 * 8 : o * 8;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (a.residual) res = residual8(a, t, 8 * o);
    float v[8] = {}, u[8] = {};
    for (int s = 0; s < splits; s++) {
        add8(v, partial_of(a, s, t, row));
        if (gated) add8(u, partial_of(a, s, t, row + 32));
    }
    if (a.bias) {
        add8(v, a.bias + 8 * o);
        if (gated) add8(u, a.bias + cols + 8 * o);
    }
    finish8(a, a.activation, a.out_codes != nullptr, cols, t, 8 * o, live, v, u, res);
}

// ------------------------------------------------------------ few tokens
// A workgroup of W waves owns G 16-row groups of a quad and NT 16-token
// tiles; each wave takes a run of the chunks of the workgroup's part of the
// inner axis, and the waves' sums meet in LDS, added in wave order.  Weights
// go from global memory to registers (a tile-layout load is a contiguous 1 KB
// per wave), token rows through the wave's own LDS, as whole 128-byte lines
// (16 rows x 16 bytes per quarter wave, which the operand order would give,
// cost a cache access per lane); both D chunks ahead.
constexpr int kSegment = 16;  // chunks whose token scales a wave holds in LDS

template <int NT, int D>
struct RowsWave {  // one wave's staged tokens
    alignas(16) uint8_t x[D][NT][16 * 128];            // rows of 128 bytes, piece p of row c in slot p ^ (c / 2 % 8)
    alignas(16) uint8_t s[NT][kSegment / 4][16 * 16];  // scale bytes [row][4 chunks][4 blocks]
};

template <int G, int NT, int W, int D>
__global__ void __launch_bounds__(W * kWave) linear_rows_kernel(moe_mxfp8_linear_args a, RowsGrid p) {
    union Smem {
        RowsWave<NT, D> wave[W];
        float sum[W][NT * 16][16 * G + 4];  // [wave][token][row], padded
    };
    __shared__ Smem sm;
    const int w = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
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
    const int run = (k1 - k0 + W - 1) / W, r0 = k0 + w * run, r1 = min(k1, r0 + run);  // this wave's chunks
    const bool gated = a.activation == MOE_EPI_SILU_MUL;
    int group[G];  // the 16-row groups of the quad; G = 2 pairs a gate group with its up group
#pragma unroll
    for (int i = 0; i < G; i++) group[i] = G == 2 && gated ? sub + 2 * i : sub * G + i;
    const uint8_t* wt = a.w_tiles + quad * chunks * 8192 + lane * 16;
    const uint8_t* ws = a.w_scales + quad * chunks * 256 + lane * 4;
    const int64_t t0 = (int64_t)tg * (16 * NT);
    const int last = (int)min((int64_t)(16 * NT), a.num_tokens - t0) - 1;  // rows past it repeat it
    const uint8_t *xr[NT][2], *xs[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int row = 8 * h + lane / 8;
            xr[t][h] = a.x_codes + (t0 + min(16 * t + row, last)) * a.inner + ((lane % 8) ^ (row / 2)) * 16;
        }
        xs[t] = a.x_scales + (t0 + min(16 * t + lane / 4, last)) * (a.inner / 32);
    }
    RowsWave<NT, D>& mine = sm.wave[w];
    f32x4_t acc[NT][G];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < G; i++) acc[t][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    struct Weights {
        u32x4_t v[G][2];
        uint32_t s;
    } wb[D];
    auto load = [&](Weights& r, int ch, int buf) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what was read of this buffer has arrived
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < 2; h++) dma16(xr[t][h] + ch * 128, lds_addr(&mine.x[buf][t][1024 * h]));
        r.s = *reinterpret_cast<const uint32_t*>(ws + (int64_t)ch * 256);
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                r.v[i][h] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(wt + (int64_t)ch * 8192 + group[i] * 2048 + h * 1024));
    };
    constexpr int kLoads = 2 * NT + 1 + 2 * G;  // of one chunk
    auto multiply = [&](const Weights& r, int k, int buf) {
        uint4 xb[NT][2];
        uint32_t sb[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int h = 0; h < 2; h++)
                xb[t][h] = *reinterpret_cast<const uint4*>(&mine.x[buf][t][c * 128 + ((2 * g + h) ^ (c / 2)) * 16]);
            sb[t] = mine.s[t][k % kSegment / 4][c * 16 + k % 4 * 4 + g];
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {  // k = 32 g + 8 q .. + 7 of each lane group
            bf16x8_t B[NT];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                const uint4& v = xb[t][q / 2];
                B[t] = q % 2 ? decode8_e4m3(v.z, v.w, e8m0_as_scale(sb[t])) : decode8_e4m3(v.x, v.y, e8m0_as_scale(sb[t]));
            }
#pragma unroll
            for (int i = 0; i < G; i++) {
                const bf16x8_t A = decode8_e4m3(r.v[i][q / 2][2 * (q % 2)], r.v[i][q / 2][2 * (q % 2) + 1],
                                                e8m0_as_scale((r.s >> (8 * group[i])) & 0xffu));
#pragma unroll
                for (int t = 0; t < NT; t++)
                    acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[t], acc[t][i], 0, 0, 0);
            }
        }
    };
    for (int seg = r0; seg < r1; seg += kSegment) {  // k % kSegment counts from the segment's start
        const int n = min(kSegment, r1 - seg);
        for (int j = 0; j < (n + 3) / 4; j++)
#pragma unroll
            for (int t = 0; t < NT; t++)
                dma4(xs[t] + min(seg + 4 * j + lane % 4, r1 - 1) * 4, lds_addr(&mine.s[t][j][0]));
        static_for<D>([&](auto d) {
            if (d < n) load(wb[d], seg + d, d);
        });
        // The wait below counts loads: the next D - 1 chunks' may stay in flight.
        // The weights are ordinary loads, though, for which the compiler waits
        // by itself, and after the conditional loads above it waits for all of
        // them once per D chunks (vmcnt(0) in the compiled loop of all eleven
        // shapes): what was issued last is then in flight for one chunk's
        // products only.
        int i = 0;
        for (; i + 2 * D <= n; i += D)
            static_for<D>([&](auto d) {
                // this chunk has landed
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * kLoads) : "memory");
                multiply(wb[d], i + d, d);
                load(wb[d], seg + i + D + d, d);
            });
        static_for<2 * D - 1>([&](auto d) {
            if (i + d >= n) return;
            if (d == 0 || d == D) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            multiply(wb[d % D], i + d, d % D);
            if (i + D + d < n) load(wb[d % D], seg + i + D + d, d % D);
        });
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // the next segment's scales go over these
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < G; i++)
            *reinterpret_cast<f32x4_t*>(&sm.sum[w][16 * t + c][16 * i + 4 * g]) = acc[t][i];
    __syncthreads();
    // one lane per (token, 8 columns)
    const int octs = gated && p.splits == 1 ? G : 2 * G;
    const int64_t cols = gated ? a.rows / 2 : a.rows;
    for (int idx = threadIdx.x; idx < NT * 16 * octs; idx += W * kWave) {
        const int tok = idx / octs, o = idx % octs;
        const int64_t t = t0 + tok;
        const bool live = tok <= last;
        if (p.splits > 1) {
            float v[8] = {};
#pragma unroll
            for (int u = 0; u < W; u++) add8(v, &sm.sum[u][tok][8 * o]);
            // groups in order (G = 4, or a gate/up pair half a quad apart)
            const int64_t row = 64 * quad + 16 * group[0] + (G == 2 && gated ? o / 2 * 32 + o % 2 * 8 : 8 * o);
            float* d = partial_of(a, split, live ? t : a.num_tokens - 1, row);
            if (live) store_piece<8>(d, v);
            continue;
        }
        const int64_t c0 = gated ? 32 * quad + 16 * sub * (G / 2) + 8 * o : 64 * quad + 16 * sub * G + 8 * o;
        uint4 res = make_uint4(0, 0, 0, 0);
        if (a.residual) res = residual8(a, live ? t : a.num_tokens - 1, c0);
        float v[8] = {}, u[8] = {};
#pragma unroll
        for (int i = 0; i < W; i++) add8(v, &sm.sum[i][tok][8 * o]);
        if (gated)
#pragma unroll
            for (int i = 0; i < W; i++) add8(u, &sm.sum[i][tok][8 * G + 8 * o]);
        if (a.bias) {
            add8(v, a.bias + c0);
            if (gated) add8(u, a.bias + cols + c0);
        }
        finish8(a, a.activation, a.out_codes != nullptr, cols, t, c0, live, v, u, res);
    }
}

// ----------------------------------------------------------- many tokens
// A workgroup computes RQ quads x TT 32-token tiles; its WR x WT waves own
// RQ / WR quads x TT / WT tiles each.  Per 128-k chunk both operands go from
// global memory straight to LDS: A as the tile layout has it, B as token rows
// of 128 bytes with 16-byte piece p of token c in slot p ^ (c / 2 % 8), so
// that the 16 lanes of a quarter wave read all banks once.  A load of B takes
// 8 whole rows: with the rows' pieces spread over the lanes in operand order
// instead (16 rows x 64 bytes per load) every quarter of a wave touches 16
// cache lines, and the loads alone took 1.55 us a chunk against 0.6.
// Products: v_mfma_f32_32x32x16_bf16 (from registers alone, on random data:
// 1.82 PFLOP/s, 1.80 with four conversions beside each, 1.51 with eight vector
// instructions, two waves per SIMD).  Its operands take half the registers
// of the 16x16x32 shape's at the same tile, which spilled (4096 x 7168 x
// 7168: 525 us, 334 in this shape).
constexpr int kStages = 2;  // chunks in LDS (three: no difference, 288 x 7168 x 7168 54.8 and 54.9 us)

template <int RQ, int TT>
struct TileSmem {
    alignas(16) uint8_t a[kStages][RQ][8192];
    alignas(16) uint8_t b[kStages][TT][4096];
    struct {
        alignas(16) uint32_t a[RQ][kWave];
        alignas(16) uint32_t b[TT * 32];
    } s[kStages];  // the block scales
};

// this wave's loads but the newest N have landed and its LDS reads arrived;
// past the barrier, every wave's
template <int N>
__device__ inline void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int ACT, bool MX, int RQ, int TT, int WR, int WT>
__global__ void __launch_bounds__(WR * WT * kWave) linear_tile_kernel(moe_mxfp8_linear_args a, TileGrid p) {
    constexpr int kWaves = WR * WT;
    constexpr int Q = RQ / WR, NR = 2 * Q, NT = TT / WT;       // a wave's quads, 32-row and 32-token tiles
    constexpr int kA = RQ * 8 / kWaves, kB = TT * 4 / kWaves;  // 1 KB loads per wave and chunk
    constexpr int kS = (RQ + TT / 2) / kWaves;                 // and 256-byte loads of block scales
    static_assert(RQ * 8 % kWaves == 0 && TT * 4 % kWaves == 0 && (RQ + TT / 2) % kWaves == 0, "loads per wave");
    extern __shared__ uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<TileSmem<RQ, TT>*>(smem_raw);
    const int w = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, c = lane % 16;
    // Workgroups go round the eight XCDs; each XCD takes a run of the tiles,
    // numbered down bands of kBand token blocks, so that what its L2 holds of
    // x and W serves several tiles (1024 x 7168 x 7168: 103 us, 108 with the
    // tiles dealt round, 105 in bands of 2 or 8; 4096 x 7168 x 7168, bound by the
    // matrix cores: 318, 319 and 318)
    const int tiles = p.row_blocks * p.tok_blocks, per_xcd = (tiles + 7) / 8;
    const int split = blockIdx.x / (8 * per_xcd), blk = blockIdx.x % (8 * per_xcd);
    const int id = blk % 8 * per_xcd + blk / 8;
    if (id >= tiles) return;
    constexpr int kBand = 4;
    const int band = id / (kBand * p.row_blocks), in_band = id - band * kBand * p.row_blocks;
    const int height = min(kBand, p.tok_blocks - band * kBand);
    const int rb = in_band / height, tb = band * kBand + in_band % height;
    const int chunks = (int)(a.inner / 128), quads = (int)(a.rows / 64);
    const int k0 = split * p.split_chunks, k1 = min(chunks, k0 + p.split_chunks);
    const int q0 = rb * RQ;
    const int64_t t0 = (int64_t)tb * (32 * TT);
    const int last = (int)min((int64_t)(32 * TT), a.num_tokens - t0) - 1;  // rows past it repeat it

    // This wave's loads of a chunk: a scalar base that moves on by a fixed
    // step per chunk, and a 32-bit offset per lane (tokens relative to the
    // workgroup's first row).  Quads past the end repeat the last one.
    const uint8_t* baseA[kA];
    uint32_t offB[kB];
#pragma unroll
    for (int i = 0; i < kA; i++) {
        const int piece = w * kA + i;  // quad piece / 8, 1 KB piece % 8
        baseA[i] = a.w_tiles + ((int64_t)min(q0 + piece / 8, quads - 1) * chunks + k0) * 8192 + piece % 8 * 1024;
    }
#pragma unroll
    for (int i = 0; i < kB; i++) {
        const int row = (w * kB + i) * 8 + lane / 8;  // eight token rows per load
        offB[i] = (uint32_t)min(row, last) * (uint32_t)a.inner + ((lane % 8) ^ (row / 2 % 8)) * 16;
    }
    const uint8_t* baseB = a.x_codes + t0 * a.inner + (int64_t)k0 * 128;
    const uint8_t* baseS[kS];
    uint32_t offS[kS];
    int step_s[kS];
#pragma unroll
    for (int i = 0; i < kS; i++) {
        const int n = w * kS + i;
        if (n < RQ) {
            baseS[i] = a.w_scales + ((int64_t)min(q0 + n, quads - 1) * chunks + k0) * 256;
            offS[i] = lane * 4;
            step_s[i] = 256;
        } else {
            baseS[i] = a.x_scales + t0 * (a.inner / 32) + (int64_t)k0 * 4;
            offS[i] = (uint32_t)min((n - RQ) * kWave + lane, last) * (uint32_t)(a.inner / 32);
            step_s[i] = 4;
        }
    }
    const uint32_t lds = lds_addr(smem_raw);
    constexpr uint32_t kBufA = RQ * 8192, kBufB = TT * 4096, kBufS = (RQ * kWave + TT * 32) * 4;
    constexpr uint32_t kAtB = kStages * kBufA, kAtS = kAtB + kStages * kBufB;
    // load n of the kLoads of this wave's next chunk, into buffer buf
    constexpr int kLoads = kA + kB + kS;
    auto issue = [&](auto n, int buf) {
        constexpr int i = decltype(n)::value;
        if constexpr (i < kB) {
            dma16s(baseB, offB[i], lds + kAtB + buf * kBufB + (w * kB + i) * 1024);
            if constexpr (i == kB - 1) baseB += 128;
        } else if constexpr (i < kB + kA) {
            dma16s(baseA[i - kB], lane * 16, lds + buf * kBufA + (w * kA + i - kB) * 1024);
            baseA[i - kB] += 8192;
        } else {
            constexpr int j = i - kB - kA;
            dma4s(baseS[j], offS[j], lds + kAtS + buf * kBufS + (w * kS + j) * (kWave * 4));
            baseS[j] += step_s[j];
        }
    };
    const int wr = w % WR, wt = w / WR;
    f32x16_t acc[NR][NT];
#pragma unroll
    for (int i = 0; i < NR; i++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int j = 0; j < 16; j++) acc[i][t][j] = 0.f;
    // A chunk in eight steps z = 2 s + q of 16 k: lane (row l % 32, half = l / 32)
    // of an operand holds bytes 8 q .. 8 q + 7 of the 16-byte piece 2 s + half of its
    // row, of block s.  ar, br: the pieces of block s as they are in LDS, in
    // place s % 2, the next block's in the other; Ad, Bd: decoded, the row tile
    // of a product and the token tiles of a step, each beside the next one.
    const int r32 = lane % 32, half = lane / 32;
    const int a_at = lane / 16 % 2 * 2048 + half * 1024 + c * 16;  // block s is 256 s bytes on
    const int a_byte = lane / 16 % 2 * 8;                       // its group's place in a word of scales
    u32x4_t ar[2][NR], br[2][NT], Ad[2], Bd[2][NT];
    uint32_t sa[2][Q], sb[NT], sb_next[NT];  // scale words: A's of a block, B's of a chunk
    float a_scale[NR], b_scale[NT];          // of a block
    auto read_a = [&](int buf, auto s, auto i) {
        ar[s % 2][i] = *reinterpret_cast<const u32x4_t*>(&sm.a[buf][wr * Q + i / 2][a_at + i % 2 * 4096 + s * 256]);
        if constexpr (i % 2 == 0) sa[s % 2][i / 2] = sm.s[buf].a[wr * Q + i / 2][c + 16 * s];
    };
    auto read_b = [&](int buf, auto s, auto t) {
        const int row = (wt * NT + t) * 32 + r32;
        br[s % 2][t] = *reinterpret_cast<const u32x4_t*>(&sm.b[buf][0][row * 128 + ((2 * s + half) ^ (r32 / 2 % 8)) * 16]);
        if constexpr (s == 0) sb_next[t] = sm.s[buf].b[row];
    };
    auto pair = [&](const u32x4_t& raw, auto q, auto e, float scale) {  // elements 2e, 2e + 1 of the step's eight
        return __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * q.value + e.value / 2], scale, e.value % 2));
    };
    auto decode_a = [&](auto s, auto q, auto i, auto e) {
        if constexpr (q == 0 && e == 0)
            a_scale[i] = e8m0_as_scale((sa[s % 2][i / 2] >> (a_byte + i % 2 * 16)) & 0xffu);
        Ad[i % 2][e.value] = pair(ar[s % 2][i], q, e, a_scale[i]);
    };
    auto decode_b = [&](auto s, auto q, auto t, auto e) {
        if constexpr (s == 0 && q == 0 && e == 0) sb[t] = sb_next[t];
        if constexpr (q == 0 && e == 0) b_scale[t] = e8m0_as_scale((sb[t] >> (8 * s)) & 0xffu);
        Bd[q][t][e.value] = pair(br[s % 2][t], q, e, b_scale[t]);
    };
    const int n_chunks = k1 - k0;
    const std::integral_constant<int, 0> zero;
    static_for<kStages>([&](auto st) {
        if (st < n_chunks) static_for<kLoads>([&](auto n) { issue(n, st); });
    });
    // the first chunk's loads have landed (those of the others may be in flight)
    if (n_chunks >= kStages) wait_barrier<(kStages - 1) * kLoads>();
    else wait_barrier<0>();
    int buf = 0;
    auto next = [&] { return 1 - buf; };
    static_for<NT>([&](auto t) { read_b(0, zero, t); });
    static_for<NR>([&](auto i) { read_a(0, zero, i); });
    static_for<4 * NT>([&](auto n) {
        decode_b(zero, zero, std::integral_constant<int, n / 4>{}, std::integral_constant<int, n % 4>{});
    });
    static_for<4>([&](auto e) { decode_a(zero, zero, zero, e); });
    // One step: NR x NT products, and after each a part of what comes next, in
    // this order (the compiler keeps it): the next row tile is decoded, the
    // next step's token tiles, and in a block's first step the next block is
    // read.  At step 6 this wave has read all of the chunk (lgkmcnt) and its
    // loads of the next have landed (vmcnt); past the barrier that holds for
    // every wave, and the loads of the chunk after that, over this one, go out.
    constexpr int kSlots = NR * NT, kParts = 4 / NT;
    auto step = [&](auto z, auto read_next, auto load_next) {
        const std::integral_constant<int, z / 2> s;
        const std::integral_constant<int, z % 2> q;
        const std::integral_constant<int, (z + 1) % 8 / 2> s_next;  // of the next step
        const std::integral_constant<int, 1 - z % 2> q_next;
        constexpr bool more = z < 7 || decltype(read_next)::value, block = z < 6 || decltype(read_next)::value;
        if constexpr (z == 6 && decltype(read_next)::value) wait_barrier<0>();
        static_for<kSlots>([&](auto n) {
            constexpr int i = n / NT, t = n % NT;
            acc[i][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, Ad[i % 2]),
                                                                __builtin_bit_cast(bf16x8_t, Bd[q][t]), acc[i][t], 0, 0, 0);
            if constexpr (block && q == 0) {
                const std::integral_constant<int, (z / 2 + 1) % 4> ahead;
                const int from = z < 6 ? buf : next();
                if constexpr (t == 0) read_a(from, ahead, std::integral_constant<int, i>{});
                if constexpr (n < NT) read_b(from, ahead, n);
            }
            static_for<kParts>([&](auto j) {
                const std::integral_constant<int, t * kParts + j> e;
                if constexpr (i + 1 < NR) decode_a(s, q, std::integral_constant<int, i + 1>{}, e);
                else if constexpr (more) decode_a(s_next, q_next, zero, e);
            });
            if constexpr (more) {
                constexpr int lo = n * 4 * NT / kSlots, hi = (n + 1) * 4 * NT / kSlots;
                static_for<hi - lo>([&](auto j) {
                    decode_b(s_next, q_next, std::integral_constant<int, (lo + j) / 4>{},
                             std::integral_constant<int, (lo + j) % 4>{});
                });
            }
            if constexpr (z >= 6 && decltype(load_next)::value) {
                constexpr int at = (z - 6) * kSlots + n;
                constexpr int lo = at * kLoads / (2 * kSlots), hi = (at + 1) * kLoads / (2 * kSlots);
                static_for<hi - lo>([&](auto j) { issue(std::integral_constant<int, lo + j>{}, buf); });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    auto chunk = [&](auto read_next, auto load_next) {
        static_for<8>([&](auto z) { step(z, read_next, load_next); });
        buf = next();
    };
    int k = 0;
    for (; k + kStages < n_chunks; k++) chunk(std::true_type{}, std::true_type{});
    for (; k + 1 < n_chunks; k++) chunk(std::true_type{}, std::false_type{});  // nothing more to load
    chunk(std::false_type{}, std::false_type{});

    // The sums go through this wave's own part of the LDS, a token tile at
    // a time, to lanes that hold 8 consecutive columns of a token: rows of 16
    // lanes then read the residual and write the output in 256-byte runs.
    constexpr bool kGated = ACT == MOE_EPI_SILU_MUL;
    constexpr int kRow = 64 * Q + 4;                 // padded: 16-byte writes of 16 tokens cover all banks
    constexpr int kOcts = kGated ? 4 * Q : 8 * Q;    // output octets of a token
    constexpr int kItems = 32 * kOcts / kWave;       // per lane and token tile
    static_assert(sizeof(TileSmem<RQ, TT>) >= kWaves * 32 * kRow * 4, "staging of the sums");
    __syncthreads();  // every wave is done with the last chunk
    float(*mine)[kRow] = reinterpret_cast<float(*)[kRow]>(smem_raw + w * (32 * kRow * 4));
    const int64_t cols = kGated ? a.rows / 2 : a.rows;
    const int wq = q0 + wr * Q;                      // this wave's first quad
    const int64_t tw = t0 + wt * NT * 32;            // and first token
    auto stage = [&](auto t) {
#pragma unroll
        for (int i = 0; i < NR; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f32x16_t& v = acc[i][t];
                *reinterpret_cast<f32x4_t*>(&mine[r32][32 * i + 8 * j + 4 * half]) =
                    f32x4_t{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
            }
        __builtin_amdgcn_wave_barrier();
    };
    if (p.splits > 1) {
        static_for<NT>([&](auto t) {
            stage(t);
#pragma unroll 2
            for (int n = 0; n < 32 * 8 * Q / kWave; n++) {
                const int idx = n * kWave + lane, tok = idx / (8 * Q), o = idx % (8 * Q);
                float v[8] = {};
                add8(v, &mine[tok][8 * o]);
                if (tw + 32 * t + tok < a.num_tokens && wq + o / 8 < quads)
                    store_piece<8>(partial_of(a, split, tw + 32 * t + tok, (int64_t)wq * 64 + 8 * o), v);
            }
            __builtin_amdgcn_wave_barrier();
        });
        return;
    }
    const int o = lane % kOcts;
    const int64_t c0 = (int64_t)wq * (kGated ? 32 : 64) + 8 * o;
    const bool in = c0 < cols;
    float bias[8] = {}, bias_u[8] = {};
    if (a.bias && in) {
        add8(bias, a.bias + c0);
        if (kGated) add8(bias_u, a.bias + cols + c0);
    }
    static_for<NT>([&](auto t) {
        uint4 res[kItems];
#pragma unroll
        for (int n = 0; n < kItems; n++) {
            const int64_t tok = tw + 32 * t + n * (kWave / kOcts) + lane / kOcts;
            res[n] = make_uint4(0, 0, 0, 0);
            if (a.residual && in && tok < a.num_tokens) res[n] = residual8(a, tok, c0);
        }
        stage(t);
#pragma unroll
        for (int n = 0; n < kItems; n++) {
            const int row = n * (kWave / kOcts) + lane / kOcts;
            float v[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = bias[i], u[i] = bias_u[i];
            add8(v, &mine[row][kGated ? o / 4 * 64 + o % 4 * 8 : 8 * o]);
            if (kGated) add8(u, &mine[row][o / 4 * 64 + 32 + o % 4 * 8]);
            finish8(a, ACT, MX, cols, tw + 32 * t + row, c0, in && tw + 32 * t + row < a.num_tokens, v, u, res[n]);
        }
        __builtin_amdgcn_wave_barrier();
    });
}

// ------------------------------------------------------------ the launch
template <int G, int NT, int W>
hipError_t launch_rows(const moe_mxfp8_linear_args& a, const RowsGrid& p, hipStream_t stream) {
    const unsigned grid = (unsigned)(p.splits * 8 * p.groups * ((p.units + 7) / 8));
    linear_rows_kernel<G, NT, W, 2><<<grid, W * kWave, 0, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, bool MX, int RQ, int TT, int WR, int WT>
hipError_t launch_tile(const moe_mxfp8_linear_args& a, const TileGrid& p, hipStream_t stream) {
    constexpr int bytes = sizeof(TileSmem<RQ, TT>);  // more than 64 KB: has to be asked for
    const auto kernel = linear_tile_kernel<ACT, MX, RQ, TT, WR, WT>;
    const hipError_t err =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != hipSuccess) return err;
    const unsigned grid = (unsigned)((int64_t)p.splits * 8 * ((p.row_blocks * p.tok_blocks + 7) / 8));
    kernel<<<grid, WR * WT * kWave, bytes, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, bool MX>
hipError_t launch_tiles(const moe_mxfp8_linear_args& a, const LinearPlan& p, hipStream_t stream) {
    return p.wide ? launch_tile<ACT, MX, 4, 8, 2, 4>(a, p.tile, stream) : launch_tile<ACT, MX, 2, 4, 2, 2>(a, p.tile, stream);
}

}  // namespace

int64_t mxfp8_linear_workspace(int64_t T, int64_t rows, int64_t inner, int32_t activation) {
    if (T == 0) return 0;
    // either output may be asked for: MXFP8 splits wherever bf16 does
    const int splits = linear_plan(T, rows, inner, activation, true).splits;
    return splits > 1 ? splits * T * rows * 4 : 0;
}

hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream) {
    const bool mx = a.out_codes != nullptr;
    const LinearPlan p = linear_plan(a.num_tokens, a.rows, a.inner, a.activation, mx);
    const RowsGrid& r = p.grid;
    hipError_t err;
    if (!p.rows) {
        switch (p.splits > 1 ? MOE_EPI_NONE : a.activation) {  // a split leaves the epilogue to the finishing kernel
            case MOE_EPI_SILU: err = mx ? launch_tiles<MOE_EPI_SILU, true>(a, p, stream)
                                        : launch_tiles<MOE_EPI_SILU, false>(a, p, stream); break;
            case MOE_EPI_GELU: err = mx ? launch_tiles<MOE_EPI_GELU, true>(a, p, stream)
                                        : launch_tiles<MOE_EPI_GELU, false>(a, p, stream); break;
            case MOE_EPI_SILU_MUL: err = mx ? launch_tiles<MOE_EPI_SILU_MUL, true>(a, p, stream)
                                            : launch_tiles<MOE_EPI_SILU_MUL, false>(a, p, stream); break;
            default: err = mx && p.splits == 1 ? launch_tiles<MOE_EPI_NONE, true>(a, p, stream)
                                               : launch_tiles<MOE_EPI_NONE, false>(a, p, stream); break;
        }
    } else {
        switch (p.G * 10 + p.NT) {
            case 11: err = launch_rows<1, 1, 8>(a, r, stream); break;
            case 12: err = launch_rows<1, 2, 8>(a, r, stream); break;
            case 13: err = launch_rows<1, 3, 8>(a, r, stream); break;
            case 21: err = launch_rows<2, 1, 8>(a, r, stream); break;
            case 22: err = launch_rows<2, 2, 8>(a, r, stream); break;
            case 23: err = launch_rows<2, 3, 8>(a, r, stream); break;
            case 24: err = launch_rows<2, 4, 4>(a, r, stream); break;
            case 41: err = launch_rows<4, 1, 8>(a, r, stream); break;
            case 42: err = launch_rows<4, 2, 8>(a, r, stream); break;
            case 43: err = launch_rows<4, 3, 8>(a, r, stream); break;
            default: err = launch_rows<4, 4, 4>(a, r, stream); break;
        }
    }
    if (err != hipSuccess || p.splits == 1) return err;
    const int64_t octs = a.num_tokens * (a.activation == MOE_EPI_SILU_MUL ? a.rows / 2 : a.rows) / 8;
    linear_finish_kernel<<<(unsigned)((octs + 255) / 256), 256, 0, stream>>>(a, p.splits);
    return hipGetLastError();
}

}  // namespace moe
