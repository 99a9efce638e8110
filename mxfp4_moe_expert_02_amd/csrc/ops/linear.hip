// linear.hip -- out = act(x W^T + bias) + residual with x and W in MXFP8.
//
// The weights come in the MXFP8 tile layout of moe_mxfp8_prepack (prepack.hip):
// per 64-row quad and 128-k chunk 8 KB of codes [group][half][lane][16] and
// 256 scale bytes [lane][group], lane (r, g) = (l % 16, l / 16) holding block
// g (k = 32g .. 32g+31) of row r.
//
// Few tokens (linear_rows_kernel): the weights' bytes bound the call.  Both
// operands are decoded to bf16 (exact: E4M3 has four significant bits, the
// block scale is a power of two) and multiplied on the bf16 matrix cores,
// whose products and sums are exact to float32; the FP8 matrix cores drop
// bits below about 2^-16 of the largest product of a group (measured: 1.4e-5
// of the sum's rms against 4e-8), and at these sizes their rate is not
// needed.  9 x 6144 x 6144 10.5 us (39 MB, 3.7 TB/s), 72 x 4096 x 7168 16.9.
// Many tokens (linear_tile_kernel): the FP8 matrix cores, tiles of up to
// 256 x 256 staged through LDS.  4096 x 7168 x 7168 with bias and residual 200
// us (2.1 PFLOP/s; weights and tokens from the caches 177), where the matrix
// cores are busy 56 % of the time and their clock falls with random operands;
// 288 x 7168 x 7168 34 us; 1001 x 2048 x 6144 27 us, 6 of them the pass over
// the split sums.
// Either may split the inner axis over workgroups that leave float32 sums in
// the workspace for linear_finish_kernel.
#include "lds_dma.h"
#include "ops_internal.h"

namespace moe {
namespace {

__device__ inline i32x8_t operand(const uint4& lo, const uint4& hi) {
    return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// v / (1 + exp(-v)); the hardware exponential and reciprocal (about 1 ulp each)
__device__ inline float silu(float v) { return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

// v / 2 * (1 + erf(v / sqrt 2)) = v / 2 * erfc(-v / sqrt 2): erfc keeps the
// relative precision of the left tail that 1 + erf loses.  For a >= 0,
// erfc(a) = t exp(-a^2) f(t) with t = 1 / (1 + 0.4 a); f is a least-squares
// polynomial for f(t) = erfc(a) exp(a^2) / t, weighted towards the smallest
// largest relative error (2e-8, with float32 roundings 1.5e-7).
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

struct RowsGrid {
    int units, groups;          // weight units (rows / 16G), token groups of NT tiles
    int splits, split_chunks;   // parts of the inner axis, chunks of one
};

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
        // In the steady loop every load is unconditional (a skipped one makes
        // the compiler wait for all); the last chunks have none to skip.
        int i = 0;
        for (; i + 2 * D <= n; i += D)
            static_for<D>([&](auto d) {
                // this chunk has landed, the next D - 1 may be in flight
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
// Products: v_mfma_scale_f32_16x16x128_f8f6f4, lane (r, g) of an operand
// holding the 16-byte pieces g and g + 4 of row r's 128 bytes and the scale of
// block g (from registers alone, on random data: 3.79 PFLOP/s; the 32x32x64
// shape, whose clock falls further, 3.28).
template <int RQ, int TT, int STAGES>
struct TileSmem {
    alignas(16) uint8_t a[STAGES][RQ][8192];
    alignas(16) uint8_t b[STAGES][TT][4096];
    struct {
        alignas(16) uint32_t a[RQ][kWave];
        alignas(16) uint32_t b[TT * 32];
    } s[STAGES];  // the block scales
};

struct TileGrid {
    int row_blocks, tok_blocks;
    int splits, split_chunks;
};

// this wave's loads but the newest N have landed and its LDS reads arrived;
// past the barrier, every wave's
template <int N>
__device__ inline void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Two waves per SIMD: with registers for one only the compiler keeps the sums
// of 256 threads in accumulation registers and copies them around the second
// phase (288 x 7168 x 7168: 39.2 us, 35.4 without).
template <int ACT, bool MX, int RQ, int TT, int WR, int WT, int STAGES>
__global__ void __launch_bounds__(WR * WT * kWave, 2) linear_tile_kernel(moe_mxfp8_linear_args a, TileGrid p) {
    constexpr int kStages = STAGES, kWaves = WR * WT;
    constexpr int Q = RQ / WR, NT = TT * 2 / WT;               // a wave's quads and 16-token tiles
    constexpr int NG = 4 * Q;                                  // and 16-row groups
    constexpr int kA = RQ * 8 / kWaves, kB = TT * 4 / kWaves;  // 1 KB loads per wave and chunk
    constexpr int kS = (RQ + TT / 2) / kWaves;                 // and 256-byte loads of block scales
    static_assert(RQ * 8 % kWaves == 0 && TT * 4 % kWaves == 0 && (RQ + TT / 2) % kWaves == 0, "loads per wave");
    extern __shared__ uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<TileSmem<RQ, TT, kStages>*>(smem_raw);
    const int w = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
    // Workgroups go round the eight XCDs; each XCD takes a run of the tiles,
    // numbered down bands of kBand token blocks, so that what its L2 holds of
    // x and W serves several tiles (4096 x 7168 x 7168 from HBM: 206 us with
    // the tiles dealt round, 200 with bands of 4, 203 of 2, 201 of 8)
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
    f32x4_t acc[NG][NT];
#pragma unroll
    for (int i = 0; i < NG; i++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int a_at = (g & 1) * 1024 + (c + 16 * (g >> 1)) * 16;  // piece g; piece g + 4 is 512 bytes on
    const int b_at = c * 128 + (g ^ (c / 2)) * 16;               // piece g; piece g + 4 is in slot ^ 4
    i32x8_t A[NG], B[NT];
    uint32_t sa[Q], sb[NT], sa_first = 0;  // sa_first: the next chunk's sa[0]
    auto read_a = [&](int buf, auto i) {
        const uint8_t* p = &sm.a[buf][wr * Q + i / 4][a_at + i % 4 * 2048];
        A[i] = operand(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 512));
        if constexpr (i % 4 == 0) {
            const uint32_t v = sm.s[buf].a[wr * Q + i / 4][lane];
            if constexpr (i == 0) sa_first = v;
            else sa[i / 4] = v;
        }
    };
    auto read_b = [&](int buf, auto t) {
        const int row = (wt * NT + t) * 16;
        const uint8_t* p = &sm.b[buf][0][row * 128];
        B[t] = operand(*reinterpret_cast<const uint4*>(p + b_at), *reinterpret_cast<const uint4*>(p + (b_at ^ 64)));
        sb[t] = reinterpret_cast<const uint8_t*>(&sm.s[buf].b[row + c])[g];
    };
    // one product, after which also() goes out; the compiler keeps that order
    auto product = [&](auto i, auto t, auto&& also) {
        acc[i][t] = mfma_scaled<0, decltype(i)::value % 4, 0>(A[i], B[t], acc[i][t], sa[i / 4], sb[t]);
        also();
        __builtin_amdgcn_sched_barrier(0);
    };
    // step n of `of` of something done in `count` parts
    auto part = [&](auto n, auto of, auto count, auto&& f) {
        constexpr int lo = decltype(n)::value * decltype(count)::value / decltype(of)::value;
        constexpr int hi = (decltype(n)::value + 1) * decltype(count)::value / decltype(of)::value;
        static_for<hi - lo>([&](auto j) { f(std::integral_constant<int, lo + decltype(j)::value>{}); });
    };
    // A chunk in two phases.  First the groups up to kFirst, one after the
    // other, while the rest of A is read, a group a product; then this wave
    // has read all of the chunk (lgkmcnt) and its loads of the next have
    // landed (vmcnt), and past the barrier that holds for every wave.  Then
    // the last groups, tile by tile: a tile of B done, its registers take the
    // next chunk's, whose first kAheadA groups of A are read and the loads of the
    // chunk kStages on (over this one) go out meanwhile.  A short first phase
    // leaves B's reads more time (4 groups: 34.3 us with 1, 35.8 with 2, 37.0
    // with 3, 288 x 7168 x 7168), a long one A's (8 groups: 200 us with 5, 201
    // with 4, 208 with 3, 4096 x 7168 x 7168).
    constexpr int kFirst = NG == 8 ? 5 : 1, kAheadA = NG == 8 ? 3 : 2, kLast = NG - kFirst;
    const std::integral_constant<int, kLast * NT> in_second;
    const std::integral_constant<int, kLoads> loads;
    const std::integral_constant<int, kAheadA> ahead;
    const int n_chunks = k1 - k0;
    static_for<kStages>([&](auto st) {
        if (st < n_chunks) static_for<kLoads>([&](auto n) { issue(n, st); });
    });
    // the first chunk's loads have landed (those of the others may be in flight)
    if (n_chunks >= kStages) wait_barrier<(kStages - 1) * kLoads>();
    else wait_barrier<0>();
    static_for<NT>([&](auto t) { read_b(0, t); });
    static_for<kAheadA>([&](auto i) { read_a(0, i); });
    int buf = 0;
    auto next = [&] { return buf + 1 == kStages ? 0 : buf + 1; };
    auto first_phase = [&] {
        sa[0] = sa_first;
        static_for<kFirst>([&](auto i) {
            static_for<NT>([&](auto t) {
                product(i, t, [&] {
                    constexpr int next_a = decltype(i)::value * NT + decltype(t)::value + kAheadA;
                    if constexpr (next_a < NG) read_a(buf, std::integral_constant<int, next_a>{});
                });
            });
        });
    };
    auto second_phase = [&](auto read_next, auto load_next) {
        static_for<NT>([&](auto t) {
            static_for<kLast>([&](auto j) {
                constexpr int n = decltype(t)::value * kLast + decltype(j)::value;
                product(std::integral_constant<int, kFirst + decltype(j)::value>{}, t, [&] {
                    const std::integral_constant<int, n> at;
                    if constexpr (decltype(load_next)::value)
                        part(at, in_second, loads, [&](auto u) { issue(u, buf); });
                    if constexpr (decltype(read_next)::value) {
                        part(at, in_second, ahead, [&](auto u) { read_a(next(), u); });
                        if constexpr (j == kLast - 1) read_b(next(), t);
                    }
                });
            });
        });
    };
    int k = 0;
    for (; k + kStages < n_chunks; k++) {
        first_phase();
        wait_barrier<(kStages - 2) * kLoads>();
        second_phase(std::true_type{}, std::true_type{});
        buf = next();
    }
    for (; k + 1 < n_chunks; k++) {  // nothing more to load
        first_phase();
        wait_barrier<0>();
        second_phase(std::true_type{}, std::false_type{});
        buf = next();
    }
    first_phase();
    second_phase(std::false_type{}, std::false_type{});

    // The sums go through this wave's own part of the LDS, two token tiles at
    // a time, to lanes that hold 8 consecutive columns of a token: rows of 16
    // lanes then read the residual and write the output in 256-byte runs.
    constexpr bool kGated = ACT == MOE_EPI_SILU_MUL;
    constexpr int kRow = 64 * Q + 4;                 // padded: 16-byte writes of 16 tokens cover all banks
    constexpr int kOcts = kGated ? 4 * Q : 8 * Q;    // output octets of a token
    constexpr int kItems = 32 * kOcts / kWave;       // per lane and token tile
    static_assert(sizeof(TileSmem<RQ, TT, kStages>) >= kWaves * 32 * kRow * 4, "staging of the sums");
    __syncthreads();  // every wave is done with the last chunk
    float(*mine)[kRow] = reinterpret_cast<float(*)[kRow]>(smem_raw + w * (32 * kRow * 4));
    const int64_t cols = kGated ? a.rows / 2 : a.rows;
    const int wq = q0 + wr * Q;                      // this wave's first quad
    const int64_t tw = t0 + wt * NT * 16;            // and first token
    auto stage = [&](auto t) {  // token tiles 2t, 2t + 1
#pragma unroll
        for (int half = 0; half < 2; half++)
#pragma unroll
            for (int i = 0; i < NG; i++)
                *reinterpret_cast<f32x4_t*>(&mine[16 * half + c][16 * i + 4 * g]) = acc[i][2 * t + half];
        __builtin_amdgcn_wave_barrier();
    };
    if (p.splits > 1) {
        static_for<NT / 2>([&](auto t) {
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
    static_for<NT / 2>([&](auto t) {
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

// ------------------------------------------------------------ the choice
// Tokens of linear_rows_kernel: at 128 it is exact at about the tiles' speed
// (128 x 4096 x 7168: 17.9 us, tiles 19.2; 128 x 7168 x 7168: 24.7 and 22.1).
constexpr int kRowsMaxTok = 128, kRowsMostTok = 1024;
constexpr int64_t kRowsMostWork = (int64_t)256 * 6144;  // workgroups times inner axis
constexpr int kWideTiles = 160;    // from as many on 256 x 256 tiles
constexpr int kMaxSplits = 8;
constexpr int kSplitTok = 8192;    // most tokens times splits (the workspace's bound)
constexpr int kCus = 256;

struct LinearPlan {
    bool rows;       // linear_rows_kernel
    int G, NT, W;
    RowsGrid grid;
    bool wide;       // 256 x 256 tiles (else 128 x 128)
    bool deep;       // 128 x 128 tiles staged three chunks deep (else two)
    TileGrid tile;
    int splits;
};

LinearPlan make_plan(int64_t T, int64_t rows, int64_t inner, int32_t activation, bool mx) {
    LinearPlan p{};
    const int tiles = (int)((T + 15) / 16), chunks = (int)(inner / 128);
    const bool gated = activation == MOE_EPI_SILU_MUL;
    // linear_rows_kernel: few tokens, and more where its largest workgroups (64 rows x 64 tokens)
    // all run at once and the work is small, so that the tiles' launches of few
    // workgroups would mostly wait (320 x 2048 x 2048: 8.2 us, tiles 13.6; 1024
    // x 1024 x 1024: 8.0 and 10.6; 192 x 4096 x 7168: 19.4 and 20.0; past the
    // bound 1024 x 1024 x 8192: 26.9 and 23.4)
    const int64_t most = rows / 64 * ((T + 63) / 64);
    p.rows = T <= kRowsMaxTok || (T <= kRowsMostTok && most <= kCus && most * inner <= kRowsMostWork);
    int64_t splits = 1;
    if (!p.rows) {
        // 256 x 256 tiles move half the bytes per product, 128 x 128 leave fewer
        // CUs idle (1536 x 7168 x 7168: 168 wide tiles 86 us, narrow ones 106;
        // 1024 x 7168 x 7168: 112 wide tiles 82 us, narrow ones 66)
        const int64_t wide_blocks = (rows + 255) / 256 * ((T + 255) / 256);
        p.wide = wide_blocks >= kWideTiles;
        const int n = p.wide ? 256 : 128;
        p.tile.row_blocks = (int)((rows + n - 1) / n);
        p.tile.tok_blocks = (int)((T + n - 1) / n);
        // A 128-k chunk of a workgroup takes about 0.5 us, the pass over the
        // split sums 2 us and 0.5 us per MB of them; the number of splits that
        // leaves the least, of those that fit on the CUs (1024 x 2048 x 6144:
        // 28.6 us in 2, 30.8 in 1; x 2048: 23.2 and 14.6).
        const int64_t blocks = (int64_t)p.tile.row_blocks * p.tile.tok_blocks;
        const int64_t sums = T * rows * 4 / 1000000;  // MB
        int64_t best = chunks;                        // in units of 0.5 us
        for (int64_t n = 2; !p.wide && n <= kMaxSplits && n * blocks <= kCus && n * T <= kSplitTok; n++) {
            const int64_t t = (chunks + n - 1) / n + 4 + n * sums;
            if (t < best) best = t, splits = n;
        }
    } else {
        // Of the tile shapes, the one whose workgroups come closest to one
        // per CU from below: fewer leave CUs idle, more take a second round
        // (and read the tokens or the weights more often).  Measured on 30
        // shapes of 9 to 128 tokens; e.g. 24 x 7168 x 7168: 224 workgroups
        // 15.3 us, 448 17.6, 112 19.3; 96 x 4096 x 7168: 256 15.1, 192 16.4,
        // 384 18.9.  Equal counts: the smaller tile.
        int64_t best = 0;
        for (int G = mx && gated ? 4 : mx || gated ? 2 : 1; G <= 4; G *= 2)
            for (int NT = 1; NT <= 4; NT++) {
                if (NT > tiles || (NT == 4 && G == 1)) continue;
                const int64_t n = rows / (16 * G) * ((tiles + NT - 1) / NT);
                const bool fits = n <= kCus, best_fits = best <= kCus;
                if (best && (fits != best_fits ? best_fits : fits ? n < best : n > best)) continue;
                if (best == n && G * NT >= p.G * p.NT) continue;
                best = n;
                p.G = G;
                p.NT = NT;
            }
        p.W = p.NT == 4 ? 4 : 8;  // what the staged tokens leave room for
        p.grid.groups = (tiles + p.NT - 1) / p.NT;
        // MXFP8 output needs whole blocks of columns in a workgroup; where
        // that leaves few of them the inner axis is split (9 x 4096 x 6144
        // gated: 64 workgroups 13.2 us, 4 times as many 11.1)
        if (mx && best <= kCus / 4) splits = 4;
    }
    if (splits > chunks / 8) splits = chunks / 8;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < 1) splits = 1;
    // 128 x 128 tiles: up to one workgroup per CU the loads of two chunks
    // are kept in flight (three stages, 101 KB of LDS); beyond that two
    // workgroups per CU hide each other's waits (two stages).  512 x 4096 x
    // 7168: 256 workgroups 31.6 us deep, 34.4 otherwise; 1024 x 7168 x 7168:
    // 448 workgroups 76.7 deep, 66.3 otherwise.
    p.deep = !p.rows && !p.wide && (int64_t)p.tile.row_blocks * p.tile.tok_blocks * splits <= kCus;
    const int per = (int)((chunks + splits - 1) / splits);
    p.splits = (chunks + per - 1) / per;
    p.grid.splits = p.tile.splits = p.splits;
    p.grid.split_chunks = p.tile.split_chunks = per;
    if (p.rows) p.grid.units = (int)(rows / (16 * p.G));
    return p;
}

template <int G, int NT, int W>
hipError_t launch_rows(const moe_mxfp8_linear_args& a, const RowsGrid& p, hipStream_t stream) {
    const unsigned grid = (unsigned)(p.splits * 8 * p.groups * ((p.units + 7) / 8));
    linear_rows_kernel<G, NT, W, 2><<<grid, W * kWave, 0, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, bool MX, int RQ, int TT, int WR, int WT, int STAGES>
hipError_t launch_tile(const moe_mxfp8_linear_args& a, const TileGrid& p, hipStream_t stream) {
    constexpr int bytes = sizeof(TileSmem<RQ, TT, STAGES>);  // more than 64 KB: has to be asked for
    const auto kernel = linear_tile_kernel<ACT, MX, RQ, TT, WR, WT, STAGES>;
    const hipError_t err =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != hipSuccess) return err;
    const unsigned grid = (unsigned)((int64_t)p.splits * 8 * ((p.row_blocks * p.tok_blocks + 7) / 8));
    kernel<<<grid, WR * WT * kWave, bytes, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, bool MX>
hipError_t launch_tiles(const moe_mxfp8_linear_args& a, const LinearPlan& p, hipStream_t stream) {
    if (p.wide) return launch_tile<ACT, MX, 4, 8, 2, 4, 2>(a, p.tile, stream);
    return p.deep ? launch_tile<ACT, MX, 2, 4, 2, 2, 3>(a, p.tile, stream)
                  : launch_tile<ACT, MX, 2, 4, 2, 2, 2>(a, p.tile, stream);
}

}  // namespace

int64_t mxfp8_linear_workspace(int64_t T, int64_t rows, int64_t inner, int32_t activation) {
    if (T == 0) return 0;
    // either output may be asked for: MXFP8 splits wherever bf16 does
    const int splits = make_plan(T, rows, inner, activation, true).splits;
    return splits > 1 ? splits * T * rows * 4 : 0;
}

hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream) {
    const bool mx = a.out_codes != nullptr;
    const LinearPlan p = make_plan(a.num_tokens, a.rows, a.inner, a.activation, mx);
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
