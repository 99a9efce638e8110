// rmsnorm.hip -- residual addition, RMS norm and MXFP8 encoding in one pass.
//
//   s = x + residual,  n = s * weight / sqrt(mean(s^2) + eps)
//
// One workgroup owns a row and holds it in registers: every thread loads
// its pieces of 8 elements (16 bytes of bf16), adds the residual, writes
// the sum back, squares it into the row's sum (one cross-lane and one LDS
// reduction), and then scales and encodes what it still holds.  A row is
// read once and written once; the kernel is bound by those bytes: 4096 x 7168
// with a residual and both outputs 59.5 us, 4.5 TB/s (a copy moves 5.0 to 5.5);
// 288 x 6144 7.5 us and one row 5.9, where the loads' and the launch's latency
// is the time.
//
// Everything between the loads and the roundings is in 64 bits, where the
// vector ALU of gfx950 runs as many multiply-adds per clock as in (unpacked)
// 32: about 16 operations per element.  The 8-bit codes are a decision on n,
// and a float32 n takes it differently about once per million elements;
// here the codes are the formula's.
#include "ops_internal.h"

namespace moe {
namespace {

// v's value of the lane that CTRL (a DPP control) names
template <int CTRL>
__device__ inline double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ inline double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// sum over the wave, the same in every lane (every lane takes part)
__device__ inline double wave_sum(double v) {
    v += dpp<0xB1>(v);   // lanes 1, 0, 3, 2 of a quad
    v += dpp<0x4E>(v);   // lanes 2, 3, 0, 1
    v += dpp<0x141>(v);  // half a row mirrored: the other quad of 8
    v += dpp<0x140>(v);  // a row mirrored: the other 8 of 16
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// 1 / sqrt(m) for m >= 0: the hardware's estimate and two Newton steps (to
// about 2^-52); 0 for infinity, as the quotient by sqrt(m) would give
__device__ inline double rsqrt_full(double m) {
    double r = __builtin_amdgcn_rsq(m);
    r = r * fma(-0.5 * m * r, r, 1.5);
    r = r * fma(-0.5 * m * r, r, 1.5);
    return m == __builtin_inf() ? 0.0 : r;
}

// v with its low word folded into the last bit of the high one (set if any
// low bit is): 21 significant bits that a later rounding to 8 bits takes
// for the whole value, exact in float32 over float32's range.
__device__ inline double sticky(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t hi = (uint32_t)(b >> 32) | (uint32_t)((uint32_t)b != 0);
    return __builtin_bit_cast(double, (uint64_t)hi << 32);
}

constexpr int kNormPiece = 8;

// double -> the float32 whose rounding to bf16 is the double's: the sticky
// form holds every bit that matters, and float32's rounding to bf16 sees a tie
// only where there is one.  Below float32's normal range its steps (2^-149)
// lose the sticky bit: there v is rounded to bf16's subnormals (steps of
// 2^-133) in 64 bits.
__device__ inline void round_once(const double (&v)[kNormPiece], float (&o)[kNormPiece]) {
    bool small = false;
#pragma unroll
    for (int e = 0; e < kNormPiece; e++) {
        o[e] = (float)sticky(v[e]);
        small |= fabsf(o[e]) < 0x1p-126f;
    }
    if (small)
#pragma unroll
        for (int e = 0; e < kNormPiece; e++)
            if (fabs(v[e]) < 0x1p-126) o[e] = (float)(rint(v[e] * 0x1p133) * 0x1p-133);
}

// WPR: waves per row, 1 (four rows per workgroup of 256 threads) or more
// (one row per workgroup); NP: pieces of 8 elements per thread.
template <typename X, typename R, int WPR, int NP>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR)
rmsnorm_kernel(moe_rmsnorm_args a) {
    constexpr int kThreads = 64 * WPR;  // of a row
    __shared__ double part[WPR];
    const int tid = WPR == 1 ? threadIdx.x % 64 : threadIdx.x;
    const int64_t t = WPR == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : (int64_t)blockIdx.x;
    if (t >= a.num_tokens) return;  // WPR == 1 only: whole waves, no barrier below
    const int H = (int)a.hidden, pieces = H / kNormPiece;
    const X* x = (const X*)a.x + t * a.x_stride;
    const R* r = a.residual ? (const R*)a.residual + t * a.residual_stride : nullptr;
    R* ro = a.residual_out ? (R*)a.residual_out + t * a.residual_out_stride : nullptr;
    // every load of the row is issued before the first store (the outputs may
    // be the inputs, so the compiler keeps loads behind stores)
    float xv[NP][kNormPiece], rv[NP][kNormPiece], wv[NP][kNormPiece];
#pragma unroll
    for (int p = 0; p < NP; p++) {
        const int i = p * kThreads + tid;
#pragma unroll
        for (int e = 0; e < kNormPiece; e++) xv[p][e] = rv[p][e] = wv[p][e] = 0.f;
        if (i < pieces) {
            load_piece<kNormPiece>(x + i * kNormPiece, xv[p]);
            if (r) load_piece<kNormPiece>(r + i * kNormPiece, rv[p]);
            if (a.weight_dtype == MOE_DT_F32)
                load_piece<kNormPiece>((const float*)a.weight + i * kNormPiece, wv[p]);
            else
                load_piece<kNormPiece>((const uint16_t*)a.weight + i * kNormPiece, wv[p]);
        }
    }
    double s[NP][kNormPiece];
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < NP; p++)
#pragma unroll
        for (int e = 0; e < kNormPiece; e++) {
            s[p][e] = r ? (double)xv[p][e] + (double)rv[p][e] : (double)xv[p][e];
            sum = fma(s[p][e], s[p][e], sum);
        }
    if (ro) {
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const int i = p * kThreads + tid;
            float o[kNormPiece];
            // s is a whole multiple of 2^-149: float32's below its normal range
#pragma unroll
            for (int e = 0; e < kNormPiece; e++) o[e] = (float)(sizeof(R) == 2 ? sticky(s[p][e]) : s[p][e]);
            if (i < pieces) store_piece<kNormPiece>(ro + i * kNormPiece, o);
        }
    }
    sum = wave_sum(sum);
    if constexpr (WPR > 1) {
        if (tid % kWave == 0) part[tid / kWave] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < WPR; w++) sum += part[w];
    }
    const double rinv = rsqrt_full(sum / H + a.eps);
    uint16_t* y = a.y ? (uint16_t*)a.y + t * a.y_stride : nullptr;
#pragma unroll
    for (int p = 0; p < NP; p++) {
        const int i = p * kThreads + tid;
        const bool live = i < pieces;
        double n[kNormPiece];
#pragma unroll
        for (int e = 0; e < kNormPiece; e++) n[e] = s[p][e] * (double)wv[p][e] * rinv;
        if (y && live) {
            float o[kNormPiece];
            round_once(n, o);
            store_piece<kNormPiece>(y + i * kNormPiece, o);
        }
        if (!a.codes) continue;
        // a block of 32 lies in four neighbouring lanes, which agree on its
        // largest exponent (the high words order like the magnitudes)
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kNormPiece; e++) {
            const uint32_t hi = (uint32_t)(__builtin_bit_cast(uint64_t, n[e]) >> 32) & 0x7fffffffu;
            top = hi > top ? hi : top;
        }
        top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));
        top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));
        if (!live) continue;
        const bool bad = top >= 0x7ff00000u;  // a NaN or an infinity
        int se = (int)(top >> 20) - 1023 - 8;  // a zero or subnormal block: below -127
        se = se < -127 ? -127 : (se > 127 ? 127 : se);
        uint32_t code[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; e++) q[e] = bad ? 0.f : (float)sticky(ldexp(n[4 * h + e], -se));
            code[h] = e4m3_pack4(q);
        }
        *reinterpret_cast<uint2*>(a.codes + t * H + i * kNormPiece) = make_uint2(code[0], code[1]);
        if ((i & 3) == 0) a.scales[t * (H / 32) + i / 4] = bad ? 255 : (uint8_t)(se + 127);
    }
}

template <typename X, typename R>
hipError_t launch_typed(const moe_rmsnorm_args& a, hipStream_t stream) {
    const int pieces = (int)(a.hidden / kNormPiece);
    const unsigned T = (unsigned)a.num_tokens;
    // Waves per row: one piece per thread up to 4096 columns, two beyond (4096
    // rows of 4096: 8 waves 28 us, 4 waves 30, 16 waves 37; of 7168: 8 x 2
    // pieces 59, 16 x 1 61, 4 x 4 70; 2048 of 16384: 16 x 2 81, 8 x 4 91)
    if (pieces <= 64) rmsnorm_kernel<X, R, 1, 1><<<(T + 3) / 4, 256, 0, stream>>>(a);
    else if (pieces <= 128) rmsnorm_kernel<X, R, 2, 1><<<T, 128, 0, stream>>>(a);
    else if (pieces <= 256) rmsnorm_kernel<X, R, 4, 1><<<T, 256, 0, stream>>>(a);
    else if (pieces <= 512) rmsnorm_kernel<X, R, 8, 1><<<T, 512, 0, stream>>>(a);
    else if (pieces <= 1024) rmsnorm_kernel<X, R, 8, 2><<<T, 512, 0, stream>>>(a);
    else rmsnorm_kernel<X, R, 16, 2><<<T, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const moe_rmsnorm_args& a, hipStream_t stream) {
    const bool xb = a.x_dtype == MOE_DT_BF16, rb = !a.residual || a.residual_dtype == MOE_DT_BF16;
    if (xb) return rb ? launch_typed<uint16_t, uint16_t>(a, stream) : launch_typed<uint16_t, float>(a, stream);
    return rb ? launch_typed<float, uint16_t>(a, stream) : launch_typed<float, float>(a, stream);
}

}  // namespace moe
