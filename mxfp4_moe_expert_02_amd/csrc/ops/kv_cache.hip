// kv_cache.hip -- keys and values into the MXFP8 cache and out of it.
//
// Write: per block of 32 elements the scale 2^(floor(log2 amax) - 8), then each
// element to the nearest E4M3 value; the block's four lanes agree on amax
// through two quad exchanges.  Read: code * 2^scale.  Both move each byte
// once and have next to no arithmetic: memory bounds them, and with few tokens
// the launch (2.9 and 2.4 us).  16 bytes a thread in (write) or in and
// twice that out (read), whole cache lines a wave: 4096 tokens of 8 heads of
// 128 elements are written in 8.5 us (25 MB, 3.0 TB/s), 16001 read in 17.8 us
// (99 MB, 5.6 TB/s).
#include "attention_internal.h"

namespace moe {
namespace {

constexpr int kKvThreads = 256;

// Rows (tokens) and pieces of them to threads: a row of `pieces` pieces takes
// a workgroup of its own, or shares one where several fit.
struct KvGrid {
    int pieces, rows;  // pieces of a row, rows of a workgroup
};
inline KvGrid kv_grid(const moe_kv_rows_args& a, int piece) {
    KvGrid g;
    g.pieces = a.cache.kv_heads * a.cache.head_dim / piece;
    g.rows = g.pieces >= kKvThreads ? 1 : kKvThreads / g.pieces;
    return g;
}

// Where a slot's codes of head h are (its scales are at the 32nd part within
// the page), or no place
struct Place {
    int64_t page;
    int at;  // position in the page
    bool live;
};
__device__ inline Place place_of(const moe_kv_cache& c, int64_t slot) {
    const int shift = __builtin_ctz(c.page_size);
    Place p;
    p.page = slot >> shift;
    p.at = (int)(slot & (c.page_size - 1));
    p.live = slot >= 0 && p.page < c.num_pages;
    return p;
}

// blockIdx.y: 0 keys, 1 values
template <typename X>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(moe_kv_rows_args a, KvGrid g) {
    const bool val = blockIdx.y != 0;
    const int D = a.cache.head_dim;
    const int64_t t = (int64_t)blockIdx.x * g.rows + (g.rows > 1 ? threadIdx.x / g.pieces : 0);
    if (t >= a.num_tokens || (int)threadIdx.x >= g.rows * g.pieces) return;  // whole quads: a row is whole blocks of 32
    const X* x = val ? (const X*)a.v + t * a.v_stride : (const X*)a.k + t * a.k_stride;
    uint8_t* codes = val ? a.cache.v_codes : a.cache.k_codes;
    uint8_t* scales = val ? a.cache.v_scales : a.cache.k_scales;
    const Place p = place_of(a.cache, a.slots[t]);
    codes += p.page * a.cache.codes_page_stride;
    scales += p.page * a.cache.scales_page_stride;
    for (int i = g.rows > 1 ? threadIdx.x % g.pieces : threadIdx.x; i < g.pieces; i += kKvThreads) {
        float v[8];
        load_piece<8>(x + i * 8, v);  // (does not wait for the slot)
        if (!p.live) return;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));
        top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));
        const bool bad = top >= 0x7f800000u;  // a NaN or an infinity
        const int se = mxfp8_scale_exp(top);
        uint32_t code[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; e++) q[e] = bad ? 0.f : ldexpf(v[4 * h + e], -se);
            code[h] = e4m3_pack4(q);
        }
        const int h = i * 8 / D, d = i * 8 % D;
        const int at = (h * a.cache.page_size + p.at) * D + d;
        *reinterpret_cast<uint2*>(codes + at) = make_uint2(code[0], code[1]);
        if ((i & 3) == 0) scales[at / 32] = bad ? 255 : (uint8_t)(se + 127);
    }
}

// 16 codes as X, scale applied and rounded by the conversion (to nearest even)
__device__ inline void decode16(const uint4& c, float s, uint16_t* p) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, false));
        o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, true));
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}
__device__ inline void decode16(const uint4& c, float s, float* p) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], s, false);
        const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], s, true);
        reinterpret_cast<float4*>(p)[i] = make_float4(lo[0], lo[1], hi[0], hi[1]);
    }
}

template <typename X>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(moe_kv_rows_args a, KvGrid g) {
    const bool val = blockIdx.y != 0;
    const int D = a.cache.head_dim;
    const int64_t t = (int64_t)blockIdx.x * g.rows + (g.rows > 1 ? threadIdx.x / g.pieces : 0);
    if (t >= a.num_tokens || (int)threadIdx.x >= g.rows * g.pieces) return;
    X* x = val ? (X*)a.v + t * a.v_stride : (X*)a.k + t * a.k_stride;
    const uint8_t* codes = val ? a.cache.v_codes : a.cache.k_codes;
    const uint8_t* scales = val ? a.cache.v_scales : a.cache.k_scales;
    const Place p = place_of(a.cache, a.slots[t]);
    if (p.live) {
        codes += p.page * a.cache.codes_page_stride;
        scales += p.page * a.cache.scales_page_stride;
    }
    for (int i = g.rows > 1 ? threadIdx.x % g.pieces : threadIdx.x; i < g.pieces; i += kKvThreads) {
        const int h = i * 16 / D, d = i * 16 % D;
        const int at = (h * a.cache.page_size + p.at) * D + d;
        uint4 c = make_uint4(0, 0, 0, 0);
        uint32_t s = 127;
        if (p.live) {
            c = *reinterpret_cast<const uint4*>(codes + at);
            s = scales[at / 32];
        }
        decode16(c, e8m0_as_scale(s), x + i * 16);
    }
}

unsigned blocks(int64_t rows, const KvGrid& g) { return (unsigned)((rows + g.rows - 1) / g.rows); }

}  // namespace

hipError_t launch_kv_write(const moe_kv_rows_args& a, hipStream_t stream) {
    const KvGrid g = kv_grid(a, 8);
    const dim3 grid(blocks(a.num_tokens, g), 2);
    if (a.dtype == MOE_DT_BF16) kv_write_kernel<uint16_t><<<grid, kKvThreads, 0, stream>>>(a, g);
    else kv_write_kernel<float><<<grid, kKvThreads, 0, stream>>>(a, g);
    return hipGetLastError();
}

hipError_t launch_kv_read(const moe_kv_rows_args& a, hipStream_t stream) {
    const KvGrid g = kv_grid(a, 16);
    const dim3 grid(blocks(a.num_tokens, g), 2);
    if (a.dtype == MOE_DT_BF16) kv_read_kernel<uint16_t><<<grid, kKvThreads, 0, stream>>>(a, g);
    else kv_read_kernel<float><<<grid, kKvThreads, 0, stream>>>(a, g);
    return hipGetLastError();
}

}  // namespace moe
