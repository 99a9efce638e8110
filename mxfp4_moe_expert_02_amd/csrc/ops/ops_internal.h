// ops_internal.h -- declarations shared by the operators around the expert
// layer (include/ops/moe_ops.h).  Not part of the C ABI.
#pragma once

#include "../../../include/ops/moe_ops.h"
#include "../device_common.h"

namespace moe {

// The launchers take arguments that moe_ops.h's checks have passed, with
// every stride filled in (never 0), and return the hipError_t of the launch.
hipError_t launch_rmsnorm(const moe_rmsnorm_args& a, hipStream_t stream);
hipError_t launch_mxfp8_linear(const moe_mxfp8_linear_args& a, hipStream_t stream);
int64_t mxfp8_linear_workspace(int64_t T, int64_t rows, int64_t inner, int32_t activation);
hipError_t launch_dispatch(const moe_dispatch_args& a, hipStream_t stream);
int64_t dispatch_workspace(int64_t T, int64_t E, int32_t k);
hipError_t launch_ops_combine(const moe_combine_args& a, hipStream_t stream);
hipError_t launch_ops_combine_backward(const moe_combine_args& a, hipStream_t stream);

// N consecutive elements of a bf16 (uint16_t) or float32 row as float32,
// and back (bf16: nearest even).  N > 1 needs 16-byte aligned pieces.
template <int N>
__device__ inline void load_piece(const uint16_t* p, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = bf16_to_f32(*p);
    } else if constexpr (N == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        static_assert(N == 8, "pieces are 1, 4 or 8 elements");
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <int N>
__device__ inline void load_piece(const float* p, float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; i++) {
            const float4 u = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
    }
}
template <int N>
__device__ inline void store_piece(uint16_t* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = f32_to_bf16_rne(v[0]);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; i++)
            w[i] = (uint32_t)f32_to_bf16_rne(v[2 * i]) | ((uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16);
        if constexpr (N == 4)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <int N>
__device__ inline void store_piece(float* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; i++)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

// A value's E4M3 codes come from v_cvt_scalef32_pk_fp8_f32 (two values,
// nearest even, subnormals included, not saturating): |v| is clamped to 448
// first, the format's largest value.
__device__ inline uint32_t e4m3_pack4(const float (&q)[4]) {
    typedef short s16x2_t __attribute__((ext_vector_type(2)));
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; i++) c[i] = __builtin_amdgcn_fmed3f(q[i], -448.f, 448.f);
    s16x2_t w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c[0], c[1], 1.0f, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c[2], c[3], 1.0f, true);
    return (uint32_t)(uint16_t)w[0] | ((uint32_t)(uint16_t)w[1] << 16);
}

}  // namespace moe
