// What the norm-and-rotation kernels (qk_norm_rope.cu, latent_cache.cu) compute, and the
// conversions they share.
//
//   norm      y_i = x_i * rsqrt(mean(x^2) + eps) * w_i, in fp32
//   rotation  the first `rot` dims of a row as rot / 2 planes; plane f turns by
//             the angle whose cosine and sine the table row of the token's
//             position holds at f and rot / 2 + f:
//               (a, b) -> (a c - b s, b c + a s)
//             with (a, b) = dims (f, rot / 2 + f), or (2 f, 2 f + 1) interleaved
//
// Both are fp32; a row is rounded once, on its way out.
#pragma once

#include <cuda_fp8.h>

#include "pkv_common.cuh"

namespace pkv {

__device__ __forceinline__ void bf16x8_to_f32(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// A divisor on the way to E4M3 codes.  The code of a quotient depends on which side of the
// midpoints between codes it lies; they have at most 5 significant bits, so the low 19 bits of
// their fp32 form are zero.  x * RN(1 / scale) is less than 2.5 ulps off the rounded quotient
// (2^-24 of it from either rounding, half an ulp from the quotient's; 5 ulps below the one
// midpoint that is a power of two), so where it lies more than 8 ulps from every such number
// its code is the quotient's.  Only the others are divided.  2048 tokens of 64/8 heads, one
// row in five with codes: 17.4 us, with every element divided 19.5 (the registers that the
// divisions took cost a CTA an SM too).
struct E4m3Scale {
    float scale, inv;
    int32_t near;             // divide if a product is as near as this: 16, -1 never, 2^19 always
};

__host__ inline E4m3Scale e4m3_scale(float scale) {
    E4m3Scale s;
    s.scale = scale, s.inv = 1.f / scale;
    int e;
    const float m = frexpf(scale, &e);
    // far from the ends of the exponents, what the product loses below them has code 0 anyway;
    // by a power of two it is exact
    s.near = e < -100 || e > 100 ? 1 << 19 : (m == 0.5f ? -1 : 16);
    return s;
}

// The E4M3 codes nearest to the fp32 quotients x / scale (ties to even, held at +-448).
__device__ __forceinline__ uint2 f32_to_e4m3x8(const float (&x)[8], const E4m3Scale &s) {
    int32_t nearest = 1 << 19;
#pragma unroll
    for (int i = 0; i < 8; ++i) nearest = min(nearest, (__float_as_int(x[i] * s.inv) + 8) & 0x7FFFF);
    float q[8];
    if (nearest <= s.near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], s.scale);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = x[i] * s.inv;
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 lo = make_float2(q[4 * i], q[4 * i + 1]);
        const float2 hi = make_float2(q[4 * i + 2], q[4 * i + 3]);
        w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
    }
    return make_uint2(w[0], w[1]);
}

}  // namespace pkv
