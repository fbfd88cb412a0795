// Pieces of the norm-and-rotation kernels (latent_cache.cu; qk_norm_rope.cu, which lays
// its rows out otherwise, takes the conversions): a row of a head lies across a group of
// lanes, 8 elements (16 bytes of bf16) per lane.
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

// The E4M3 codes nearest to the fp32 quotients x / scale (ties to even, held at +-448).
__device__ __forceinline__ uint2 f32_to_e4m3x8(const float (&x)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 lo = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
        const float2 hi = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
        w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
    }
    return make_uint2(w[0], w[1]);
}

// Cosines and sines of one lane's 8 elements, dims e0 .. e0 + 7 (e0 < rot):
// 8 planes of each, or 4 where a plane's two dims are neighbours.
template <bool INTER>
struct LaneAngles {
    static constexpr int kPlanes = INTER ? 4 : 8;
    float c[kPlanes], s[kPlanes];
    __device__ __forceinline__ void load(const float *row, int e0, int rot) {
        const int half = rot >> 1;
        const int f0 = INTER ? e0 >> 1 : (e0 < half ? e0 : e0 - half);
#pragma unroll
        for (int i = 0; i < kPlanes; i += 4) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + f0 + i));
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + f0 + i));
            c[i] = c4.x, c[i + 1] = c4.y, c[i + 2] = c4.z, c[i + 3] = c4.w;
            s[i] = s4.x, s[i + 1] = s4.y, s[i + 2] = s4.z, s[i + 3] = s4.w;
        }
    }
};

// Rotates one lane's 8 elements in place.  Every lane of the warp calls it
// (split planes exchange their halves by shuffle: the partner dim lies rot / 16
// lanes away); lanes with e0 >= rot keep their elements.
template <bool INTER>
__device__ __forceinline__ void rotate8(float (&x)[8], const LaneAngles<INTER> &a, int e0, int rot) {
    if constexpr (INTER) {
        if (e0 < rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = x[2 * i], q = x[2 * i + 1];
                x[2 * i] = p * a.c[i] - q * a.s[i];
                x[2 * i + 1] = q * a.c[i] + p * a.s[i];
            }
        }
    } else {
        const int lane = threadIdx.x & 31;
        const bool first = e0 < (rot >> 1);
        const int partner = e0 < rot ? (first ? lane + (rot >> 4) : lane - (rot >> 4)) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __shfl_sync(0xffffffffu, x[i], partner);
            if (e0 < rot) x[i] = first ? x[i] * a.c[i] - y * a.s[i] : x[i] * a.c[i] + y * a.s[i];
        }
    }
}

}  // namespace pkv
