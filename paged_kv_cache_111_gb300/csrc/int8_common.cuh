// The int8 cache: int8 codes in the pages of the other caches,
//     int8 [num_blocks][num_kv_heads][2][16][head_size],
// and an fp32 scale for each block, kv head and side (K, V),
//     float [num_blocks][num_kv_heads][2];
// code c stands for c * scale.  What its kernels share.
#pragma once

#include "prefill_common.cuh"

namespace pkv {

// The smallest scale.  It keeps 1 / scale finite and a block of zeros from having no scale at all; values
// below 2^-61 are held as 0.
constexpr float kInt8LeastScale = 8.673617379884035e-19f;      // 2^-60

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Four codes -> two pairs of fp32.  A byte u = code + 128 in the low bits of the fp32 number 2^23 gives 2^23 + u
// exactly.
__device__ __forceinline__ void int8x4_to_f32(uint32_t w, uint64_t &p01, uint64_t &p23) {
    const uint32_t u = w ^ 0x80808080u;
    const uint64_t bias = f2_pack(-8388736.f, -8388736.f);
    p01 = f2_add(f2_pack(__uint_as_float(prmt(u, 0x4B000000u, 0x7540)), __uint_as_float(prmt(u, 0x4B000000u, 0x7541))),
                 bias);
    p23 = f2_add(f2_pack(__uint_as_float(prmt(u, 0x4B000000u, 0x7542)), __uint_as_float(prmt(u, 0x4B000000u, 0x7543))),
                 bias);
}

// Four codes -> f16 numbers 1152 + code (a byte u = code + 128 in the low bits of the f16 number 1024 gives 1024 + u
// exactly).
constexpr float kInt8Bias = 1152.f;
__device__ __forceinline__ void int8x4_to_biased_f16(uint32_t w, uint32_t &h01, uint32_t &h23) {
    const uint32_t u = w ^ 0x80808080u;
    h01 = prmt(u, 0x64646464u, 0x4140);
    h23 = prmt(u, 0x64646464u, 0x4342);
}
// ... and back to the codes.
__device__ __forceinline__ uint32_t unbias_f16(uint32_t h) {
    const uint32_t b = 0x64806480u;                            // 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Attention's weights p' = 2^(e - m) enter P V as one f16 each, so a weight below 2^-14, a subnormal, is off by 2^-25
// absolute.  The reference m lies a lift below a row's largest e (or further): f16 has the room, and what counts is
// 2^-(25 + lift) of the largest weight, for long tails beside a key that takes most of the sum.  In the decode kernel a
// weight may grow by 2^8 before the reference moves, as without the lift.  In the chunk kernel, which looks for a row's
// largest e only where a tile's 128 weights sum to more than f16 holds, a higher lift has it look more often: 2046
// tokens at 8190 keys of 32/8 heads 282 us with scores four times as far apart as normal data's and a lift of 3
// (without one, and a bound of 2^13, 283), 290 with 4, 302 with 6; on normal data 238 with any.
constexpr float kInt8DecodeLift = 7.f, kInt8DecodeMost = 15.f;      // 2^15 fits f16
constexpr float kInt8ChunkLift = 3.f, kInt8ChunkMost = 6e4f;        // a sum that no weight in it passes f16 with

// rint(x r) of two pairs as four codes.  |x r| is below 128, so that in 1.5 * 2^23 + x r, rounded once, the low byte is
// the code.  (A product rounded by itself would have to be kept from the addition: f32x2 products and sums are fused.)
__device__ __forceinline__ uint32_t f32_to_int8x4(uint64_t x01, uint64_t x23, uint64_t r2) {
    const uint64_t magic = f2_pack(12582912.f, 12582912.f);
    float a, b, c, d;
    f2_unpack(f2_fma(x01, r2, magic), a, b);
    f2_unpack(f2_fma(x23, r2, magic), c, d);
    return prmt(prmt(__float_as_uint(a), __float_as_uint(b), 0x0040),
                prmt(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

}  // namespace pkv
