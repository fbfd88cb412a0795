// The latent cache: one row a token, shared by every head, of 512 latent dims
// (keys and values both) followed by 64 rotated key dims.
#pragma once

#include "tc_common.cuh"

namespace pkv {

constexpr int kLatent = PKV_LATENT_DIM;              // 512: latent dims, the values' width
constexpr int kLatRope = PKV_LATENT_ROPE_DIM;        // 64: rotated key dims
constexpr int kLatRow = kLatent + kLatRope;          // 576: a cached row, the keys' width
constexpr int kLatRowBytes = kLatRow * 2;            // 1152
constexpr int kLatPageBytes = kBlock * kLatRowBytes; // 18432

// ---- issuing MMAs from a converged warp -----------------------------------------
//
// tcgen05.mma takes its descriptors from uniform registers.  When one lane
// issues inside `if (lane == 0)`, the compiler moves every operand of every
// product there from per-lane registers, and a product costs at least 45 cycles
// of issue whatever its shape (measured alone on an SM: 64 x 64 x 16 at 50
// cycles).  A warp that stays converged, with the lane chosen by elect.sync only
// around the products, keeps the operands uniform: 64 x 64 x 16 at 33 cycles, 128 x
// 64 x 16 at 50, 128 x 128 x 16 at 65, which is what their shared-memory reads
// (128 bytes a cycle) and arithmetic take.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}

// A value that is the same in every lane, in a form the compiler knows to be.
template <typename T> __device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }

// A converged warp's bounded wait; false (and the error recorded) once it gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *status) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
    if (!ok) set_status(status, PKV_ERR_DEVICE_TIMEOUT);
    return ok;
}

// A converged warp's wait for an event that may be any number of key tiles away (the end of an
// item, the tiles on the causal diagonal): it gives up once no tile has been loaded between two
// looks at `tiles`, which the loading warp counts up; a bounded wait lies before each look.
// (That one is over after 13.8 M keys at 1.85 us a 128-key tile, or 10 M at 1.25 us a 64-key one.)
__device__ __forceinline__ bool warp_wait_tiles(uint64_t *bar, uint32_t parity, const volatile int32_t *tiles,
                                                int32_t *status) {
    int32_t seen = -1;
    while (!__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity))) {
        const int32_t now = uniform(*tiles);
        if (now == seen) {
            set_status(status, PKV_ERR_DEVICE_TIMEOUT);
            return false;
        }
        seen = now;
    }
    return true;
}

}  // namespace pkv
