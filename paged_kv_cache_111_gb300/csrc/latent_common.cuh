// The latent cache: one row a token, shared by every head, of 512 latent dims
// (keys and values both) followed by 64 rotated key dims.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kLatent = PKV_LATENT_DIM;              // 512: latent dims, the values' width
constexpr int kLatRope = PKV_LATENT_ROPE_DIM;        // 64: rotated key dims
constexpr int kLatRow = kLatent + kLatRope;          // 576: a cached row, the keys' width
constexpr int kLatRowBytes = kLatRow * 2;            // 1152
constexpr int kLatPageBytes = kBlock * kLatRowBytes; // 18432

}  // namespace pkv
