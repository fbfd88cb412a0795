// Norm of query and key heads, their rotation to the tokens' positions, and
// the cache write, in one pass over the projections' outputs.
//
// For token t with position p and slot b * 16 + o, per head of d dims
// (norm and rotation as in norm_rope.cuh):
//     query_out[t][h]   = R_p(norm(query[t][h]; q_weight))
//     cache[b][h][0][o] = R_p(norm(key[t][h]; k_weight))
//     cache[b][h][1][o] = value[t][h]                       (bit copy)
// and the same with E4M3 codes of the quotients by the scales.  The key goes
// from fp32 straight to the cache's type: one rounding (a bf16 key written by
// the separate cache write would be rounded twice over an E4M3 cache).
//
// What bounds it: memory.  A row is d / 8 lanes of 16 bytes, so a warp holds
// 2 rows (d = 128) or 4 (d = 64) at a time; it takes kRowsUnroll times that of
// one token and issues every load (rows, position, slot, then the table row)
// before any arithmetic, and reads the angles once for all of them.  The rows
// of a token are its query heads, key heads, then value heads.
#include "norm_rope.cuh"

namespace pkv {

constexpr int kRowsUnroll = 4;

struct QkParams {
    __nv_bfloat16 *query_out;
    int64_t out_stride;                       // elements between tokens, as the others
    const __nv_bfloat16 *query, *key, *value;
    int64_t q_stride, k_stride, v_stride;
    const __nv_bfloat16 *q_weight, *k_weight;   // NULL: no norm
    const float *cos_sin;
    int64_t max_position;
    const int64_t *positions, *slots;
    uint8_t *cache;
    int64_t num_slots;
    int32_t num_tokens, hq, hkv, rot, chunks;   // chunks: warps per token
    float eps, k_scale, v_scale;
    int32_t *status;
};

template <int HD, bool FP8, bool INTER>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkParams p) {
    pdl_trigger();                            // the attention plan may start (it reads no cache and no query)
    constexpr int kLanes = HD / 8;            // lanes of a row
    constexpr int kGroups = 32 / kLanes;      // rows side by side in a warp
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t = item / p.chunks;
    if (t >= p.num_tokens) return;            // whole warps
    const int chunk = static_cast<int>(item - t * p.chunks);
    const int group = lane / kLanes, e0 = (lane % kLanes) * 8;
    const int rows = p.hq + 2 * p.hkv;
    const int row0 = chunk * kRowsUnroll * kGroups + group;

    const int64_t pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
    uint4 raw[kRowsUnroll];
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
        const int row = row0 + u * kGroups;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (row < rows) {
            const __nv_bfloat16 *src = row < p.hq ? p.query + t * p.q_stride + static_cast<int64_t>(row) * HD
                                       : row < p.hq + p.hkv
                                           ? p.key + t * p.k_stride + static_cast<int64_t>(row - p.hq) * HD
                                           : p.value + t * p.v_stride + static_cast<int64_t>(row - p.hq - p.hkv) * HD;
            raw[u] = *reinterpret_cast<const uint4 *>(src + e0);   // (not __ldg: query_out may be query)
        }
    }
    // a token past the table is skipped; with a negative slot it is padding and no error
    if (pos < 0 || pos >= p.max_position || slot >= p.num_slots) {
        if (lane == 0 && (slot >= 0)) set_status(p.status, PKV_ERR_DEVICE_INDEX);
        if (pos < 0 || pos >= p.max_position) return;
    }
    const bool stored = slot >= 0 && slot < p.num_slots;
    LaneAngles<INTER> ang{};
    if (e0 < p.rot) ang.load(p.cos_sin + pos * p.rot, e0, p.rot);
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (p.q_weight) wq = __ldg(reinterpret_cast<const uint4 *>(p.q_weight + e0));
    if (p.k_weight) wk = __ldg(reinterpret_cast<const uint4 *>(p.k_weight + e0));
    const int64_t blk = stored ? slot / kBlock : 0;
    const int off = static_cast<int>(stored ? slot - blk * kBlock : 0);

#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
        const int row = row0 + u * kGroups;
        if (row - group >= rows) break;       // no row of this warp left
        const bool is_q = row < p.hq, is_v = row >= p.hq + p.hkv;
        float x[8];
        bf16x8_to_f32(raw[u], x);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
        const bool normed = is_q ? p.q_weight != nullptr : (!is_v && p.k_weight != nullptr);
        if (normed) {
            const float inv = rsqrtf(sq * (1.f / HD) + p.eps);
            float w[8];
            bf16x8_to_f32(is_q ? wq : wk, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
        }
        if (row - group < p.hq + p.hkv) {     // some row of the warp is a query or key
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
            rotate8<INTER>(y, ang, e0, p.rot);
            if (!is_v) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = y[i];
            }
        }
        if (row >= rows) continue;
        if (is_q) {
            *reinterpret_cast<uint4 *>(p.query_out + t * p.out_stride + static_cast<int64_t>(row) * HD + e0) =
                f32_to_bf16x8(x);
        } else if (stored) {
            const int h = is_v ? row - p.hq - p.hkv : row - p.hq;
            const int64_t dst = (((blk * p.hkv + h) * 2 + (is_v ? 1 : 0)) * kBlock + off) * HD + e0;
            if constexpr (FP8)
                *reinterpret_cast<uint2 *>(p.cache + dst) = f32_to_e4m3x8(x, is_v ? p.v_scale : p.k_scale);
            else
                *reinterpret_cast<uint4 *>(p.cache + dst * 2) = is_v ? raw[u] : f32_to_bf16x8(x);
        }
    }
}

// Argument checks and the launch, shared by the bf16 and E4M3 calls.
static int qk_norm_rope(bool fp8, void *query_out, int64_t out_stride, void *kv_cache, int64_t num_blocks,
                        int32_t hq, int32_t hkv, int32_t head_size, int32_t block_size, const void *query,
                        int64_t q_stride, const void *key, int64_t k_stride, const void *value, int64_t v_stride,
                        const void *q_weight, const void *k_weight, float eps, const float *cos_sin,
                        int64_t max_position, int32_t rotary_dim, int32_t interleaved, const int64_t *positions,
                        const int64_t *slot_mapping, int32_t num_tokens, float k_scale, float v_scale,
                        int32_t *device_status, void *stream) {
    if (num_tokens < 0 || hq <= 0 || hkv <= 0 || num_blocks <= 0 || max_position <= 0) return PKV_ERR_SHAPE;
    if (block_size != kBlock || (head_size != 64 && head_size != 128)) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > head_size || rotary_dim % 16) return PKV_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.0e38f) return PKV_ERR_SHAPE;
    if (fp8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || k_scale > 3.0e38f || v_scale > 3.0e38f)) return PKV_ERR_SHAPE;
    if (hq > (1 << 20) || hkv > (1 << 20)) return PKV_ERR_SHAPE;
    if (num_blocks > INT64_MAX / kBlock || max_position > INT64_MAX / rotary_dim / 4) return PKV_ERR_SHAPE;
    if (num_tokens == 0) return PKV_OK;
    if (!query_out || !kv_cache || !query || !key || !value || !cos_sin || !positions || !slot_mapping)
        return PKV_ERR_NULL;
    const int64_t qrow = static_cast<int64_t>(hq) * head_size, kvrow = static_cast<int64_t>(hkv) * head_size;
    if (out_stride < qrow || q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return PKV_ERR_SHAPE;
    if ((out_stride % 8) || (q_stride % 8) || (k_stride % 8) || (v_stride % 8)) return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(query_out) | reinterpret_cast<uintptr_t>(kv_cache) |
         reinterpret_cast<uintptr_t>(query) | reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value) |
         reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight) |
         reinterpret_cast<uintptr_t>(cos_sin)) & 15u)
        return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slot_mapping)) & 7u)
        return PKV_ERR_ALIGNMENT;

    QkParams p;
    p.query_out = static_cast<__nv_bfloat16 *>(query_out);
    p.out_stride = out_stride;
    p.query = static_cast<const __nv_bfloat16 *>(query);
    p.key = static_cast<const __nv_bfloat16 *>(key);
    p.value = static_cast<const __nv_bfloat16 *>(value);
    p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.q_weight = static_cast<const __nv_bfloat16 *>(q_weight);
    p.k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.positions = positions, p.slots = slot_mapping;
    p.cache = static_cast<uint8_t *>(kv_cache);
    p.num_slots = num_blocks * kBlock;
    p.num_tokens = num_tokens, p.hq = hq, p.hkv = hkv, p.rot = rotary_dim;
    const int per_warp = kRowsUnroll * (32 / (head_size / 8));
    p.chunks = (hq + 2 * hkv + per_warp - 1) / per_warp;
    p.eps = eps, p.k_scale = k_scale, p.v_scale = v_scale;
    p.status = device_status;
    const int64_t warps = static_cast<int64_t>(num_tokens) * p.chunks;
    const int64_t blocks = (warps + 7) / 8;
    if (blocks > INT32_MAX) return PKV_ERR_SHAPE;
    void (*kernel)(QkParams);
    const bool it = interleaved != 0;
    if (head_size == 128)
        kernel = fp8 ? (it ? qk_norm_rope_kernel<128, true, true> : qk_norm_rope_kernel<128, true, false>)
                     : (it ? qk_norm_rope_kernel<128, false, true> : qk_norm_rope_kernel<128, false, false>);
    else
        kernel = fp8 ? (it ? qk_norm_rope_kernel<64, true, true> : qk_norm_rope_kernel<64, true, false>)
                     : (it ? qk_norm_rope_kernel<64, false, true> : qk_norm_rope_kernel<64, false, false>);
    kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv

extern "C" int pkv_qk_norm_rope_kv_write(void *query_out, int64_t query_out_token_stride, void *kv_cache,
                                         int64_t num_blocks, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_size, int32_t block_size, const void *query,
                                         int64_t query_token_stride, const void *key, int64_t key_token_stride,
                                         const void *value, int64_t value_token_stride, const void *q_weight,
                                         const void *k_weight, float eps, const float *cos_sin, int64_t max_position,
                                         int32_t rotary_dim, int32_t interleaved, const int64_t *positions,
                                         const int64_t *slot_mapping, int32_t num_tokens, int32_t *device_status,
                                         void *stream) {
    return pkv::qk_norm_rope(false, query_out, query_out_token_stride, kv_cache, num_blocks, num_q_heads,
                             num_kv_heads, head_size, block_size, query, query_token_stride, key, key_token_stride,
                             value, value_token_stride, q_weight, k_weight, eps, cos_sin, max_position, rotary_dim,
                             interleaved, positions, slot_mapping, num_tokens, 1.f, 1.f, device_status, stream);
}

extern "C" int pkv_qk_norm_rope_kv_write_fp8(void *query_out, int64_t query_out_token_stride, void *kv_cache,
                                             int64_t num_blocks, int32_t num_q_heads, int32_t num_kv_heads,
                                             int32_t head_size, int32_t block_size, const void *query,
                                             int64_t query_token_stride, const void *key, int64_t key_token_stride,
                                             const void *value, int64_t value_token_stride, const void *q_weight,
                                             const void *k_weight, float eps, const float *cos_sin,
                                             int64_t max_position, int32_t rotary_dim, int32_t interleaved,
                                             const int64_t *positions, const int64_t *slot_mapping,
                                             int32_t num_tokens, float k_scale, float v_scale,
                                             int32_t *device_status, void *stream) {
    return pkv::qk_norm_rope(true, query_out, query_out_token_stride, kv_cache, num_blocks, num_q_heads,
                             num_kv_heads, head_size, block_size, query, query_token_stride, key, key_token_stride,
                             value, value_token_stride, q_weight, k_weight, eps, cos_sin, max_position, rotary_dim,
                             interleaved, positions, slot_mapping, num_tokens, k_scale, v_scale, device_status,
                             stream);
}
