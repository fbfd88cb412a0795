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
// What bounds it: memory, and close behind it the instructions.  A warp takes one
// token's query rows, key rows or value rows, 8 rows of 128 dims (16 of 64), d / 8
// lanes a row, so that what it does with them is the same for all of them: a value
// row is copied, and of the others each lane has four dims and the four that they
// turn with (two 8-byte pieces), so that no lane needs another's.  Every load (rows,
// position, slot, then the table row) is issued before any arithmetic; the
// arithmetic runs on pairs (f32x2).  Whole rows on 16-byte pieces, with the partner
// dims fetched from other lanes, took four times the instructions: 60 us on 8192
// tokens of 32/8 heads of 128 (206 MB), against 36 us (5.7 TB/s, 84% of a plain copy's
// rate).  The E4M3 form, 2048 tokens of 64/8 heads (80 MB): 17.4 us (neighbouring dims), 18.9 (halves).
#include "norm_rope.cuh"
#include "prefill_common.cuh"

namespace pkv {

constexpr int kRowsUnroll = 4;                   // rows a lane
constexpr int kQkThreads = 128;                  // (256: 41 us where 128 take 39)
// CTAs an SM: nine leave 56 registers, with which the E4M3 forms spill (halves: 28 bytes stored and 100
// loaded a thread, pairs: 12 and 48); they are the fastest all the same.  2048 tokens of 64/8 heads, at
// nine, eight (64 registers, 4 bytes spilled) and seven (72, none): E4M3 pairs 17.3, 18.2, 18.8 us,
// halves 18.9, 19.2, 19.9, bf16 17.8, 18.6, 18.6; the 8192-token chunk 36, 38 at eight, 37 at ten.
constexpr int kQkCtas = 9;

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
    int32_t num_tokens, hq, hkv, rot;
    int32_t q_chunks, kv_chunks, chunks;        // warps per token: of the query, of key or value, in all
    float eps;
    E4m3Scale k_scale, v_scale;
    int32_t *status;
};

template <int HD, bool FP8, bool INTER>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) qk_norm_rope_kernel(const QkParams p) {
    pdl_trigger();                            // the attention plan may start (it reads no cache and no query)
    constexpr int kLanes = HD / 8;            // lanes of a row
    constexpr int kGroups = 32 / kLanes;      // rows side by side in a warp
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);     // below 2^31
    const uint32_t token = item / static_cast<uint32_t>(p.chunks);
    if (token >= static_cast<uint32_t>(p.num_tokens)) return;                      // whole warps
    int chunk = static_cast<int>(item - token * p.chunks);
    const int64_t t = token;
    const int64_t pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
    // query, key or value rows
    const int kind = chunk < p.q_chunks ? 0 : (chunk < p.q_chunks + p.kv_chunks ? 1 : 2);
    chunk -= kind == 0 ? 0 : (kind == 1 ? p.q_chunks : p.q_chunks + p.kv_chunks);
    const int rows = kind == 0 ? p.hq : p.hkv;
    const __nv_bfloat16 *src = kind == 0 ? p.query + t * p.q_stride
                                         : (kind == 1 ? p.key + t * p.k_stride : p.value + t * p.v_stride);
    const int l = lane % kLanes;
    const int row0 = chunk * kRowsUnroll * kGroups + lane / kLanes;
    // this lane's two pieces of four dims: turned together, or neighbours
    const bool turns = kind < 2 && l * 8 < p.rot;
    const bool split = !INTER && turns;
    const bool whole = INTER || kind == 2;    // 16 bytes in one piece, in every lane
    const int da = split ? l * 4 : l * 8, db = split ? (p.rot >> 1) + l * 4 : l * 8 + 4;
    uint2 ra[kRowsUnroll], rb[kRowsUnroll];
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
        const int row = row0 + u * kGroups;
        if (row < rows) {                     // (not __ldg: query_out may be query)
            if (whole) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + row * HD + da);
                ra[u] = make_uint2(v.x, v.y), rb[u] = make_uint2(v.z, v.w);
            } else {
                ra[u] = *reinterpret_cast<const uint2 *>(src + row * HD + da);
                rb[u] = *reinterpret_cast<const uint2 *>(src + row * HD + db);
            }
        }
    }
    // a token past the table is skipped; with a negative slot it is padding and no error
    const bool known = pos >= 0 && pos < p.max_position;
    if (slot >= 0 && (!known || slot >= p.num_slots) && lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
    if (!known) return;
    const bool stored = slot >= 0 && slot < p.num_slots;
    if (kind > 0 && !stored) return;

    // where a row goes: element offset of its first dim, of row 0 and from row to row
    const int64_t blk = slot / kBlock;
    const int64_t dst0 = kind == 0 ? t * p.out_stride
                                   : ((blk * p.hkv * 2 + (kind - 1)) * kBlock + (slot - blk * kBlock)) * HD;
    const int step = kind == 0 ? HD : 2 * kBlock * HD;
    auto store = [&](int row, const uint64_t (&x)[4]) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(x[i], f[2 * i], f[2 * i + 1]);
        const int64_t dst = dst0 + static_cast<int64_t>(row) * step;
        if (FP8 && kind > 0) {
            const uint2 c = f32_to_e4m3x8(f, kind == 1 ? p.k_scale : p.v_scale);
            if (whole) {
                *reinterpret_cast<uint2 *>(p.cache + dst + da) = c;
            } else {
                *reinterpret_cast<uint32_t *>(p.cache + dst + da) = c.x;
                *reinterpret_cast<uint32_t *>(p.cache + dst + db) = c.y;
            }
        } else {
            __nv_bfloat16 *out = (kind == 0 ? p.query_out : reinterpret_cast<__nv_bfloat16 *>(p.cache)) + dst;
            const uint4 v = f32_to_bf16x8(f);
            if (whole) {
                *reinterpret_cast<uint4 *>(out + da) = v;
            } else {
                *reinterpret_cast<uint2 *>(out + da) = make_uint2(v.x, v.y);
                *reinterpret_cast<uint2 *>(out + db) = make_uint2(v.z, v.w);
            }
        }
    };
    auto pair = [](uint32_t w) { return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); };
    auto mul = [](uint64_t a, uint64_t b) {
        uint64_t d;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
        return d;
    };

    if (kind == 2) {
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
            const int row = row0 + u * kGroups;
            if (row >= rows) return;
            if constexpr (FP8) {
                const uint64_t x[4] = {pair(ra[u].x), pair(ra[u].y), pair(rb[u].x), pair(rb[u].y)};
                store(row, x);
            } else {                          // a bit copy
                uint8_t *out = p.cache + 2 * (dst0 + static_cast<int64_t>(row) * step);
                *reinterpret_cast<uint4 *>(out + 2 * da) = make_uint4(ra[u].x, ra[u].y, rb[u].x, rb[u].y);
            }
        }
        return;
    }

    // cosines and sines of planes 4 l .. 4 l + 3
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {
        const float *angles = p.cos_sin + pos * p.rot + l * 4;
        c4 = __ldg(reinterpret_cast<const float4 *>(angles));
        s4 = __ldg(reinterpret_cast<const float4 *>(angles + (p.rot >> 1)));
    }
    const __nv_bfloat16 *weight = kind == 0 ? p.q_weight : p.k_weight;
    uint2 wa = make_uint2(0, 0), wb = wa;
    if (weight) {
        wa = __ldg(reinterpret_cast<const uint2 *>(weight + da));
        wb = __ldg(reinterpret_cast<const uint2 *>(weight + db));
    }
    const uint64_t w[4] = {pair(wa.x), pair(wa.y), pair(wb.x), pair(wb.y)};
    const uint64_t c01 = f2_pack(c4.x, c4.y), c23 = f2_pack(c4.z, c4.w);
    const uint64_t s01 = f2_pack(s4.x, s4.y), s23 = f2_pack(s4.z, s4.w);
    const uint64_t n01 = f2_pack(-s4.x, -s4.y), n23 = f2_pack(-s4.z, -s4.w);
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
        const int row = row0 + u * kGroups;
        if (row - lane / kLanes >= rows) break;               // no row of this warp left
        uint64_t x[4] = {pair(ra[u].x), pair(ra[u].y), pair(rb[u].x), pair(rb[u].y)};
        if (weight) {                                         // (rows past the last: of no use, and not stored)
            float q0, q1;
            f2_unpack(f2_add(f2_fma(x[0], x[0], mul(x[1], x[1])), f2_fma(x[2], x[2], mul(x[3], x[3]))), q0, q1);
            float sq = q0 + q1;
#pragma unroll
            for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            const float inv = rsqrtf(sq * (1.f / HD) + p.eps);
            const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = mul(mul(x[i], inv2), w[i]);
        }
        if (turns) {
            if constexpr (INTER) {
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b;
                    f2_unpack(x[i], a, b);
                    x[i] = f2_pack(a * c[i] - b * s[i], b * c[i] + a * s[i]);
                }
            } else {
                const uint64_t a01 = x[0], a23 = x[1], b01 = x[2], b23 = x[3];
                x[0] = f2_fma(a01, c01, mul(b01, n01));
                x[1] = f2_fma(a23, c23, mul(b23, n23));
                x[2] = f2_fma(b01, c01, mul(a01, s01));
                x[3] = f2_fma(b23, c23, mul(a23, s23));
            }
        }
        if (row < rows) store(row, x);
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
    p.q_chunks = (hq + per_warp - 1) / per_warp;
    p.kv_chunks = (hkv + per_warp - 1) / per_warp;
    p.chunks = p.q_chunks + 2 * p.kv_chunks;
    p.eps = eps, p.k_scale = e4m3_scale(k_scale), p.v_scale = e4m3_scale(v_scale);
    p.status = device_status;
    const int64_t warps = static_cast<int64_t>(num_tokens) * p.chunks;
    const int64_t blocks = (warps + kQkThreads / 32 - 1) / (kQkThreads / 32);
    if (warps > INT32_MAX - kQkThreads) return PKV_ERR_SHAPE;
    void (*kernel)(QkParams);
    const bool it = interleaved != 0;
    if (head_size == 128)
        kernel = fp8 ? (it ? qk_norm_rope_kernel<128, true, true> : qk_norm_rope_kernel<128, true, false>)
                     : (it ? qk_norm_rope_kernel<128, false, true> : qk_norm_rope_kernel<128, false, false>);
    else
        kernel = fp8 ? (it ? qk_norm_rope_kernel<64, true, true> : qk_norm_rope_kernel<64, true, false>)
                     : (it ? qk_norm_rope_kernel<64, false, true> : qk_norm_rope_kernel<64, false, false>);
    kernel<<<static_cast<unsigned>(blocks), kQkThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
