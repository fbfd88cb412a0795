// The latent cache's write and its gather.
//
// Write, for token t with position p and slot s (norm and rotation as in
// norm_rope.cuh):
//     cache[s][0 .. 511]   = norm(latent[t]; weight)
//     cache[s][512 .. 575] = R_p(key_rope[t])
//     query_rope_out[t][h] = R_p(query_rope[t][h])        (when a query is given)
// Rounded once, from fp32.  A warp takes a token's latent and key part (512
// dims in two 16-byte vectors a lane, the 64 rotated dims on 8 lanes), or 16 of
// its query heads (four heads side by side, four loads a lane in flight).
//
// Gather: the cached rows of every request, in order, into one contiguous
// array (the input of the up-projection to per-head keys and values).  A page
// is one run of 18432 bytes in both, so this is a copy of runs.  The grid is requests x pages of
// the longest, so a batch with one request far longer than the others launches mostly CTAs that
// leave at once.
//
// Both move bytes and compute next to nothing.  The gather is bound by memory (204 k rows of
// 256 requests, 471 MB: 78 us, 6.0 TB/s, 89% of a plain copy's rate).  The write is bound
// by the latency of its chain (position and slot, table row, sums over the warp) at four waves
// of CTAs: 8191 tokens with 16 query heads, 54.7 MB, 12.4 us, 65% of a copy's
// rate (13.7 with the partner dims fetched from other lanes and 64 registers).
#include "latent_common.cuh"
#include "norm_rope.cuh"

namespace pkv {

struct LatentWriteParams {
    uint4 *cache;                                  // rows of 72 16-byte vectors
    int64_t num_slots;
    const __nv_bfloat16 *latent, *key_rope, *weight;   // weight NULL: no norm
    int64_t latent_stride, key_stride;             // elements, as all strides
    float eps;
    const float *cos_sin;
    int64_t max_position;
    const int64_t *positions, *slots;
    __nv_bfloat16 *q_out;
    int64_t qo_token, qo_head;
    const __nv_bfloat16 *q;
    int64_t q_token, q_head;
    int32_t num_tokens, heads, warps_per_token;
    int32_t *status;
};

constexpr int kRopeRows = 16;                      // query heads per warp
constexpr int kWriteThreads = 128;
// CTAs an SM: ten leave 48 registers and 32 spilled bytes a thread: 12.4 us on 8191 tokens with 16 query
// heads; nine (56, 4 bytes) 12.6, eight (64, none) 13.0, twelve (40) 13.3.
constexpr int kWriteCtas = 10;

// Lane l of eight has planes 4 l .. 4 l + 3 of a row's 64 rotated dims: two pieces of four dims that
// turn with one another, or of two planes each where a plane's dims are neighbours.  No lane
// needs another's.
template <bool INTER> struct RopeLane {
    static __device__ __forceinline__ int first(int l) { return INTER ? l * 8 : l * 4; }
    static __device__ __forceinline__ int second(int l) { return INTER ? l * 8 + 4 : kLatRope / 2 + l * 4; }
    static __device__ __forceinline__ uint4 load(const __nv_bfloat16 *row, int l) {    // (not __ldg: rows may be rotated in place)
        if constexpr (INTER) return *reinterpret_cast<const uint4 *>(row + first(l));
        const uint2 a = *reinterpret_cast<const uint2 *>(row + first(l)), b = *reinterpret_cast<const uint2 *>(row + second(l));
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ uint4 turn(const uint4 &v, const float4 &c4, const float4 &s4) {
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
        float x[8], y[8];
        bf16x8_to_f32(v, x);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int i = INTER ? 2 * f : f, j = INTER ? 2 * f + 1 : f + 4;
            y[i] = x[i] * c[f] - x[j] * s[f];
            y[j] = x[j] * c[f] + x[i] * s[f];
        }
        return f32_to_bf16x8(y);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *row, int l, const uint4 &v) {
        if constexpr (INTER) {
            *reinterpret_cast<uint4 *>(row + first(l)) = v;
        } else {
            *reinterpret_cast<uint2 *>(row + first(l)) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2 *>(row + second(l)) = make_uint2(v.z, v.w);
        }
    }
};

template <bool INTER>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas) latent_write_kernel(const LatentWriteParams p) {
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);     // below 2^31
    const uint32_t token = item / static_cast<uint32_t>(p.warps_per_token);
    if (token >= static_cast<uint32_t>(p.num_tokens)) return;                         // whole warps
    const int part = static_cast<int>(item - token * p.warps_per_token);
    const int64_t t = token;
    using Rope = RopeLane<INTER>;
    const int l = lane & 7;
    const int64_t pos = __ldg(p.positions + t);
    const bool bad_pos = pos < 0 || pos >= p.max_position;
    if (part == 0) {
        const int64_t slot = __ldg(p.slots + t);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + t * p.latent_stride);
        const uint4 raw0 = __ldg(src + lane), raw1 = __ldg(src + 32 + lane);
        const uint4 rawk = Rope::load(p.key_rope + t * p.key_stride, l);
        if (slot < 0) return;                      // padding
        if (bad_pos || slot >= p.num_slots) {
            if (lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
            return;
        }
        const float *angles = p.cos_sin + pos * kLatRope + l * 4;
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(angles));
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(angles + kLatRope / 2));
        float x[8], y[8];
        bf16x8_to_f32(raw0, x);
        bf16x8_to_f32(raw1, y);
        uint4 *dst = p.cache + slot * (kLatRow / 8);
        if (p.weight) {
            float w0[8], w1[8];
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.weight) + lane), w0);
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p.weight) + 32 + lane), w1);
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], fmaf(y[i], y[i], sq));
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            const float inv = rsqrtf(sq * (1.f / kLatent) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = x[i] * inv * w0[i];
                y[i] = y[i] * inv * w1[i];
            }
        }
        dst[lane] = f32_to_bf16x8(x);
        dst[32 + lane] = f32_to_bf16x8(y);
        const uint4 k = Rope::turn(rawk, c4, s4);  // four copies side by side, one stored
        if (lane < 8) Rope::store(reinterpret_cast<__nv_bfloat16 *>(dst + kLatent / 8), l, k);
    } else {
        const int h0 = (part - 1) * kRopeRows + (lane >> 3);
        uint4 raw[kRopeRows / 4];
#pragma unroll
        for (int u = 0; u < kRopeRows / 4; ++u) {
            raw[u] = make_uint4(0, 0, 0, 0);
            if (h0 + 4 * u < p.heads) raw[u] = Rope::load(p.q + t * p.q_token + (h0 + 4 * u) * p.q_head, l);
        }
        if (bad_pos) {
            if (lane == 0 && __ldg(p.slots + t) >= 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
            return;
        }
        const float *angles = p.cos_sin + pos * kLatRope + l * 4;
        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(angles));
        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(angles + kLatRope / 2));
#pragma unroll
        for (int u = 0; u < kRopeRows / 4; ++u)
            if (h0 + 4 * u < p.heads)
                Rope::store(p.q_out + t * p.qo_token + (h0 + 4 * u) * p.qo_head, l, Rope::turn(raw[u], c4, s4));
    }
}

// One CTA copies up to kGatherPages pages of one request.
constexpr int kGatherPages = 2;
constexpr int kGatherThreads = 256;
constexpr int kGatherVecs = kGatherPages * kLatPageBytes / 16;                        // 2304
constexpr int kGatherPerThread = kGatherVecs / kGatherThreads;                        // 9
static_assert(kGatherVecs % kGatherThreads == 0, "whole rounds");

__global__ void __launch_bounds__(kGatherThreads) latent_gather_kernel(
    uint4 *out, int64_t out_rows, const uint4 *cache, int64_t num_blocks, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *key_start_loc, int32_t max_seq_len,
    int32_t *status) {
    const int r = blockIdx.y;
    const int page0 = blockIdx.x * kGatherPages;
    const int L = __ldg(seq_lens + r);
    const int64_t base = __ldg(key_start_loc + r);
    // (the first pages' ids are read beside the lengths, before anything is known of them)
    const int32_t *table = block_tables + static_cast<int64_t>(r) * max_blocks_per_seq;
    int id[kGatherPages];
#pragma unroll
    for (int i = 0; i < kGatherPages; ++i) id[i] = page0 + i < max_blocks_per_seq ? __ldg(table + page0 + i) : -1;
    if (L < 0 || L > max_seq_len || L > static_cast<int64_t>(max_blocks_per_seq) * kBlock ||
        (L > 0 && (base < 0 || base + L > out_rows))) {
        if (threadIdx.x == 0 && blockIdx.x == 0) set_status(status, PKV_ERR_DEVICE_METADATA);
        return;
    }
    const int rows = min(L - page0 * kBlock, kGatherPages * kBlock);   // rows of this CTA
    if (rows <= 0) return;
    const int vecs = rows * (kLatRowBytes / 16);
    uint4 *dst = out + (base + static_cast<int64_t>(page0) * kBlock) * (kLatRowBytes / 16);
    bool bad = false;
    const uint4 *src[kGatherPages];
#pragma unroll
    for (int i = 0; i < kGatherPages; ++i) {
        const bool inside = id[i] >= 0 && id[i] < num_blocks;
        bad |= !inside && i * kBlock < rows;
        src[i] = inside ? cache + static_cast<int64_t>(id[i]) * (kLatPageBytes / 16) : nullptr;
    }
    if (bad && threadIdx.x == 0) set_status(status, PKV_ERR_DEVICE_INDEX);
    uint4 val[kGatherPerThread];
#pragma unroll
    for (int u = 0; u < kGatherPerThread; ++u) {
        const int v = u * kGatherThreads + threadIdx.x;
        const int page = v >= kLatPageBytes / 16;
        const uint4 *s = page ? src[1] : src[0];
        if (v < vecs && s) val[u] = __ldg(s + v - page * (kLatPageBytes / 16));
    }
#pragma unroll
    for (int u = 0; u < kGatherPerThread; ++u) {
        const int v = u * kGatherThreads + threadIdx.x;
        if (v < vecs && (v >= kLatPageBytes / 16 ? src[1] : src[0])) dst[v] = val[u];
    }
}
static_assert(kGatherPages == 2, "the copy picks one of two pages");

}  // namespace pkv

extern "C" int pkv_latent_kv_write(void *latent_cache, int64_t num_blocks, int32_t block_size, const void *latent,
                                   int64_t latent_token_stride, const void *key_rope, int64_t key_rope_token_stride,
                                   const void *weight, float eps, const float *cos_sin, int64_t max_position,
                                   int32_t interleaved, const int64_t *positions, const int64_t *slot_mapping,
                                   int32_t num_tokens, void *query_rope_out, int64_t query_rope_out_token_stride,
                                   int64_t query_rope_out_head_stride, const void *query_rope,
                                   int64_t query_rope_token_stride, int64_t query_rope_head_stride, int32_t num_heads,
                                   int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_tokens < 0 || num_blocks <= 0 || max_position <= 0 || num_heads < 0 || num_heads > (1 << 20))
        return PKV_ERR_SHAPE;
    if (block_size != kBlock) return PKV_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.0e38f) return PKV_ERR_SHAPE;
    if (num_blocks > INT64_MAX / kLatPageBytes || max_position > INT64_MAX / kLatRope / 4) return PKV_ERR_SHAPE;
    if (num_tokens == 0) return PKV_OK;
    if (!latent_cache || !latent || !key_rope || !cos_sin || !positions || !slot_mapping) return PKV_ERR_NULL;
    if (latent_token_stride < kLatent || key_rope_token_stride < kLatRope) return PKV_ERR_SHAPE;
    if ((latent_token_stride % 8) || (key_rope_token_stride % 8)) return PKV_ERR_ALIGNMENT;
    uintptr_t all = reinterpret_cast<uintptr_t>(latent_cache) | reinterpret_cast<uintptr_t>(latent) |
                    reinterpret_cast<uintptr_t>(key_rope) | reinterpret_cast<uintptr_t>(weight) |
                    reinterpret_cast<uintptr_t>(cos_sin);
    if (num_heads > 0) {
        if (!query_rope_out || !query_rope) return PKV_ERR_NULL;
        if (query_rope_out_head_stride < kLatRope || query_rope_head_stride < kLatRope ||
            query_rope_out_token_stride < (num_heads - 1) * query_rope_out_head_stride + kLatRope ||
            query_rope_token_stride < (num_heads - 1) * query_rope_head_stride + kLatRope)
            return PKV_ERR_SHAPE;
        if ((query_rope_out_head_stride % 8) || (query_rope_head_stride % 8) || (query_rope_out_token_stride % 8) ||
            (query_rope_token_stride % 8))
            return PKV_ERR_ALIGNMENT;
        all |= reinterpret_cast<uintptr_t>(query_rope_out) | reinterpret_cast<uintptr_t>(query_rope);
    }
    if (all & 15u) return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slot_mapping)) & 7u)
        return PKV_ERR_ALIGNMENT;
    LatentWriteParams p;
    p.cache = static_cast<uint4 *>(latent_cache);
    p.num_slots = num_blocks * kBlock;
    p.latent = static_cast<const __nv_bfloat16 *>(latent);
    p.key_rope = static_cast<const __nv_bfloat16 *>(key_rope);
    p.weight = static_cast<const __nv_bfloat16 *>(weight);
    p.latent_stride = latent_token_stride, p.key_stride = key_rope_token_stride;
    p.eps = eps;
    p.cos_sin = cos_sin, p.max_position = max_position;
    p.positions = positions, p.slots = slot_mapping;
    p.q_out = static_cast<__nv_bfloat16 *>(query_rope_out);
    p.qo_token = query_rope_out_token_stride, p.qo_head = query_rope_out_head_stride;
    p.q = static_cast<const __nv_bfloat16 *>(query_rope);
    p.q_token = query_rope_token_stride, p.q_head = query_rope_head_stride;
    p.num_tokens = num_tokens, p.heads = num_heads;
    p.warps_per_token = 1 + (num_heads + kRopeRows - 1) / kRopeRows;
    p.status = device_status;
    const int64_t warps = static_cast<int64_t>(num_tokens) * p.warps_per_token;
    if (warps > INT32_MAX - kWriteThreads) return PKV_ERR_SHAPE;
    const int64_t blocks = (warps + kWriteThreads / 32 - 1) / (kWriteThreads / 32);
    (interleaved ? latent_write_kernel<true> : latent_write_kernel<false>)<<<
        static_cast<unsigned>(blocks), kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int pkv_latent_gather(void *out, int64_t out_rows, const void *latent_cache, int64_t num_blocks,
                                 int32_t block_size, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *key_start_loc, int32_t num_seqs,
                                 int32_t max_seq_len, int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_seqs < 0 || out_rows < 0 || num_blocks <= 0 || max_seq_len < 0 || max_blocks_per_seq < 0)
        return PKV_ERR_SHAPE;
    if (block_size != kBlock) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535) return PKV_ERR_SHAPE;
    if (num_blocks > INT64_MAX / kLatPageBytes) return PKV_ERR_SHAPE;
    if (num_seqs == 0) return PKV_OK;
    // a bound of no rows: nothing is copied, and the lengths are looked at for the status alone
    const bool any = max_seq_len > 0;
    if (!any && !device_status) return PKV_OK;
    if ((static_cast<int64_t>(max_seq_len) + kBlock - 1) / kBlock > max_blocks_per_seq) return PKV_ERR_SHAPE;
    if (!seq_lens || !key_start_loc || (any && ((!out && out_rows > 0) || !latent_cache || !block_tables))) return PKV_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(latent_cache)) & 15u) return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
         reinterpret_cast<uintptr_t>(key_start_loc)) & 3u)
        return PKV_ERR_ALIGNMENT;
    const int per = kGatherPages * kBlock;
    const int64_t most = any ? (static_cast<int64_t>(max_seq_len) + per - 1) / per : 1;
    const dim3 grid(static_cast<unsigned>(most), static_cast<unsigned>(num_seqs));
    latent_gather_kernel<<<grid, kGatherThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<uint4 *>(out), out_rows, static_cast<const uint4 *>(latent_cache), num_blocks, block_tables,
        any ? max_blocks_per_seq : 0, seq_lens, key_start_loc, max_seq_len, device_status);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
