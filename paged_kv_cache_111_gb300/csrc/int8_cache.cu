// The int8 cache (int8_common.cuh): the quantising write, alone and behind norm and rotation, reading
// requests back, and copies of blocks.
//
// Write.  The rows of one block, head and side that a call writes are quantised together:
//     a = max |x| over them,  s' = max(a / 127, 2^-60)
//     s = s' where the block's first row is among them, else max(the block's scale, s')
//     code = rint(x / s);  rows that were there, where s grew: code = rint(code * old / s)
// (quotients as products with the fp32 number r = 1 / s, rounded once: x r, and code (old r) with old r in fp32).  A
// new code is off by at most half a step s, one that saw g growths by at most (g + 1) / 2 steps.  If an x is no number,
// s is NaN.
//
// The tokens of a block stand side by side in a call (a stretch, at most 16), and every one of its warps finds its
// ends from the slots around its own token.  A stretch of n tokens is n warps' work: with n = 1 (decode) a warp
// takes its token's rows of 16 heads (of fewer where the call has few tokens); with more, the j-th token's warp takes
// heads j, j + n, ... of them, all n rows of each, so that a scale is made where all of its rows are.  So a chunk and a
// decode step both put every warp to work, without a plan and without atomics.
//
// What bounds it: of few tokens a chain of three trips to memory (slots, rows, the store; 64 tokens of 8 heads of 128,
// GPU time with their read-back: 5.9 us); of many, some 600 instructions a warp and 16 rows (issue 50%, 8331 tokens: 15
// us, 3.4 TB/s).  Behind norm and rotation a lane's fp32 rows wait for their scale in registers (128; 2046 tokens of
// 32/8 heads: 18 us); made a second time from the bf16 rows instead they leave room for more warps, and take 19.
//
// Reading back moves whole pages, 99% of a copy's rate where there are many; so do the copies.
#include "int8_common.cuh"
#include "norm_rope.cuh"

namespace pkv {

constexpr int kI8Threads = 128;
constexpr int kI8Warps = kI8Threads / 32;

struct Int8WriteParams {
    int8_t *cache;
    float *scales;
    int64_t num_blocks;
    const __nv_bfloat16 *key, *value;
    int64_t k_stride, v_stride;               // elements between tokens, as the others
    const int64_t *slots;
    int32_t num_tokens, hkv;
    int32_t q_chunks, kv_chunks, chunks;      // warps per token: query, one side (plain: both), all
    int32_t *status;
    // norm and rotation
    __nv_bfloat16 *query_out;
    int64_t out_stride;
    const __nv_bfloat16 *query;
    int64_t q_stride;
    const __nv_bfloat16 *q_weight, *k_weight; // NULL: no norm
    const float *cos_sin;
    int64_t max_position;
    const int64_t *positions;
    int32_t hq, rot;
    float eps;
};

__device__ __forceinline__ uint64_t bf16x2_to_f2(uint32_t w) {
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t largest_bits(const uint64_t (&x)[4]) {      // of |x|, as fp32 bits
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(x[i], a, b);
        m = max(m, max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
    }
    return m;
}

// A row's norm and rotation.  A lane has two pieces of four dims, x[0 .. 1] and x[2 .. 3]: four planes.
template <int HD, bool INTER>
__device__ __forceinline__ void norm_turn(uint64_t (&x)[4], bool normed, const uint64_t (&w)[4], float eps, bool turns,
                                          const float4 &c4, const float4 &s4) {
    if (normed) {
        float q0, q1;
        f2_unpack(f2_add(f2_fma(x[0], x[0], f2_mul(x[1], x[1])), f2_fma(x[2], x[2], f2_mul(x[3], x[3]))), q0, q1);
        float sq = q0 + q1;
#pragma unroll
        for (int m = HD / 16; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
        const float inv = rsqrtf(sq * (1.f / HD) + eps);
        const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_mul(x[i], inv2), w[i]);
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
            const uint64_t c01 = f2_pack(c4.x, c4.y), c23 = f2_pack(c4.z, c4.w);
            const uint64_t s01 = f2_pack(s4.x, s4.y), s23 = f2_pack(s4.z, s4.w);
            const uint64_t n01 = f2_pack(-s4.x, -s4.y), n23 = f2_pack(-s4.z, -s4.w);
            const uint64_t a01 = x[0], a23 = x[1], b01 = x[2], b23 = x[3];
            x[0] = f2_fma(a01, c01, f2_mul(b01, n01));
            x[1] = f2_fma(a23, c23, f2_mul(b23, n23));
            x[2] = f2_fma(b01, c01, f2_mul(a01, s01));
            x[3] = f2_fma(b23, c23, f2_mul(a23, s23));
        }
    }
}

// The scale of a block, head and side from the largest |x| of its new rows (fp32 bits) and the scale that it had.
__device__ __forceinline__ float int8_scale(uint32_t largest, float old, bool fresh) {
    const float least = fmaxf(__fmul_rn(__uint_as_float(largest), 1.f / 127.f), kInt8LeastScale);
    const float want = largest >= 0x7F800000u ? __int_as_float(0x7FC00000) : least;
    return fresh ? want : (old >= want || old != old ? old : want);
}

// The rows of one block, head and side that the call does not write, held to a scale that grew: by a whole warp.
template <int HD>
__device__ __forceinline__ void int8_requantise(int8_t *page, uint32_t written, float ratio, int lane) {
    const uint64_t r2 = f2_pack(ratio, ratio);
#pragma unroll
    for (int u = 0; u < kBlock * HD / 512; ++u) {
        const int at = (u * 32 + lane) * 16;
        if ((written >> (at / HD)) & 1u) continue;
        uint4 v = *reinterpret_cast<const uint4 *>(page + at);
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint64_t a, b;
            int8x4_to_f32(w[e], a, b);
            w[e] = f32_to_int8x4(a, b, r2);
        }
        *reinterpret_cast<uint4 *>(page + at) = v;
    }
}

// FORM 0: keys and values as they are; 1: norm and rotation, planes of halves; 2: of neighbouring dims.  UA: rows a
// lane takes of one token.
template <int HD, int FORM, int UA>
__global__ void __launch_bounds__(kI8Threads, FORM == 0 ? 7 : 4) int8_write_kernel(const Int8WriteParams p) {
    pdl_trigger();                            // the attention plan may start (it reads no cache and no query)
    constexpr bool INTER = FORM == 2;
    constexpr int kLanes = HD / 8;            // lanes of a row
    constexpr int kGroups = 32 / kLanes;      // rows side by side in a warp
    constexpr int U = kBlock / kGroups;       // rows of a block a lane
    constexpr int kHeads = UA * kGroups;      // heads a warp
    __shared__ int8_t s_row[kI8Warps][kBlock];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * kI8Warps + warp;                            // below 2^31
    const uint32_t token = item / static_cast<uint32_t>(p.chunks);
    if (token >= static_cast<uint32_t>(p.num_tokens)) return;                      // whole warps
    int chunk = static_cast<int>(item - token * p.chunks);
    const int64_t t = token;
    const int l = lane % kLanes, g = lane / kLanes;

    // query rows, or those of one side of the cache
    const int kind = FORM == 0 ? 2 : (chunk < p.q_chunks ? 0 : (chunk < p.q_chunks + p.kv_chunks ? 1 : 2));
    chunk -= FORM == 0 || kind == 0 ? 0 : (kind == 1 ? p.q_chunks : p.q_chunks + p.kv_chunks);
    const int heads = FORM == 0 ? 2 * p.hkv : (kind == 0 ? p.hq : p.hkv);
    const int h0 = chunk * kHeads, cnt = min(kHeads, heads - h0);

    // this lane's two pieces of four dims: turned together, or neighbours
    const bool turns = FORM != 0 && kind < 2 && l * 8 < p.rot;
    const bool split = !INTER && turns;
    const bool whole = FORM == 0 || INTER || kind == 2;       // 16 bytes in one piece, in every lane
    const int da = split ? l * 4 : l * 8, db = split ? (p.rot >> 1) + l * 4 : l * 8 + 4;
    auto load = [&](const __nv_bfloat16 *src) {               // (not __ldg: query_out may be query)
        if (whole) return *reinterpret_cast<const uint4 *>(src + da);
        const uint2 a = *reinterpret_cast<const uint2 *>(src + da), b = *reinterpret_cast<const uint2 *>(src + db);
        return make_uint4(a.x, a.y, b.x, b.y);
    };
    const __nv_bfloat16 *weight = FORM != 0 && kind < 2 ? (kind == 0 ? p.q_weight : p.k_weight) : nullptr;
    uint64_t w[4] = {};
    if (FORM != 0 && weight) {
        const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(weight + da));
        const uint2 wb = __ldg(reinterpret_cast<const uint2 *>(weight + db));
        w[0] = bf16x2_to_f2(wa.x), w[1] = bf16x2_to_f2(wa.y), w[2] = bf16x2_to_f2(wb.x), w[3] = bf16x2_to_f2(wb.y);
    }
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    auto angles = [&](int64_t pos) {                          // cosines and sines of planes 4 l .. 4 l + 3
        const float *at = p.cos_sin + pos * p.rot + l * 4;
        c4 = __ldg(reinterpret_cast<const float4 *>(at));
        s4 = __ldg(reinterpret_cast<const float4 *>(at + (p.rot >> 1)));
    };
    // a row in fp32, normed and turned where it is a key (or query)
    auto finish = [&](const uint4 &raw, uint64_t (&x)[4]) {
        x[0] = bf16x2_to_f2(raw.x), x[1] = bf16x2_to_f2(raw.y), x[2] = bf16x2_to_f2(raw.z), x[3] = bf16x2_to_f2(raw.w);
        if (FORM != 0 && kind < 2) norm_turn<HD, INTER>(x, weight != nullptr, w, p.eps, turns, c4, s4);
    };

    if (FORM != 0 && kind == 0) {
        const int64_t slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
        uint4 raw[UA];
#pragma unroll
        for (int u = 0; u < UA; ++u) {
            const int i = u * kGroups + g;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (i < cnt) raw[u] = load(p.query + t * p.q_stride + static_cast<int64_t>(h0 + i) * HD);
        }
        if (pos < 0 || pos >= p.max_position) {
            if (slot >= 0 && lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
            return;
        }
        if (turns) angles(pos);
#pragma unroll
        for (int u = 0; u < UA; ++u) {
            const int i = u * kGroups + g;
            uint64_t x[4];
            finish(raw[u], x);
            if (i >= cnt) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) f2_unpack(x[e], f[2 * e], f[2 * e + 1]);
            const uint4 v = f32_to_bf16x8(f);
            __nv_bfloat16 *out = p.query_out + t * p.out_stride + static_cast<int64_t>(h0 + i) * HD;
            if (whole) {
                *reinterpret_cast<uint4 *>(out + da) = v;
            } else {
                *reinterpret_cast<uint2 *>(out + da) = make_uint2(v.x, v.y);
                *reinterpret_cast<uint2 *>(out + db) = make_uint2(v.z, v.w);
            }
        }
        return;
    }

    // the slots (and positions) of tokens t - 16 .. t + 15
    const int64_t near = t - kBlock + lane;
    const bool there = near >= 0 && near < p.num_tokens;
    const int64_t slot_l = there ? __ldg(p.slots + near) : -1;
    bool known_l = there;
    int64_t pos_l = 0;
    if constexpr (FORM != 0) {
        pos_l = there ? __ldg(p.positions + near) : -1;
        known_l = pos_l >= 0 && pos_l < p.max_position;
    }
    const int64_t slot = __shfl_sync(0xffffffffu, slot_l, kBlock), pos = __shfl_sync(0xffffffffu, pos_l, kBlock);

    // the stretch: tokens start .. start + n - 1 of the 32 have slots in this token's block
    if (slot < 0) return;                                     // padding
    const int64_t blk = slot / kBlock;
    if (blk >= p.num_blocks) {
        if (lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
        return;
    }
    const uint32_t same = __ballot_sync(0xffffffffu, slot_l >= 0 && slot_l / kBlock == blk);
    if ((same & 0xFFFFu) == 0xFFFFu) {                        // the 17th of a stretch, or later: a slot given twice
        if (lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
        return;
    }
    const int start = 32 - __clz(~same & 0xFFFFu);            // 1 .. 16; the 32 lanes hold all of the first 16
    const int n = min(kBlock, __ffs(static_cast<int>(~(same >> start))) - 1);
    const int j = kBlock - start;
    const bool in = lane >= start && lane < start + n;
    const int off0 = static_cast<int>(slot & (kBlock - 1)) - j;   // of the first token, where offsets ascend by one
    uint32_t written;                                         // rows of the block
    const bool plain = !__any_sync(0xffffffffu, in && (slot_l != slot + (lane - kBlock) || !known_l));
    if (plain) {
        written = ((1u << n) - 1u) << off0;
    } else {
        // any order: of two tokens with one slot the last is written
        const int off_l = static_cast<int>(slot_l & (kBlock - 1));
        const uint32_t twins = __match_any_sync(0xffffffffu, in && known_l ? off_l : 32 + lane);
        const bool last = in && known_l && (twins >> lane) == 1u;
        written = __reduce_or_sync(0xffffffffu, last ? 1u << off_l : 0u);
        if (lane < kBlock) s_row[warp][lane] = -1;
        __syncwarp();
        if (last) s_row[warp][off_l] = static_cast<int8_t>(lane);
        __syncwarp();
    }
    if (!written) return;
    const bool fresh = written & 1u;
    auto side_of = [&](int h) { return FORM == 0 ? (h >= p.hkv ? 1 : 0) : kind - 1; };
    auto head_of = [&](int h) { return FORM == 0 && h >= p.hkv ? h - p.hkv : h; };
    auto row_of = [&](int h, int64_t tok) {
        return side_of(h) ? p.value + tok * p.v_stride + static_cast<int64_t>(head_of(h)) * HD
                          : p.key + tok * p.k_stride + static_cast<int64_t>(head_of(h)) * HD;
    };
    auto unit_of = [&](int h) { return (blk * p.hkv + head_of(h)) * 2 + side_of(h); };
    auto store = [&](int8_t *row, const uint64_t (&x)[4], float r) {
        const uint64_t r2 = f2_pack(r, r);
        const uint32_t a = f32_to_int8x4(x[0], x[1], r2), b = f32_to_int8x4(x[2], x[3], r2);
        if (whole) {
            *reinterpret_cast<uint2 *>(row + da) = make_uint2(a, b);
        } else {
            *reinterpret_cast<uint32_t *>(row + da) = a;
            *reinterpret_cast<uint32_t *>(row + db) = b;
        }
    };

    if (n == 1) {
        // one row of each of the heads: row u * kGroups + g is head h0 + it
        const int off = static_cast<int>(slot & (kBlock - 1));
        if (turns) angles(pos);
        uint4 raw[UA];
        float old[UA];
#pragma unroll
        for (int u = 0; u < UA; ++u) {
            const int i = u * kGroups + g;
            raw[u] = i < cnt ? load(row_of(h0 + i, t)) : make_uint4(0, 0, 0, 0);
            old[u] = i < cnt && !fresh ? p.scales[unit_of(h0 + i)] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < UA; ++u) {
            const int i = u * kGroups + g;
            uint64_t x[4];
            finish(raw[u], x);
            uint32_t m = largest_bits(x);
#pragma unroll
            for (int k = kLanes / 2; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
            const float s = int8_scale(m, old[u], fresh), r = __frcp_rn(s);
            if (i < cnt) {
                const int64_t unit = unit_of(h0 + i);
                store(p.cache + (unit * kBlock + off) * HD, x, r);
                if (l == 0 && !(s == old[u])) p.scales[unit] = s;
            }
            // the older rows of the heads whose scale grew, one head after the other
            const float ratio = __fmul_rn(old[u], r);
            uint32_t grown = __ballot_sync(0xffffffffu, l == 0 && i < cnt && !fresh && s > old[u]);
            while (grown) {
                const int from = __ffs(static_cast<int>(grown)) - 1;
                grown &= grown - 1;
                int8_requantise<HD>(p.cache + unit_of(h0 + u * kGroups + from / kLanes) * kBlock * HD, written,
                                    __shfl_sync(0xffffffffu, ratio, from), lane);
            }
        }
        return;
    }

    // the rows of one head at a time: row u * kGroups + g of the block, from the token that is written there
    int at[U];                                                // of the 32 tokens, or -1
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = u * kGroups + g;
        at[u] = !plain ? s_row[warp][row] : (((written >> row) & 1u) ? start + row - off0 : -1);
    }
    for (int hh = j; hh < cnt; hh += n) {
        const int h = h0 + hh;
        const int64_t unit = unit_of(h);
        const float old = fresh ? 0.f : p.scales[unit];
        const __nv_bfloat16 *rows = row_of(h, t - kBlock);
        const int64_t step = side_of(h) ? p.v_stride : p.k_stride;
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = at[u] >= 0 ? load(rows + at[u] * step) : make_uint4(0, 0, 0, 0);
        uint64_t x[U][4];                                     // (FORM 0: made twice, for fewer registers)
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (FORM != 0) {
                const int64_t here = __shfl_sync(0xffffffffu, pos_l, max(at[u], 0));
                if (turns && at[u] >= 0) angles(here);
                finish(raw[u], x[u]);
                if (at[u] >= 0) m = max(m, largest_bits(x[u]));
            } else {                                          // the largest |bf16| of either half of each word
                uint32_t a = __vmaxu2(raw[u].x & 0x7FFF7FFFu, raw[u].y & 0x7FFF7FFFu);
                a = __vmaxu2(a, __vmaxu2(raw[u].z & 0x7FFF7FFFu, raw[u].w & 0x7FFF7FFFu));
                m = __vmaxu2(m, a);
            }
        }
        if constexpr (FORM == 0) m = max(m & 0xFFFF0000u, m << 16);
        m = __reduce_max_sync(0xffffffffu, m);
        const float s = int8_scale(m, old, fresh), r = __frcp_rn(s);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at[u] >= 0) {
                if constexpr (FORM == 0) finish(raw[u], x[u]);
                store(p.cache + (unit * kBlock + u * kGroups + g) * HD, x[u], r);
            }
        if (lane == 0 && !(s == old)) p.scales[unit] = s;
        if (!fresh && s > old) int8_requantise<HD>(p.cache + unit * kBlock * HD, written, __fmul_rn(old, r), lane);
    }
}

// ---- reading back -----------------------------------------------------------------------------------------------

struct Int8GatherParams {
    __nv_bfloat16 *key_out, *value_out;
    int64_t rows;
    const int8_t *cache;
    const float *scales;
    int64_t num_blocks;
    const int32_t *block_tables;
    int32_t width, hkv, max_seq_len, per;     // per: pages of a CTA
    const int32_t *seq_lens, *starts;
    int32_t *status;
};

// A CTA takes some pages of one request, a warp one head of one page at a time: 16 rows of K and of V.
constexpr int kGatherThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kGatherThreads) int8_gather_kernel(const Int8GatherParams p) {
    constexpr int kLanes = HD / 8, kGroups = 32 / kLanes, U = kBlock / kGroups;
    const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a write of this cache may be the kernel before (so no load here is one of memory that never changes, __ldg's)
    pdl_wait();
    const int L = p.seq_lens[r];
    const int64_t row0 = p.starts[r];
    const int page0 = blockIdx.x * p.per;
    if (L < 0 || L > p.max_seq_len || row0 < 0 || row0 + L > p.rows) {
        if (L != 0 && blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, PKV_ERR_DEVICE_METADATA);
        return;
    }
    const int pages = min(p.per, (L + kBlock - 1) / kBlock - page0);
    if (pages <= 0) return;
    const int l = lane % kLanes, g = lane / kLanes;
    for (int unit = warp; unit < pages * p.hkv; unit += kGatherThreads / 32) {
        const int page = unit / p.hkv, h = unit - page * p.hkv;
        const int b = p.block_tables[static_cast<int64_t>(r) * p.width + page0 + page];
        if (b < 0 || b >= p.num_blocks) {
            if (h == 0 && lane == 0) set_status(p.status, PKV_ERR_DEVICE_INDEX);
            continue;
        }
        const int64_t at = static_cast<int64_t>(b) * p.hkv + h;
        const int8_t *src = p.cache + at * 2 * kBlock * HD + g * HD + l * 8;
        const float2 s = reinterpret_cast<const float2 *>(p.scales)[at];
        const int first = (page0 + page) * kBlock;
        uint2 c[2][U];
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int u = 0; u < U; ++u)
                c[side][u] = *reinterpret_cast<const uint2 *>(src + (side * kBlock + u * kGroups) * HD);
        const int64_t dst = ((row0 + first + g) * p.hkv + h) * HD + l * 8;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            __nv_bfloat16 *out = (side ? p.value_out : p.key_out) + dst;
            const float one = side ? s.y : s.x;
            const uint64_t s2 = f2_pack(one, one);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint64_t x[4];
                int8x4_to_f32(c[side][u].x, x[0], x[1]);
                int8x4_to_f32(c[side][u].y, x[2], x[3]);
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) f2_unpack(f2_mul(x[e], s2), f[2 * e], f[2 * e + 1]);
                if (first + u * kGroups + g < L)
                    *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(u) * kGroups * p.hkv * HD) = f32_to_bf16x8(f);
            }
        }
    }
}

// ---- copies of blocks -------------------------------------------------------------------------------------------

// A block's codes (all heads, K and V) are one run of memory, its scales another.  A CTA copies a piece of one block.
constexpr int kCopyThreads = 256;
constexpr int kCopyVectors = 4;               // of 16 bytes a thread

__global__ void __launch_bounds__(kCopyThreads)
    int8_copy_kernel(uint4 *cache, float2 *scales, int64_t num_blocks, int32_t hkv, int32_t vectors, int32_t pieces,
                     const int64_t *mapping, int32_t *status) {
    const int pair = blockIdx.x / pieces, piece = blockIdx.x - pair * pieces;
    const int64_t from = __ldg(mapping + 2 * pair), to = __ldg(mapping + 2 * pair + 1);
    if (from < 0 || from >= num_blocks || to < 0 || to >= num_blocks) {
        if (piece == 0 && threadIdx.x == 0) set_status(status, PKV_ERR_DEVICE_INDEX);
        return;
    }
    if (from == to) return;
    const uint4 *src = cache + from * vectors;
    uint4 *dst = cache + to * vectors;
    const int v0 = piece * kCopyThreads * kCopyVectors + threadIdx.x;
    uint4 v[kCopyVectors];
#pragma unroll
    for (int i = 0; i < kCopyVectors; ++i)
        if (v0 + i * kCopyThreads < vectors) v[i] = src[v0 + i * kCopyThreads];
    if (piece == 0)
        for (int h = threadIdx.x; h < hkv; h += kCopyThreads) scales[to * hkv + h] = scales[from * hkv + h];
#pragma unroll
    for (int i = 0; i < kCopyVectors; ++i)
        if (v0 + i * kCopyThreads < vectors) dst[v0 + i * kCopyThreads] = v[i];
}

// ---- host side ---------------------------------------------------------------------------------------------------

// Checks that every call over the cache makes.
static int check_cache(int64_t num_blocks, int32_t num_kv_heads, int32_t head_size, int32_t block_size) {
    if (num_kv_heads <= 0 || num_blocks <= 0) return PKV_ERR_SHAPE;
    if (block_size != kBlock || (head_size != 64 && head_size != 128)) return PKV_ERR_UNSUPPORTED;
    // a block id and head count as 31 bits each
    if (num_blocks > INT32_MAX || num_kv_heads > (1 << 20)) return PKV_ERR_SHAPE;
    return PKV_OK;
}

static bool misaligned(const void *a, unsigned bytes) { return (reinterpret_cast<uintptr_t>(a) & (bytes - 1)) != 0; }

static int int8_write(Int8WriteParams &p, int form, int32_t head_size, void *stream) {
    // Heads a warp: 16, or two rows a lane where that would put fewer than 16 warps on each of the 152 SMs.  GPU time,
    // two rows a lane against 16 heads: keys and values of 8 heads of 128, one prompt of 100 tokens 2.3 us against 4.3,
    // 600 3.0 against 3.1, 1000 3.5 against 3.4, 2000 4.9 against 4.4, 4000 7.5 against 5.4, of 600 decodes 2.8 against
    // 4.1; queries, keys and values of 32/8 heads, 100 tokens 4.9 against 6.3, 300 6.2 against 5.1, 600 8.1 against
    // 5.7, 1000 11.2 against 8.5, 2046 24.0 against 18.7.  So the two meet at some 1000 warps of 16 heads (prompts;
    // decodes later).
    const int few = 2 * (32 / (head_size / 8));
    auto spread = [&](int heads) {
        p.q_chunks = form ? (p.hq + heads - 1) / heads : 0;
        p.kv_chunks = form ? (p.hkv + heads - 1) / heads : 0;
        p.chunks = form ? p.q_chunks + 2 * p.kv_chunks : (2 * p.hkv + heads - 1) / heads;
        return static_cast<int64_t>(p.num_tokens) * p.chunks;
    };
    int64_t warps = spread(kBlock);
    const bool small = warps < 152 * 16;
    if (small) warps = spread(few);
    if (warps > INT32_MAX - kI8Threads) return PKV_ERR_SHAPE;
    void (*kernel)(Int8WriteParams);
    if (head_size == 128)
        kernel = small ? (form == 0 ? int8_write_kernel<128, 0, 2>
                                    : (form == 1 ? int8_write_kernel<128, 1, 2> : int8_write_kernel<128, 2, 2>))
                       : (form == 0 ? int8_write_kernel<128, 0, 8>
                                    : (form == 1 ? int8_write_kernel<128, 1, 8> : int8_write_kernel<128, 2, 8>));
    else
        kernel = small ? (form == 0 ? int8_write_kernel<64, 0, 2>
                                    : (form == 1 ? int8_write_kernel<64, 1, 2> : int8_write_kernel<64, 2, 2>))
                       : (form == 0 ? int8_write_kernel<64, 0, 4>
                                    : (form == 1 ? int8_write_kernel<64, 1, 4> : int8_write_kernel<64, 2, 4>));
    const unsigned ctas = static_cast<unsigned>((warps + kI8Warps - 1) / kI8Warps);
    kernel<<<ctas, kI8Threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv

extern "C" int pkv_kv_write_int8(void *kv_cache, float *kv_scales, int64_t num_blocks, int32_t num_kv_heads,
                                 int32_t head_size, int32_t block_size, const void *key, int64_t key_token_stride,
                                 const void *value, int64_t value_token_stride, const int64_t *slot_mapping,
                                 int32_t num_tokens, int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_tokens < 0) return PKV_ERR_SHAPE;
    if (const int rc = check_cache(num_blocks, num_kv_heads, head_size, block_size)) return rc;
    if (num_tokens == 0) return PKV_OK;
    if (!kv_cache || !kv_scales || !key || !value || !slot_mapping) return PKV_ERR_NULL;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_size;
    if (key_token_stride < row || value_token_stride < row) return PKV_ERR_SHAPE;
    if ((key_token_stride % 8) || (value_token_stride % 8)) return PKV_ERR_ALIGNMENT;
    if (misaligned(kv_cache, 16) || misaligned(key, 16) || misaligned(value, 16) || misaligned(kv_scales, 8) ||
        misaligned(slot_mapping, 8))
        return PKV_ERR_ALIGNMENT;
    Int8WriteParams p = {};
    p.cache = static_cast<int8_t *>(kv_cache);
    p.scales = kv_scales;
    p.num_blocks = num_blocks;
    p.key = static_cast<const __nv_bfloat16 *>(key);
    p.value = static_cast<const __nv_bfloat16 *>(value);
    p.k_stride = key_token_stride, p.v_stride = value_token_stride;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens, p.hkv = num_kv_heads;
    p.status = device_status;
    return int8_write(p, 0, head_size, stream);
}

extern "C" int pkv_qk_norm_rope_kv_write_int8(void *query_out, int64_t query_out_token_stride, void *kv_cache,
                                              float *kv_scales, int64_t num_blocks, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_size, int32_t block_size,
                                              const void *query, int64_t query_token_stride, const void *key,
                                              int64_t key_token_stride, const void *value, int64_t value_token_stride,
                                              const void *q_weight, const void *k_weight, float eps,
                                              const float *cos_sin, int64_t max_position, int32_t rotary_dim,
                                              int32_t interleaved, const int64_t *positions,
                                              const int64_t *slot_mapping, int32_t num_tokens, int32_t *device_status,
                                              void *stream) {
    using namespace pkv;
    if (num_tokens < 0 || num_q_heads <= 0 || max_position <= 0) return PKV_ERR_SHAPE;
    if (const int rc = check_cache(num_blocks, num_kv_heads, head_size, block_size)) return rc;
    if (rotary_dim < 16 || rotary_dim > head_size || rotary_dim % 16) return PKV_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.0e38f) return PKV_ERR_SHAPE;
    if (num_q_heads > (1 << 20) || max_position > INT64_MAX / rotary_dim / 4) return PKV_ERR_SHAPE;
    if (num_tokens == 0) return PKV_OK;
    if (!query_out || !kv_cache || !kv_scales || !query || !key || !value || !cos_sin || !positions || !slot_mapping)
        return PKV_ERR_NULL;
    const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_size;
    const int64_t kvrow = static_cast<int64_t>(num_kv_heads) * head_size;
    if (query_out_token_stride < qrow || query_token_stride < qrow || key_token_stride < kvrow ||
        value_token_stride < kvrow)
        return PKV_ERR_SHAPE;
    if ((query_out_token_stride % 8) || (query_token_stride % 8) || (key_token_stride % 8) || (value_token_stride % 8))
        return PKV_ERR_ALIGNMENT;
    for (const void *a : {static_cast<const void *>(query_out), static_cast<const void *>(kv_cache), query, key, value,
                          q_weight, k_weight, static_cast<const void *>(cos_sin)})
        if (misaligned(a, 16)) return PKV_ERR_ALIGNMENT;
    if (misaligned(positions, 8) || misaligned(slot_mapping, 8) || misaligned(kv_scales, 8)) return PKV_ERR_ALIGNMENT;
    Int8WriteParams p = {};
    p.cache = static_cast<int8_t *>(kv_cache);
    p.scales = kv_scales;
    p.num_blocks = num_blocks;
    p.key = static_cast<const __nv_bfloat16 *>(key);
    p.value = static_cast<const __nv_bfloat16 *>(value);
    p.k_stride = key_token_stride, p.v_stride = value_token_stride;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens, p.hkv = num_kv_heads;
    p.status = device_status;
    p.query_out = static_cast<__nv_bfloat16 *>(query_out);
    p.out_stride = query_out_token_stride;
    p.query = static_cast<const __nv_bfloat16 *>(query);
    p.q_stride = query_token_stride;
    p.q_weight = static_cast<const __nv_bfloat16 *>(q_weight);
    p.k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.positions = positions;
    p.hq = num_q_heads, p.rot = rotary_dim;
    p.eps = eps;
    return int8_write(p, interleaved ? 2 : 1, head_size, stream);
}

extern "C" int pkv_kv_gather_int8(void *key_out, void *value_out, int64_t out_rows, const void *kv_cache,
                                  const float *kv_scales, int64_t num_blocks, int32_t num_kv_heads, int32_t head_size,
                                  int32_t block_size, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *seq_lens, const int32_t *key_start_loc, int32_t num_seqs,
                                  int32_t max_seq_len, int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || out_rows < 0 || max_seq_len < 0 || max_blocks_per_seq < 0)
        return PKV_ERR_SHAPE;
    if (const int rc = check_cache(num_blocks, num_kv_heads, head_size, block_size)) return rc;
    if (static_cast<int64_t>(max_blocks_per_seq) * kBlock < max_seq_len) return PKV_ERR_SHAPE;
    if (num_seqs == 0) return PKV_OK;
    if (!kv_cache || !kv_scales || !block_tables || !seq_lens || !key_start_loc) return PKV_ERR_NULL;
    if (out_rows && (!key_out || !value_out)) return PKV_ERR_NULL;
    if (misaligned(key_out, 16) || misaligned(value_out, 16) || misaligned(kv_cache, 16) || misaligned(kv_scales, 8) ||
        misaligned(block_tables, 4) || misaligned(seq_lens, 4) || misaligned(key_start_loc, 4))
        return PKV_ERR_ALIGNMENT;
    Int8GatherParams p;
    p.key_out = static_cast<__nv_bfloat16 *>(key_out);
    p.value_out = static_cast<__nv_bfloat16 *>(value_out);
    p.rows = out_rows;
    p.cache = static_cast<const int8_t *>(kv_cache);
    p.scales = kv_scales;
    p.num_blocks = num_blocks;
    p.block_tables = block_tables;
    p.width = max_blocks_per_seq, p.hkv = num_kv_heads, p.max_seq_len = max_seq_len;
    p.seq_lens = seq_lens, p.starts = key_start_loc;
    p.status = device_status;
    // (one CTA a request where none may have rows: the lengths are looked at all the same)
    const int64_t pages = (static_cast<int64_t>(max_seq_len) + kBlock - 1) / kBlock;
    // Pages a CTA: two where there are enough of them, else one.  One page against two: 8 heads of 128, four requests
    // of up to 128 tokens 2.5 us against 3.3, 8 requests of 2048 tokens 17.6 against 19.4, 16 (the bound) 32.2 against
    // 33.1, 32 61.7 against 62.8, 256 of up to 4096 193 against 188; 2 heads, 8 requests 6.0 against 5.2, 16 12.3
    // against 10.6, 32 20.2 against 18.0; 1 head, 16 requests 8.3 against 6.0, 32 15.7 against 12.6 (fewer units than
    // warps in one page).
    p.per = pages * num_seqs > 2048 ? 2 : 1;
    const dim3 grid(static_cast<unsigned>(pages ? (pages + p.per - 1) / p.per : 1), static_cast<unsigned>(num_seqs));
    const cudaError_t e = launch_pdl(head_size == 128 ? int8_gather_kernel<128> : int8_gather_kernel<64>, grid,
                                     dim3(kGatherThreads), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int pkv_copy_blocks_int8(void *kv_cache, float *kv_scales, int64_t num_blocks, int32_t num_kv_heads,
                                    int32_t head_size, int32_t block_size, const int64_t *block_mapping,
                                    int32_t num_pairs, int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_pairs < 0) return PKV_ERR_SHAPE;
    if (const int rc = check_cache(num_blocks, num_kv_heads, head_size, block_size)) return rc;
    if (num_pairs == 0) return PKV_OK;
    if (!kv_cache || !kv_scales || !block_mapping) return PKV_ERR_NULL;
    if (misaligned(kv_cache, 16) || misaligned(kv_scales, 8) || misaligned(block_mapping, 8)) return PKV_ERR_ALIGNMENT;
    const int32_t vectors = num_kv_heads * (2 * kBlock * head_size / 16);      // of a block (at most 2^28)
    const int32_t per = kCopyThreads * kCopyVectors, pieces = (vectors + per - 1) / per;
    const int64_t ctas = static_cast<int64_t>(num_pairs) * pieces;
    if (ctas > INT32_MAX) return PKV_ERR_SHAPE;
    int8_copy_kernel<<<static_cast<unsigned>(ctas), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<uint4 *>(kv_cache), reinterpret_cast<float2 *>(kv_scales), num_blocks, num_kv_heads, vectors,
        pieces, block_mapping, device_status);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
