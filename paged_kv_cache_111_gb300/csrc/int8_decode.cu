// Decode kernel over an int8 cache (int8_common.cuh): split-K and 16-row tiles, as decode.cu does for the other caches
// (the plan that lists its chunks and the combine that merges split rows are theirs too).
//
// With K_j = ks k_j and V_j = vs v_j (codes k_j, v_j, the scales of their block), for a query row q
//     s_j = scale ks <q, k_j>,   out = sum_j 2^(s_j) vs v_j / sum_j 2^(s_j)     (log2 domain)
// Products are f16 mma.sync with the keys as the rows: S^T = K Q^T and O^T = V^T P^T, so that 16 keys or dims fill a
// tile whatever the number of query rows (8 or 16 columns; decode has a few).  Codes widen to f16 exactly: a byte
// next to 0x64 is 1152 + code.  K is left like that, and S starts at -1152 sum q; V has the 1152 taken off (left in, it
// would be most of O).  The query row is scaled by a power of two into f16.
//
// vs goes into the weights, p'_j = 2^(s_j + log2 vs - m), with m 7 below a row's largest s_j + log2 vs (it moves only
// when passed by 2^15): whatever the blocks' scales are, p' fits f16 where it counts.  The sum is that of p' / vs.
//
// A lane has the same 16 (8) dims of four keys of V as its part of V^T and 32 (16) dims of two keys as its part of K:
// whole words of a raw page, which TMA lays out so that no two lanes meet in a bank; P^T goes from the products'
// result to their operand through movmatrix.  No value is staged in shared memory a second time.
//
// What bounds it: memory in large batches (256 requests of up to 4096 keys, 40 heads of 128, with plan and combine: 346
// us, 98% of a copy's rate); in small ones the chain of plan, tables, first pages and partial rows, and some 300
// instructions a page (64 requests of 512 to 2048 keys, 32/4 heads of 64: 17.4 us, 4.9 of them the combine).
#include <mutex>

#include "decode_plan.cuh"
#include "int8_common.cuh"

namespace pkv {

// ROWS: columns of the products, rows of a chunk at most.  Two ring stages a warp: 48 KB (16 columns of 64 dims) to 96
// KB in flight an SM are more than an SM's share of memory's rate times its latency, some 35 KB, and what shared memory
// leaves is L1 (256 requests of 40 heads of 128: 347 us, with three stages 361, with three and a CTA more, of 128
// registers that spill, 382; 64 requests of 512 to 2048 keys, 32/4 heads of 64: 17.7 us, with six stages 20.2; 256
// requests of 64/4 heads of 64: 68.9 us, with three stages 69.4).
constexpr int kInt8Depth = 2;

// CTAs an SM.  Sixteen columns of 128 dims spill at the 168 registers of three; a large batch, which the decode kernel
// does not plan itself, is faster with two (512 requests of 64/4 heads: 167 us, three 186), a small one slower (64: 44
// us, three 32).
constexpr int int8_ctas(int head_size, bool wide, bool self_plan) {
    if (head_size == 64) return wide ? 3 : 4;
    return wide && !self_plan ? 2 : 3;
}

template <int HD, int ROWS, int CTAS>
struct Int8DecodeCfg {
    static constexpr int kStage = 2 * kBlock * HD;           // a raw page of one kv head
    static constexpr int kWarpBytes = kInt8Depth * kStage;
    // (before the rings are used, a plan lies where they are)
    static constexpr int kPlanBytes = ((8 * kSelfPlanSeqs + 1) * 4 + 15) & ~15;
    static constexpr int kOffBar = kDecodeWarps * kWarpBytes > kPlanBytes ? kDecodeWarps * kWarpBytes : kPlanBytes;
    static constexpr int kSmem = kOffBar + kDecodeWarps * kInt8Depth * 8 + 1024;
    static_assert((kSmem + 1024) * CTAS <= 228 * 1024, "the tiling's CTAs fit one SM's shared memory");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {       // an 8 x 8 matrix of 16 bits, transposed
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int HD, int ROWS, int CTAS>
__global__ void __launch_bounds__(kDecodeWarps * 32, CTAS)
    int8_decode_kernel(const __grid_constant__ CUtensorMap kv_map, const AttnParams p) {
    using Cfg = Int8DecodeCfg<HD, ROWS, CTAS>;
    constexpr int NW = kDecodeWarps, DEPTH = kInt8Depth;
    constexpr int KSTEPS = HD / 16;               // of S^T = K Q^T
    constexpr int MT = HD / 16;                   // 16-dim tiles of O^T
    constexpr int NT = ROWS / 8;                  // 8-row tiles of the columns
    constexpr int VW = HD / 32;                   // words of a V row a lane
    // V's words are read when the scores are done (fewer registers at a time: 256 requests of 40 heads 345 -> 343 us,
    // 512 of 64/4 heads 191 -> 186), of 64 dims at once (256 requests of 32 heads: 256 us, 260 so)
    constexpr bool kLateV = HD == 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * Cfg::kWarpBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kOffBar) + warp * DEPTH;
    const uint32_t ring_u32 = smem_u32(ring);
    if (lane < DEPTH) mbar_init(&bars[lane], 1);
    if (threadIdx.x == 0) tma_prefetch_desc(&kv_map);
    fence_barrier_init();
    __syncwarp();
    WsHeader *hdr = reinterpret_cast<WsHeader *>(p.ws);
    int32_t *status = reinterpret_cast<int32_t *>(p.ws);
    __shared__ SelfPlanShared sp_shared;
    SelfChunk self_chunks[2];
    int n_items = 0;
    if (p.self_plan) {                            // (uniform over the CTA; see decode_plan.cuh)
        const bool warp_plan = p.num_seqs <= 32 * kWarpPlanPer && blockIdx.x != gridDim.x - 1;
        if (warp_plan)
            n_items = decode_warp_plan(p, self_chunks, (gridDim.x - 1) * NW, blockIdx.x * NW + warp);
        else
            n_items = decode_self_plan<NW>(p, reinterpret_cast<int *>(smem), sp_shared, self_chunks);
        pdl_wait();                               // the cache write before this kernel is complete
        if (blockIdx.x == gridDim.x - 1) {
            decode_self_plan_publish<NW>(p, reinterpret_cast<const int *>(smem), sp_shared);
            pdl_trigger();
            return;
        }
        if (!warp_plan) {
            __syncthreads();                      // the plan's shared memory is the rings' from here on
            fence_proxy_async_smem();
        }
    } else {
        pdl_wait();                               // the plan (and the cache write before it) are complete
    }
    pdl_trigger();
    // an error of a self-planned call is stored once the last CTA has reset the status
    const int epoch0 = p.self_plan ? *reinterpret_cast<volatile int32_t *>(&hdr->epoch) : 0;
    auto report = [&](int32_t code) {
        if (p.self_plan) {
            const uint64_t t0 = global_ns();
            while (*reinterpret_cast<volatile int32_t *>(&hdr->epoch) == epoch0 && global_ns() - t0 < kWaitLimitNs) {
            }
        }
        set_status(status, code);
    };
    const int4 *req = reinterpret_cast<const int4 *>(p.ws + p.lay.off_req);
    const int4 *chunks = reinterpret_cast<const int4 *>(p.ws + p.lay.off_chunks);
    float *part_lse = reinterpret_cast<float *>(p.ws + p.lay.off_part_lse);
    float *part_o = reinterpret_cast<float *>(p.ws + p.lay.off_part_o);
    if (!p.self_plan) n_items = __ldcg(&hdr->n_chunks) * p.num_kv_heads;

    const int W = (p.self_plan ? gridDim.x - 1 : gridDim.x) * NW;
    const int wid = blockIdx.x * NW + warp;
    uint32_t st = 0, par = 0;                     // this warp's next ring stage, and its barrier's phase there
    const int g4 = lane >> 2, t4 = lane & 3;
    const float NEG_INF = -__int_as_float(0x7f800000);
    // the sign of the scale goes into the query, so that the largest score has the largest weight
    const float sl2 = fabsf(p.scale_log2), flip = p.scale_log2 < 0.f ? -1.f : 1.f;

    for (int round = 0; round * W < n_items; ++round) {
        const int item = (round & 1) ? round * W + (W - 1 - wid) : round * W + wid;   // snake order
        if (item >= n_items) continue;
        const SelfChunk sc = (round & 1) ? self_chunks[1] : self_chunks[0];
        const int4 ch = p.self_plan ? make_int4(sc.r, sc.k, sc.pb, sc.pb + sc.npages)
                                    : __ldcg(chunks + item / p.num_kv_heads);
        const int g = item % p.num_kv_heads;
        const int r = ch.x;
        const int pb = ch.z;
        const int npages = ch.w - ch.z;
        const int32_t *bt = p.block_tables + static_cast<int64_t>(r) * p.max_blocks_per_seq + pb;
        // windows of 32 pages: lane l holds page (window + l)'s block, and of that block's scales K's, and log2 of V's;
        // the next window's come while this one is at work
        auto blocks_of = [&](int first) { return first + lane < npages ? bt[first + lane] : -1; };
        auto scales_of = [&](int blk) {
            float2 s = make_float2(0.f, 0.f);
            if (blk >= 0 && blk < p.num_blocks)
                s = reinterpret_cast<const float2 *>(p.kv_scales)[static_cast<int64_t>(blk) * p.num_kv_heads + g];
            return s;
        };
        float ks_win, lv_win;
        auto scales_in = [&](float2 s) {
            ks_win = s.x, lv_win = __log2f(s.y < kInt8LeastScale ? kInt8LeastScale : s.y);      // (NaN stays)
        };
        int wbase = 0;
        int win = blocks_of(0), win_next = blocks_of(32);
        const int L = p.seq_lens[r];
        const int qs = p.qsl[r];
        const int qlen = p.qsl[r + 1] - qs;
        const int ctx = L - qlen;
        const int rows_total = qlen * p.G;
        const bool split_mode = rows_total <= 16;
        const int tile = split_mode ? 0 : ch.y;
        const int split = split_mode ? ch.y : 0;
        const int4 info = p.self_plan ? make_int4(sc.n_split, sc.pbase, 0, 0) : __ldcg(req + r);
        const int n_split = split_mode ? info.x : 1;
        const int rows = min(16, rows_total - 16 * tile);

        auto issue = [&](uint32_t stage, int blk) {               // a page of this chunk -> its ring stage
            if (lane == 0) {
                if (blk < 0 || blk >= p.num_blocks) report(PKV_ERR_DEVICE_INDEX);   // (read as zeros)
                mbar_arrive_expect_tx(&bars[stage], Cfg::kStage);
                tma_load_5d(ring + stage * Cfg::kStage, &kv_map, &bars[stage], 0, 0, 0, g, blk);
            }
        };
        int issued = min(DEPTH, npages);
        for (int k = 0; k < issued; ++k)
            issue(st + k < DEPTH ? st + k : st + k - DEPTH, __shfl_sync(0xffffffffu, win, k));
        const float2 scale_first = scales_of(win);
        float2 scale_next = make_float2(0.f, 0.f);
        // query token and head of the group of the tile's row R
        auto place_of = [&](int R) {
            const int row = 16 * tile + R;
            if (qlen == 1) return make_int2(0, row);
            return make_int2(row / p.G, row % p.G);
        };

        // the query rows this lane holds dims of: g4, and g4 + 8.  Lane column t4 takes dims t4 HD/4 .. of a row, four
        // a k-step, so that its part of a key is whole words of the page (the order of a product's terms is free)
        uint32_t qf[NT][KSTEPS][2];
        float bias[NT], factor[NT];               // of row g4 (+ 8): -1152 sum q, and what brings S to log2 units
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int R = g4 + 8 * nt;
            const int2 at = place_of(R);
            const __nv_bfloat16 *qp = p.query + static_cast<int64_t>(qs + at.x) * p.q_stride +
                                      static_cast<int64_t>(g * p.G + at.y) * HD + t4 * (HD / 4);
#pragma unroll
            for (int kk = 0; kk < KSTEPS; kk += 2) {
                const uint4 v = R < rows ? *reinterpret_cast<const uint4 *>(qp + 4 * kk) : make_uint4(0, 0, 0, 0);
                qf[nt][kk][0] = v.x, qf[nt][kk][1] = v.y, qf[nt][kk + 1][0] = v.z, qf[nt][kk + 1][1] = v.w;
            }
            float a = 0.f;
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    a = fmaxf(a, fmaxf(fabsf(__uint_as_float(qf[nt][kk][e] << 16)),
                                       fabsf(__uint_as_float(qf[nt][kk][e] & 0xFFFF0000u))));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            // into [2^14, 2^15): exact but for parts below 2^-24 of the row's largest; the exponent is held where
            // 2^e and 2^-e are normal
            const int e2 = a > 0.f ? min(126, max(-114, 14 - ilogbf(a))) : 0;
            const float up = __int_as_float((e2 + 127) << 23) * flip;
            float sum = 0.f;
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w = qf[nt][kk][e];
                    const __half2 h =
                        __floats2half2_rn(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
                    const float2 f = __half22float2(h);
                    sum += f.x + f.y;
                    qf[nt][kk][e] = *reinterpret_cast<const uint32_t *>(&h);
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            bias[nt] = -kInt8Bias * sum;
            factor[nt] = sl2 * __int_as_float((127 - e2) << 23);
        }
        // the query rows whose scores this lane holds: 2 t4 and 2 t4 + 1 (+ 8)
        float S0[NT][2], sf[NT][2], m[NT][2], l[NT][2];
        int lim[NT][2], lim_least = INT32_MAX;    // keys [0, lim) visible; a row that is none sees all (for nobody)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int R = 2 * t4 + e;
                S0[nt][e] = __shfl_sync(0xffffffffu, bias[nt], 4 * R);
                sf[nt][e] = __shfl_sync(0xffffffffu, factor[nt], 4 * R);
                m[nt][e] = NEG_INF, l[nt][e] = 0.f;
                lim[nt][e] = R + 8 * nt < rows ? ctx + place_of(R + 8 * nt).x + 1 : INT32_MAX;
                lim_least = min(lim_least, lim[nt][e]);
            }
        lim_least = __reduce_min_sync(0xffffffffu, lim_least);

        float o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
        int failed_at = -1;

        scales_in(scale_first);

        for (int k = 0; k < npages; ++k) {
            const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], par));
            if (!ok) {
                failed_at = k;
                break;
            }
            const uint32_t page = ring_u32 + st * Cfg::kStage;
            // this lane's words: dims t4 HD/4 .. of keys g4 and g4 + 8; dims g4 HD/8 .. of V's keys 2 t4, + 1, + 8, + 9
            uint32_t kw[2][KSTEPS], vw[4][VW];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int row = g4 + 8 * n;
#pragma unroll
                for (int v = 0; v < KSTEPS / 4; ++v) {
                    // 16-byte piece c of row R lies at c ^ (R & 7) (HD 128), at c ^ (R / 2 & 3) (HD 64)
                    const int c = HD == 128 ? (2 * t4 + v) ^ (row & 7) : t4 ^ ((row >> 1) & 3);
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(kw[n][4 * v]), "=r"(kw[n][4 * v + 1]), "=r"(kw[n][4 * v + 2]),
                                   "=r"(kw[n][4 * v + 3])
                                 : "r"(page + row * HD + c * 16));
                }
            }
            auto load_v = [&]() {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int row = kBlock + 2 * t4 + (n & 1) + 8 * (n >> 1);
                    if constexpr (HD == 128) {
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(vw[n][0]), "=r"(vw[n][1]), "=r"(vw[n][2]), "=r"(vw[n][3])
                                     : "r"(page + row * HD + ((g4 ^ (row & 7)) << 4)));
                    } else {
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(vw[n][0]), "=r"(vw[n][1])
                                     : "r"(page + row * HD + (((g4 >> 1) ^ ((row >> 1) & 3)) << 4) + (g4 & 1) * 8));
                    }
                }
            };
            auto release = [&]() {
                // the page is in registers: its stage goes back to the copy engine
                fence_proxy_async_smem();
                __syncwarp();
                if (k - wbase == 32) {
                    wbase += 32;
                    win = win_next;
                    scales_in(scale_next);
                    win_next = blocks_of(wbase + 32);
                }
                if (k - wbase == 16) scale_next = scales_of(win_next);
                const int nk = k + DEPTH;
                if (nk < npages) {
                    const int at = nk - wbase;
                    issue(st, __shfl_sync(0xffffffffu, at < 32 ? win : win_next, at & 31));
                    ++issued;
                }
                if (++st == DEPTH) st = 0, par ^= 1u;
            };
            if (!kLateV) {
                load_v();
                release();
            }
            const int j0 = (pb + k) * kBlock;     // first key of this page
            const bool masked = j0 + kBlock > lim_least;               // (uniform over the warp)

            // S^T: keys g4, g4 + 8 by rows 2 t4, + 1
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][2] = S0[nt][0], s[nt][1] = s[nt][3] = S0[nt][1];
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
                uint32_t a[4];
                int8x4_to_biased_f16(kw[0][kk], a[0], a[2]);
                int8x4_to_biased_f16(kw[1][kk], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt], a, qf[nt][kk][0], qf[nt][kk][1]);
            }
            if (kLateV) {
                load_v();
                release();
            }
            const float ks = __shfl_sync(0xffffffffu, ks_win, k - wbase);
            const float lv = __shfl_sync(0xffffffffu, lv_win, k - wbase);
            const float vr = fast_exp2(-lv);      // (1 / vs with lv's own rounding, which so falls out of the weights)

            // s + log2 vs above the row's reference
            float x[NT][4];
            auto above = [&]() {
                bool passed = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[nt][e] = fmaf(s[nt][e], sf[nt][e & 1] * ks, lv - m[nt][e & 1]);
                        if (masked) x[nt][e] = j0 + g4 + 8 * (e >> 1) < lim[nt][e & 1] ? x[nt][e] : NEG_INF;
                        passed |= x[nt][e] > kInt8DecodeMost;
                    }
                return passed;
            };
            if (__any_sync(0xffffffffu, above())) {
                // the first key that a row sees, or one that passes its reference by 2^15: the reference moves to 7
                // below the largest
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = sf[nt][e] * ks;
                        float y0 = fmaf(s[nt][e], f, lv), y1 = fmaf(s[nt][e + 2], f, lv);
                        if (masked) {
                            y0 = j0 + g4 < lim[nt][e] ? y0 : NEG_INF;
                            y1 = j0 + g4 + 8 < lim[nt][e] ? y1 : NEG_INF;
                        }
                        float mx = fmaxf(y0, y1);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        if (mx > m[nt][e] + kInt8DecodeMost) {              // (the same in the lanes of a row)
                            const float alpha = fast_exp2(m[nt][e] - (mx - kInt8DecodeLift));      // 0 when m = -inf
                            m[nt][e] = mx - kInt8DecodeLift;
                            l[nt][e] *= alpha;
#pragma unroll
                            for (int i = 0; i < MT; ++i) o[nt][i][e] *= alpha, o[nt][i][e + 2] *= alpha;
                        }
                    }
                above();
            }
            uint32_t pb0[NT], pb1[NT];            // P^T: keys 2 t4, + 1 (+ 8, + 9) by row g4
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float pr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[e] = fast_exp2(x[nt][e]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (a row that sees none of the page's keys: not 0 times a scale that is no number)
                    const float inv = masked && j0 >= lim[nt][e] ? 0.f : vr;
                    l[nt][e] = fmaf(pr[e] + pr[e + 2], inv, l[nt][e]);
                }
                // one f16 a weight: off by 2^-11 of it (an eighth of the output's rounding to bf16) and 2^-32 of the
                // row's largest at most
                pb0[nt] = movmatrix(pack_f16x2(pr[0], pr[1]));
                pb1[nt] = movmatrix(pack_f16x2(pr[2], pr[3]));
            }
            // O^T += V^T P^T: tile i's rows g4, g4 + 8 are this lane's dims 2 i, 2 i + 1
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int v = 0; v < VW; ++v) vw[n][v] ^= 0x80808080u;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                const uint32_t lo = prmt(vw[0][i >> 1], vw[1][i >> 1], sel);
                const uint32_t hi = prmt(vw[2][i >> 1], vw[3][i >> 1], sel);
                const uint32_t top = 0x64646464u;
                const uint32_t a[4] = {unbias_f16(prmt(lo, top, 0x4140)), unbias_f16(prmt(lo, top, 0x4342)),
                                       unbias_f16(prmt(hi, top, 0x4140)), unbias_f16(prmt(hi, top, 0x4342))};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][i], a, pb0[nt], pb1[nt]);
            }
        }

        if (failed_at >= 0) {
            report(PKV_ERR_DEVICE_TIMEOUT);
            // let copies already in flight land before the CTA's memory is released
            for (int k = failed_at; k < issued; ++k) {
                mbar_wait_bounded(&bars[st], par);
                if (++st == DEPTH) st = 0, par ^= 1u;
            }
            return;
        }

        const float LN2 = 0.69314718055994531f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int R = 2 * t4 + e + 8 * nt;
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (R >= rows) continue;
                const float inv = sum <= 0.f ? 0.f : 1.f / sum;         // (NaN stays)
                const int2 at = place_of(R);
                const int i = at.x, h = g * p.G + at.y;
                if (n_split <= 1) {
                    uint32_t w[MT];
#pragma unroll
                    for (int v = 0; v < MT; ++v) w[v] = pack_bf16x2(o[nt][v][e] * inv, o[nt][v][e + 2] * inv);
                    __nv_bfloat16 *dst =
                        p.out + (static_cast<int64_t>(qs + i) * p.num_q_heads + h) * HD + g4 * (HD / 8);
#pragma unroll
                    for (int v = 0; v < MT; v += 4)
                        *reinterpret_cast<uint4 *>(dst + 2 * v) = make_uint4(w[v], w[v + 1], w[v + 2], w[v + 3]);
                } else {
                    const int64_t prow = info.y + (static_cast<int64_t>(i) * p.num_q_heads + h) * n_split + split;
                    float *dst = part_o + prow * HD + g4 * (HD / 8);
#pragma unroll
                    for (int v = 0; v < MT; v += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * v) =
                            make_float4(o[nt][v][e] * inv, o[nt][v][e + 2] * inv, o[nt][v + 1][e] * inv,
                                        o[nt][v + 1][e + 2] * inv);
                    // (a sum that is no number: a finite weight, so that the merge meets the part's NaN)
                    if (g4 == 0)
                        part_lse[prow] = sum != sum ? 0.f : (sum > 0.f ? (m[nt][e] + __log2f(sum)) * LN2 : NEG_INF);
                }
            }
    }
}

// ---- host side --------------------------------------------------------------------

// The cache as a 5-D tensor of bytes {head_size, 16, 2, Hkv, num_blocks}: a box is a page of one kv head, its 16-byte
// pieces permuted within eight rows (head size 128) or eight half rows (64).
int make_int8_map(CUtensorMap *map, const void *kv_cache, int64_t num_blocks, int32_t num_kv_heads, int32_t head_size) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(head_size), kBlock, 2, static_cast<cuuint64_t>(num_kv_heads),
                                static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t row = static_cast<cuuint64_t>(head_size);
    const cuuint64_t strides[4] = {row, row * kBlock, row * kBlock * 2, row * kBlock * 2 * num_kv_heads};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(head_size), kBlock, 2, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(kv_cache), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, head_size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

int int8_decode_ctas_per_sm(int32_t head_size, int rows, bool self_plan) {
    return int8_ctas(head_size, rows > 8, self_plan);
}

template <int HD, int ROWS, int CTAS>
static int launch_int8_decode(const CUtensorMap &map, const AttnParams &p, int grid, int dev, cudaStream_t stream) {
    using Cfg = Int8DecodeCfg<HD, ROWS, CTAS>;
    static std::mutex mu;
    static uint64_t done_mask = 0;                // devices whose shared-memory limit is already raised
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (!bit || !(done_mask & bit)) {
            if (cudaFuncSetAttribute(int8_decode_kernel<HD, ROWS, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Cfg::kSmem) != cudaSuccess)
                return PKV_ERR_CUDA;
            done_mask |= bit;
        }
    }
    return launch_pdl(int8_decode_kernel<HD, ROWS, CTAS>, dim3(grid), dim3(kDecodeWarps * 32), Cfg::kSmem, stream, map, p) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

int launch_int8_decode_path(const CUtensorMap &map, const AttnParams &p, int32_t head_size, int rows, int grid, int dev,
                            cudaStream_t st) {
    if (head_size == 64)
        return rows <= 8 ? launch_int8_decode<64, 8, int8_ctas(64, false, false)>(map, p, grid, dev, st)
                         : launch_int8_decode<64, 16, int8_ctas(64, true, false)>(map, p, grid, dev, st);
    if (rows <= 8) return launch_int8_decode<128, 8, int8_ctas(128, false, false)>(map, p, grid, dev, st);
    return p.self_plan ? launch_int8_decode<128, 16, int8_ctas(128, true, true)>(map, p, grid, dev, st)
                       : launch_int8_decode<128, 16, int8_ctas(128, true, false)>(map, p, grid, dev, st);
}

}  // namespace pkv
