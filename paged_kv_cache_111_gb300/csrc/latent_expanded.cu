// Causal attention over per-head keys and values that were expanded from latent
// rows (the expanded form of latent attention), on the 5th-generation tensor
// cores.
//
// Request r owns query tokens [query_start_loc[r], [r + 1]) (q of them) and keys
// [key_start_loc[r], [r + 1]) (L >= q); its i-th query sees keys 0 .. L - q + i.
// For head h, with query rows of 128 plain and 64 rotated dims,
//     s_j       = scale (<query[t][h][0 .. 127], key[j][h]> + <query[t][h][128 ..], key_rope[j]>)
//     out[t][h] = sum_j softmax_j(s_j) value[j][h]
// The rotated part of a key is one row for all heads and is read as such: the
// 192-wide keys of each head are put together in shared memory only.
//
// A CTA takes 256 tokens of one head of one request as two 128-row tiles that
// share every key tile.  Per 128-key tile and row tile: S = Q K^T (12
// tcgen05.mma 128 x 128 x 16, shared memory), softmax by four warps (a row per
// thread), P as bf16 over S in tensor memory, O += P V (8 tcgen05.mma 128 x 128
// x 16, P from tensor memory).  The two row tiles take turns: while one's
// softmax works, the tensor cores have the other's products.  Tensor memory: S
// of both tiles, O of both tiles (512 columns).  Shared memory: Q of both (96
// KiB) and a ring of eight 16 KiB slots, filled and released in the order of use,
// five a key tile: K's three 64-dim chunks, then V's two halves of 64 keys.  Each
// slot is loaded again when the second row tile's product has read it, a key
// tile's time or so before it is used again.  (K in two whole stages and V in one
// left V's load, about 1500 cycles, in the way of every tile: 7% of the time of 2048
// tokens at 8192 keys of 128 heads.)
//
// Against the latent-space form this does (128 + 64 + 128) / (576 + 512) = 0.29
// of the products per visible pair, and reads keys per head: the form for long
// chunks, where a key is used by many rows.
//
// Warp roles (384 threads): warp 0 loads by TMA, warp 1 issues the MMAs, warp 2
// owns tensor memory, warps 2 and 3 look V over where the causal mask cuts through a
// key tile, warps 4-7 and 8-11 are the softmax and epilogue of the
// two row tiles.  V rows past the last visible key are zeroed in shared memory
// (they belong to other requests, or to nobody).  Every mbarrier wait is bounded; that for the
// diagonal, which may be all of a long request away, by the key tiles loaded meanwhile.
//
// Where token tiles are few, the CTAs of a cluster share a tile's keys and join their
// sums through distributed shared memory (the rule and its figures: at the launch).
//
// What bounds it: per key tile and CTA about 3470 cycles, of which the products take
// 40 x 65 = 2600 on the tensor cores and their operands' way out of shared memory 2670
// (128 bytes a cycle); the rest is the turn between the two row tiles.  2048 tokens at
// 8192 keys of 128 heads (1.2 TFLOP): 790 us with cold caches, 1520 TFLOP/s, 78% of the
// dense bf16 rate; 725 us back to back.  Three requests of 300 to 2046 tokens of 16 heads
// (21 GFLOP): 33.4 to 36 us, the 16 key tiles of the longest one's last tokens one after another.
#include <mutex>

#include "latent_common.cuh"
#include "prefill_common.cuh"

namespace pkv {

constexpr int kExNope = 128, kExDim = kExNope + kLatRope, kExV = 128;
constexpr int kExRows = 128, kExKeys = 128;             // of a row tile, of a key tile
constexpr int kExTokens = 2 * kExRows;                  // of a CTA
constexpr int kExChunk = 128 * 128;                     // 64 dims of 128 rows: 16 KiB
constexpr int kExQ = 3 * kExChunk;
constexpr int kExSlots = 8, kExPerTile = 5;             // ring slots; of a key tile: K chunks 0-2, V halves 0-1
constexpr int kExThreads = 384;

constexpr int kExOffQ = 0;
constexpr int kExOffRing = kExOffQ + 2 * kExQ;
constexpr int kExOffBar = kExOffRing + kExSlots * kExChunk;   // 229376
constexpr int kExSmem = kExOffBar + 512 + 1024;         // with alignment slack
static_assert(kExSmem <= 227 * 1024, "shared memory of one CTA");

enum ExBar {
    kExQFull = 0,        // (+ row tile)
    kExFull = 2,         // (+ slot)
    kExEmpty = 10,       // (+ slot)
    kExFix = 18,         // V rows past the last visible key zeroed
    kExSFull = 19,       // (+ row tile)
    kExPFull = 21,       // (+ row tile)
    kExODone = 23,       // (+ row tile)
    kExLoaded = 25,      // V's loads of a tile on the causal diagonal are on their way (+ its number & 1)
    kExChecked = 27,     // V of that tile looked through (+ its number & 1)
    kExNumBars = 29
};
static_assert(kExNumBars * 8 + 8 + 20 * 4 <= 512, "barriers, tensor-memory address, scan");

struct ExParams {
    __nv_bfloat16 *out;
    const int32_t *qsl, *ksl;
    int32_t num_seqs, num_tokens, num_keys, max_query_len, max_key_len, heads;
    int32_t tiles;            // upper bound of the CTAs' token tiles over all requests
    int32_t by_head;          // order of the CTAs: all token tiles of one head, then the next
    int32_t split;            // CTAs (a cluster) that share the keys of a token tile: 1, 2 or 4
    float scale_log2;
    int32_t *status;
};

struct ExReq {
    int32_t qs, q, ks, L;
    bool ok;
};
__device__ __forceinline__ ExReq ex_request(const ExParams &p, int r) {
    ExReq a;
    a.qs = __ldg(p.qsl + r);
    a.q = __ldg(p.qsl + r + 1) - a.qs;
    a.ks = __ldg(p.ksl + r);
    a.L = __ldg(p.ksl + r + 1) - a.ks;
    a.ok = a.qs >= 0 && a.q >= 0 && a.qs + a.q <= p.num_tokens && a.ks >= 0 && a.L >= a.q &&
           a.ks + a.L <= p.num_keys && a.q <= p.max_query_len && a.L <= p.max_key_len;
    return a;
}

// Where the keys of a token tile are shared out over a cluster: partial sums on their way
// between its CTAs, over Q and the ring, as [CTA][group][dim / 4][row][dim % 4] of 32 rows a
// group, and behind them the rows' {reference, sum}.
constexpr uint32_t kExGroupBytes = 32 * kExV * 4;
constexpr uint32_t kExOffState = 8 * kExGroupBytes;
constexpr uint32_t kExOffStage = kExOffState + 2048;     // finished rows, 32 x 64 dims a warp
static_assert(8 * 32 * 8 <= 2048 && kExOffStage + 8 * 4096 <= kExOffBar, "the partial sums' place");

// Every thread of the cluster's CTAs comes here.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The address of this CTA's shared memory word `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// A warp's 32 finished rows of P 16-byte pieces on their way out: from the lanes, a row each,
// into shared memory, and from there in whole rows.  (Stored by the lanes, 16 bytes to 32
// rows at a time, a row tile's end took 1.5 us instead of 1.0.)
template <int P>
__device__ __forceinline__ void ex_stage(uint8_t *stage, int lane, int piece, const float (&y)[8], float inv) {
    *reinterpret_cast<uint4 *>(stage + lane * (16 * P) + ((piece ^ (lane & 7 & (P - 1))) << 4)) =
        make_uint4(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv),
                   pack_bf16x2(y[4] * inv, y[5] * inv), pack_bf16x2(y[6] * inv, y[7] * inv));
}
template <int P>
__device__ __forceinline__ void ex_store(const uint8_t *stage, int lane, int rows, __nv_bfloat16 *out, int64_t stride) {
    __syncwarp();
    const int piece = lane % P;
#pragma unroll 4
    for (int r = lane / P; r < rows; r += 32 / P)
        *reinterpret_cast<uint4 *>(out + r * stride + piece * 8) =
            *reinterpret_cast<const uint4 *>(stage + r * (16 * P) + ((piece ^ (r & 7 & (P - 1))) << 4));
}

// One row a lane, 128 / C dims a warp (loops kept short: this runs once, from a cold
// instruction cache): out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the cluster's C
// CTAs.  A state that saw no key has m = -inf, and whatever its sums hold is not used.
template <int C>
__device__ __forceinline__ void ex_join(const uint8_t *smem, int group, int d0, int lane, uint8_t *stage) {
    constexpr int kPer = 8 / C, kPieces = kExV / C / 8;
    const float NEG_INF = -__int_as_float(0x7f800000);
    float f[C], M = NEG_INF, L = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        f[c] = *reinterpret_cast<const float *>(smem + kExOffState + ((c * kPer + group) * 32 + lane) * 8);
        M = fmaxf(M, f[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        f[c] = f[c] == NEG_INF ? 0.f : fast_exp2(f[c] - M);
        if (f[c] != 0.f)
            L += f[c] * *reinterpret_cast<const float *>(smem + kExOffState + ((c * kPer + group) * 32 + lane) * 8 + 4);
    }
    const float inv = L <= 0.f ? 0.f : 1.f / L;             // (NaN stays)
#pragma unroll 1
    for (int d = 0; d < kPieces; ++d) {
        float y[8] = {};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint8_t *at = smem + (c * kPer + group) * kExGroupBytes + (d0 / 4 + 2 * d) * 512 + lane * 16;
            const float4 a = *reinterpret_cast<const float4 *>(at), b = *reinterpret_cast<const float4 *>(at + 512);
            if (f[c] != 0.f) {
                y[0] = fmaf(f[c], a.x, y[0]), y[1] = fmaf(f[c], a.y, y[1]);
                y[2] = fmaf(f[c], a.z, y[2]), y[3] = fmaf(f[c], a.w, y[3]);
                y[4] = fmaf(f[c], b.x, y[4]), y[5] = fmaf(f[c], b.y, y[5]);
                y[6] = fmaf(f[c], b.z, y[6]), y[7] = fmaf(f[c], b.w, y[7]);
            }
        }
        ex_stage<kPieces>(stage, lane, d, y, inv);
    }
}

__global__ void __launch_bounds__(kExThreads, 1)
    latent_expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                           const __grid_constant__ CUtensorMap r_map, const __grid_constant__ CUtensorMap v_map,
                           const ExParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kExOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kExNumBars);
    int32_t *scan = reinterpret_cast<int32_t *>(tmem_slot + 2);       // 12 warps' sums, then {request, tile}
    int32_t *odd_key = scan + 18;                                     // first key whose V is no number (on the diagonal)
    volatile int32_t *tiles = scan + 19;                              // key tiles loaded
    const uint32_t sQ = smem_u32(smem + kExOffQ), sRing = smem_u32(smem + kExOffRing);
    const int warp = uniform(static_cast<int>(threadIdx.x) >> 5), lane = threadIdx.x & 31;
    // Token tiles (256 tokens of a request) are ranked by the key tiles they see, the
    // most first, so that the longest are not the last to end; a CTA takes one rank of
    // one head, all heads of a rank or all ranks of a head after one another.
    const int part = blockIdx.x % p.split, item = blockIdx.x / p.split;
    const int head = p.by_head ? item / p.tiles : item % p.heads;
    const int rank = p.by_head ? item % p.tiles : item / p.heads;
    int32_t *status = p.status;

    pdl_trigger();
    // sum over the block
    auto block_sum = [&](int v) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (lane == 0) scan[warp] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < kExThreads / 32; ++w) v += scan[w];
        __syncthreads();
        return v;
    };
    const ExReq mine = threadIdx.x < p.num_seqs ? ex_request(p, threadIdx.x) : ExReq{};
    auto request = [&](int r) { return r < kExThreads ? mine : ex_request(p, r); };    // (r: one of this thread's)
    // token tiles of a request that see w key tiles or more
    auto tiles_from = [&](const ExReq &a, int w) {
        const int keys = (w - 1) * kExKeys + 1, n = (a.q + kExTokens - 1) / kExTokens;
        if (!a.ok || a.q == 0 || a.L < keys) return 0;
        const int first = max(0, (keys - (a.L - a.q) + kExTokens - 1) / kExTokens - 1);    // (but for the last)
        return max(n - first, 1);
    };
    auto count = [&](int w) {
        int c = 0;
        for (int r = threadIdx.x; r < p.num_seqs; r += kExThreads) c += tiles_from(request(r), w);
        return block_sum(c);
    };
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < p.num_seqs; r += kExThreads)
            if (!request(r).ok) set_status(status, PKV_ERR_DEVICE_METADATA);
    // A CTA without a tile waits for the kernel before this one all the same: in a call where
    // none has one, this grid would otherwise be over before that kernel, and a kernel that
    // waits for this grid would take that one's writes for complete.
    int r = 0, t0 = 0;                                  // request; first token, within it
    if (p.num_seqs == 1) {
        const ExReq a = ex_request(p, 0);
        const int n = a.ok ? (a.q + kExTokens - 1) / kExTokens : 0;
        if (rank >= n) {                                // the bound was not reached: uniform
            pdl_wait();
            return;
        }
        t0 = (n - 1 - rank) * kExTokens;
    } else {
        const int all = count(1);
        if (rank >= all) {
            pdl_wait();
            return;
        }
        // the key tiles of this rank's token tile: the largest w with more than `rank`
        // tiles from w on
        int lo = 1, hi = (p.max_key_len + kExKeys - 1) / kExKeys, above = 0;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2, c = count(mid);
            if (c > rank) lo = mid;
            else hi = mid - 1, above = c;
        }
        if (lo == (p.max_key_len + kExKeys - 1) / kExKeys) above = 0;
        // the (rank - above)-th of those with exactly lo, in the requests' order
        int base = above;
        for (int r0 = 0; r0 < p.num_seqs; r0 += kExThreads) {
            const int r = r0 + threadIdx.x;
            int here = 0, from = 0;
            if (r < p.num_seqs) {
                const ExReq a = request(r);
                from = tiles_from(a, lo);
                here = from - tiles_from(a, lo + 1);
            }
            int inc = here;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += y;
            }
            if (lane == 31) scan[warp] = inc;
            __syncthreads();
            int before = base + inc - here, total = base;
#pragma unroll
            for (int w = 0; w < kExThreads / 32; ++w) {
                if (w < warp) before += scan[w];
                total += scan[w];
            }
            if (rank >= before && rank < before + here) {
                scan[16] = r;
                scan[17] = (request(r).q + kExTokens - 1) / kExTokens - from + rank - before;
            }
            base = total;
            __syncthreads();
            if (base > rank) break;
        }
        r = scan[16];
        t0 = scan[17] * kExTokens;
    }
    const ExReq req = ex_request(p, r);
    const int ctx = req.L - req.q;
    // rows and key tiles of the two row tiles
    const int rows[2] = {min(kExRows, req.q - t0), max(0, min(kExRows, req.q - t0 - kExRows))};
    const int seen[2] = {(ctx + t0 + rows[0] + kExKeys - 1) / kExKeys,
                         rows[1] ? (ctx + t0 + kExRows + rows[1] + kExKeys - 1) / kExKeys : 0};
    const int seen_all = max(seen[0], seen[1]);
    // of these, [j0, j1) are this CTA's, and counted from j0 from here on
    const int j0 = static_cast<int>(static_cast<int64_t>(seen_all) * part / p.split);
    const int j1 = static_cast<int>(static_cast<int64_t>(seen_all) * (part + 1) / p.split);
    const int n[2] = {max(0, min(seen[0], j1) - j0), max(0, min(seen[1], j1) - j0)};
    const int n_all = j1 - j0;                          // (the later row tile sees them all)
    const int end = ctx + t0 + rows[0] + rows[1];       // keys the last row sees
    const bool fix = n_all > 0 && j1 == seen_all && end % kExKeys != 0;
    // first key that the first row does not see, and the first tile (if any) with such keys
    const int edge = ctx + t0 + 1, diag = edge < end ? max(0, edge / kExKeys - j0) : n_all;

    if (threadIdx.x == 0) *odd_key = INT32_MAX, *tiles = 0;
    if (threadIdx.x < kExNumBars)
        mbar_init(&bars[threadIdx.x], threadIdx.x >= kExPFull && threadIdx.x < kExPFull + 2 ? 4 : (threadIdx.x >= kExChecked ? 2 : 1));
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    pdl_wait();                                         // the inputs are complete

    if (warp == 0) {
        // ---------------- loads ----------------
        bool ok = true;
        int issued = 0;                                 // loads of the ring
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n[i]) {
                    mbar_arrive_expect_tx(&bars[kExQFull + i], kExQ);
                    for (int c = 0; c < 3; ++c)
                        tma_load_3d(smem + kExOffQ + i * kExQ + c * kExChunk, &q_map, &bars[kExQFull + i], c * 64, head,
                                    req.qs + t0 + i * kExRows);
                }
        }
        for (int j = 0; j < n_all && ok; ++j) {
            const int key0 = req.ks + (j0 + j) * kExKeys;
#pragma unroll 1
            for (int e = 0; e < kExPerTile && ok; ++e) {
                const int s = j * kExPerTile + e, slot = s % kExSlots;
                if (s >= kExSlots)
                    ok = __all_sync(0xffffffffu, pf_wait(&bars[kExEmpty + slot], (s / kExSlots - 1) & 1, status));
                if (!ok) break;
                if (lane == 0) {
                    uint64_t *bar = &bars[kExFull + slot];
                    uint8_t *dst = smem + kExOffRing + slot * kExChunk;
                    mbar_arrive_expect_tx(bar, kExChunk);
                    *tiles = j + 1;
                    if (e < 2) {
                        tma_load_3d(dst, &k_map, bar, e * 64, head, key0);
                    } else if (e == 2) {
                        tma_load_3d(dst, &r_map, bar, 0, 0, key0);
                    } else {
                        tma_load_3d(dst, &v_map, bar, 0, head, key0 + (e - 3) * 64);
                        tma_load_3d(dst + 8192, &v_map, bar, 64, head, key0 + (e - 3) * 64);
                    }
                }
                issued = s + 1;
            }
            if (ok && j >= diag && lane == 0) mbar_arrive(&bars[kExLoaded + ((j - diag) & 1)]);
        }
        if (ok && fix) {
            for (int e = 3; e < kExPerTile && ok; ++e) {
                const int s = (n_all - 1) * kExPerTile + e;
                ok = __all_sync(0xffffffffu, pf_wait(&bars[kExFull + s % kExSlots], (s / kExSlots) & 1, status));
            }
            const int first = end - (seen_all - 1) * kExKeys, s = (n_all - 1) * kExPerTile + 3;
            if (ok) {
                for (int e = lane; e < (kExKeys - first) * 16; e += 32) {
                    const int r = first + (e >> 4);
                    const uint32_t a = sRing + ((s + (r >> 6)) % kExSlots) * kExChunk + ((e & 15) >> 3) * 8192 +
                                       (r & 63) * 128 + (e & 7) * 16;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kExFix]);
            }
        }
        if (!ok) {                                      // the copies in flight land before the CTA ends
            for (int i = 0; i < 2; ++i)
                if (n[i]) mbar_wait_bounded(&bars[kExQFull + i], 0);
            for (int s = max(0, issued - kExSlots); s < issued; ++s)
                mbar_wait_bounded(&bars[kExFull + s % kExSlots], (s / kExSlots) & 1);
        }
    } else if (warp == 1) {
        // ---------------- MMA issue: one elected thread ----------------
        if (elect_one()) {
            constexpr uint32_t kIdescS = idesc_bf16_f32(kExRows, kExKeys, 0, 0);
            constexpr uint32_t kIdescO = idesc_bf16_f32(kExRows, kExV, 0, 1);
            const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sRing, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sRing, 8192, 1024);      // MN-major: 64-dim chunks 8 KiB apart
            auto wait = [&](int b, uint32_t parity) { return pf_wait(&bars[b], parity, status); };
            const int n0 = n[0], n1 = n[1];
            const int frees = n1 ? 1 : 0;                                // the row tile that reads a slot last
            int landed = 0;                                              // loads waited for
            auto need = [&](int s) {
                if (s < landed) return true;
                landed = s + 1;
                const bool there = wait(kExFull + s % kExSlots, (s / kExSlots) & 1);
                tc_fence_after();
                return there;
            };
            auto issue_s = [&](int i, int j) {
                const uint64_t a = dq + i * (kExQ >> 4);
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const int s = j * kExPerTile + c, slot = s % kExSlots;
                    if (!need(s)) return false;
                    const uint64_t b = dk + static_cast<uint32_t>(slot * (kExChunk >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ss(tmem + 128u * i, a + c * (kExChunk >> 4) + kk * 2, b + kk * 2, kIdescS,
                                    (c | kk) ? 1u : 0u);
                    if (i == frees) umma_commit(&bars[kExEmpty + slot]);
                }
                umma_commit(&bars[kExSFull + i]);
                return true;
            };
            auto issue_pv = [&](int i, int j) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int s = j * kExPerTile + 3 + h, slot = s % kExSlots;
                    if (!need(s)) return false;
                    const uint64_t b = dv + static_cast<uint32_t>(slot * (kExChunk >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ts(tmem + 256u + 128u * i, tmem + 128u * i + 32u * h + 8u * kk, b + kk * (2048 >> 4),
                                    kIdescO, (h | kk) ? 1u : (j > 0 ? 1u : 0u));
                    if (i == frees) umma_commit(&bars[kExEmpty + slot]);
                }
                umma_commit(&bars[kExODone + i]);
                return true;
            };
            bool ok = true;
            if (n0) ok = wait(kExQFull, 0) && issue_s(0, 0);
            if (ok && n1) ok = wait(kExQFull + 1, 0) && issue_s(1, 0);
            // tile i's P V of key tile j, then its S of j + 1 (over the P that was just read)
            for (int j = 0; j < n_all && ok; ++j) {
                if (j >= diag) ok = wait(kExChecked + ((j - diag) & 1), ((j - diag) >> 1) & 1);
                if (ok && fix && j == n_all - 1) ok = wait(kExFix, 0);
                if (ok && j < n0) {
                    ok = wait(kExPFull, j & 1);
                    tc_fence_after();
                    if (ok) ok = issue_pv(0, j);
                    if (ok && j + 1 < n0) ok = issue_s(0, j + 1);
                }
                if (ok && j < n1) {
                    ok = wait(kExPFull + 1, j & 1);
                    tc_fence_after();
                    if (ok) ok = issue_pv(1, j);
                    if (ok && j + 1 < n1) ok = issue_s(1, j + 1);
                }
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---------------- V on the diagonal: warp 2 its first half, warp 3 its second ----------------
        // Keys that some of the rows see and others do not meet weights of 0 in the others, and
        // 0 x NaN is NaN.  So V's rows with an infinity or NaN are zeroed there, and the rows that
        // see the first of them are made NaN at the end.  (The load warp's signal comes first: the
        // slot's barrier is then in the phase waited for, or one further.)
        const int h = warp - 2;
        bool ok = true;
        for (int j = diag; j < n_all && ok; ++j) {
            const int d = j - diag, s = j * kExPerTile + 3 + h;
            ok = warp_wait_tiles(&bars[kExLoaded + (d & 1)], (d >> 1) & 1, tiles, status) &&
                 __all_sync(0xffffffffu, pf_wait(&bars[kExFull + s % kExSlots], (s / kExSlots) & 1, status));
            if (!ok) break;
            const int key0 = (j0 + j) * kExKeys + 64 * h, lo = max(edge - key0, 0), hi = min(end - key0, 64);
            // 16 bytes of row r a lane, a row 16 lanes
            const uint32_t base = sRing + (s % kExSlots) * kExChunk + ((lane & 15) >> 3) * 8192 + (lane & 7) * 16;
            auto largest = [&](int r, uint32_t (&acc)[4]) {     // of |acc| and the piece, NaN if there is one
                uint32_t v[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                             : "r"(base + r * 128)
                             : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(acc[e]) : "r"(v[e]));
            };
            auto odd = [](const uint32_t (&acc)[4]) {
                bool any = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    any |= (acc[e] & 0x7F80u) == 0x7F80u || (acc[e] & 0x7F800000u) == 0x7F800000u;
                return __any_sync(0xffffffffu, any);
            };
            uint32_t acc[4] = {};
#pragma unroll 4
            for (int r = lo + (lane >> 4); r < hi; r += 2) largest(r, acc);
            if (odd(acc)) {
                for (int r = lo; r < hi; ++r) {
                    uint32_t one[4] = {};
                    largest(r, one);
                    if (!odd(one)) continue;
                    if (lane < 16)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + r * 128), "r"(0u) : "memory");
                    if (lane == 0) atomicMin(odd_key, key0 + r);
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kExChecked + (d & 1)]);
        }
    } else if (warp >= 4) {
        // ---------------- softmax (a row per thread) and epilogue ----------------
        const int i = (warp - 4) >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const bool mine = row < rows[i];
        // keys this row sees (a row that no token owns computes what it finds, for nobody,
        // rather than put its warp on the masked path)
        const int lim = mine ? ctx + t0 + i * kExRows + row + 1 : INT32_MAX;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * i;
        const uint32_t tO = tS + 256u;
        // |scale| and a flip of the scores, so that the largest score has the largest
        // weight; not quite 0, so that masked scores stay -inf
        const float sl2 = fmaxf(fabsf(p.scale_log2), 1.2e-38f);
        float m_ref = NEG_INF, l = 0.f;
        bool ok = true;
        const int n_mine = n[i];
        for (int j = 0; j < n_mine && ok; ++j) {
            ok = __all_sync(0xffffffffu, pf_wait(&bars[kExSFull + i], j & 1, status));
            if (!ok) break;
            tc_fence_after();
            float s[kExKeys];
#pragma unroll
            for (int c = 0; c < kExKeys / 32; ++c) tmem_ld32f(tS + 32 * c, s + 32 * c);
            tmem_ld_wait();
            if (p.scale_log2 < 0.f) {
#pragma unroll
                for (int c = 0; c < kExKeys; ++c) s[c] = -s[c];
            }
            const int key0 = (j0 + j) * kExKeys;
            if (__any_sync(0xffffffffu, key0 + kExKeys > lim)) {
#pragma unroll
                for (int c = 0; c < kExKeys; ++c) s[c] = key0 + c < lim ? s[c] : NEG_INF;
            }
            float mx4[4] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3]), fmaxf(s[4], s[5]), fmaxf(s[6], s[7])};
#pragma unroll
            for (int c = 8; c < kExKeys; c += 8) {
                mx4[0] = fmax3(mx4[0], s[c], s[c + 1]);
                mx4[1] = fmax3(mx4[1], s[c + 2], s[c + 3]);
                mx4[2] = fmax3(mx4[2], s[c + 4], s[c + 5]);
                mx4[3] = fmax3(mx4[3], s[c + 6], s[c + 7]);
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
            // the reference moves on the first visible key, and then only when the max
            // exceeds it by 2^40 (fp32 sums and bf16 weights keep their relative
            // accuracy at any common scale)
            const bool first = m_ref == NEG_INF;
            const bool grow = !first && mx > m_ref + 40.f;
            const float alpha = grow ? fast_exp2(m_ref - mx) : 1.f;
            if (first || grow) m_ref = mx;
            if (__any_sync(0xffffffffu, grow)) {
                // rare: O rescaled once the previous tile's product has completed
                ok = __all_sync(0xffffffffu, pf_wait(&bars[kExODone + i], (j - 1) & 1, status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < kExV / 16; ++c) {
                    float v[16];
                    uint32_t w[16];
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
                          "=f"(v[15])
                        : "r"(tO + 16 * c));
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e] * alpha);
                    tmem_st16(tO + 16 * c, w);
                }
                l *= alpha;
            }
            const float ref = m_ref == NEG_INF ? 0.f : m_ref;
            const uint64_t sc2 = f2_pack(sl2, sl2), nref2 = f2_pack(-ref, -ref);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < kExKeys / 32; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float y0, y1;
                    f2_unpack(f2_fma(f2_pack(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), sc2, nref2), y0, y1);
                    const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                    sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
                    w[e] = pack_bf16x2(p0, p1);
                }
                tmem_st16(tS + 16 * c, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kExPFull + i]);
            float a, b;
            f2_unpack(f2_add(sum2[0], sum2[1]), a, b);
            l += a + b;
        }
        if (ok && n_mine) ok = __all_sync(0xffffffffu, pf_wait(&bars[kExODone + i], (n_mine - 1) & 1, status));
        if (ok && n_mine && lim > *reinterpret_cast<volatile int32_t *>(odd_key)) l = __int_as_float(0x7fffffff);
        const int64_t stride = static_cast<int64_t>(p.heads) * kExV;
        __nv_bfloat16 *o = p.out + static_cast<int64_t>(req.qs + t0) * stride + head * kExV;
        if (p.split > 1) {
            // 32 rows (a warp's) of the 256 are one of eight groups; 8 / split of them are
            // finished in each CTA, by split warps a group, from the states and sums that
            // every CTA leaves there.
            tc_fence_after();
            if (!ok || !n_mine) m_ref = NEG_INF;
            else if (l != l) m_ref = -NEG_INF;              // (a NaN stays one in the join)
            const int per = 8 / p.split, w = warp - 4;
            cluster_sync();                             // no CTA's products read shared memory any more
            const uint32_t to = cluster_address(sQ, w / per);
            const uint32_t slot = part * per + w % per;
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + kExOffState + (slot * 32 + lane) * 8),
                         "f"(m_ref), "f"(l)
                         : "memory");
            const uint32_t at = to + slot * kExGroupBytes + lane * 16;
#pragma unroll 1
            for (int c = 0; c < kExV / 32; ++c) {
                float v[32];
                tmem_ld32f(tO + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + (8 * c + e / 4) * 512),
                                 "f"(v[e]), "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3])
                                 : "memory");
            }
            cluster_sync();
            const int g = w / p.split, dims = kExV / p.split, d0 = w % p.split * dims;
            const int row0 = (part * per + g) * 32;
            const int owned = min(32, (row0 < kExRows ? rows[0] : rows[1] + kExRows) - row0);
            uint8_t *stage = smem + kExOffStage + w * 4096;
            if (p.split == 2) {
                ex_join<2>(smem, g, d0, lane, stage);
                ex_store<8>(stage, lane, owned, o + row0 * stride + d0, stride);
            } else {
                ex_join<4>(smem, g, d0, lane, stage);
                ex_store<4>(stage, lane, owned, o + row0 * stride + d0, stride);
            }
        } else if (ok && n_mine) {
            tc_fence_after();
            const float inv = l <= 0.f ? 0.f : 1.f / l;         // (NaN stays)
            const int owned = min(32, (i ? rows[1] : rows[0]) - quad * 32);
            uint8_t *stage = smem + kExOffQ + i * kExQ + quad * 8192;      // over Q, which the last S has read
#pragma unroll 1
            for (int c = 0; c < kExV / 32; ++c) {
                float v[32];
                tmem_ld32f(tO + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y[8] = {v[8 * e],     v[8 * e + 1], v[8 * e + 2], v[8 * e + 3],
                                        v[8 * e + 4], v[8 * e + 5], v[8 * e + 6], v[8 * e + 7]};
                    ex_stage<16>(stage, lane, 4 * c + e, y, inv);
                }
            }
            ex_store<16>(stage, lane, owned, o + (i * kExRows + quad * 32) * stride, stride);
        }
    }

    if (p.split > 1 && warp < 4) cluster_sync(), cluster_sync();       // (with the softmax warps')
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The requests' check alone, where no token can be answered (no rows, no keys, or a bound of no queries).
__global__ void __launch_bounds__(kExThreads) latent_expanded_check_kernel(const ExParams p) {
    for (int r = threadIdx.x; r < p.num_seqs; r += kExThreads)
        if (!ex_request(p, r).ok) set_status(p.status, PKV_ERR_DEVICE_METADATA);
}

// {dims, heads, tokens} of 16-bit elements: a box is 64 dims of one head of box_rows tokens.
static int make_rows_map(CUtensorMap *map, const void *base, int dims_in, int64_t heads, int64_t head_stride,
                         int64_t tokens, int64_t token_stride, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dims_in), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(token_stride) * 2};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // namespace pkv

extern "C" int pkv_latent_attn_expanded(void *out, const void *query, int64_t query_token_stride, const void *key,
                                        int64_t key_token_stride, int64_t key_head_stride, const void *key_rope,
                                        int64_t key_rope_token_stride, const void *value, int64_t value_token_stride,
                                        int64_t value_head_stride, const int32_t *query_start_loc,
                                        const int32_t *key_start_loc, int32_t num_seqs, int32_t num_tokens,
                                        int32_t num_keys, int32_t max_query_len, int32_t max_key_len,
                                        int32_t num_heads, float scale, int32_t *device_status, void *stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_tokens < 0 || num_keys < 0 || max_query_len < 0 || max_key_len < 0 || num_heads <= 0)
        return PKV_ERR_SHAPE;
    if (num_heads > (1 << 16) || max_key_len > INT32_MAX - 256 || max_query_len > max_key_len) return PKV_ERR_SHAPE;
    if (num_keys > INT32_MAX - 256 || num_tokens > INT32_MAX - 256) return PKV_ERR_SHAPE;
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return PKV_ERR_SHAPE;
    if (num_seqs == 0) return num_tokens ? PKV_ERR_SHAPE : PKV_OK;
    ExParams p;
    p.qsl = query_start_loc, p.ksl = key_start_loc;
    p.num_seqs = num_seqs, p.num_tokens = num_tokens, p.num_keys = num_keys;
    p.max_query_len = max_query_len, p.max_key_len = max_key_len;
    p.heads = num_heads;
    p.status = device_status;
    if (num_tokens == 0 || num_keys == 0 || max_query_len == 0) {
        if (!device_status) return PKV_OK;
        if (!query_start_loc || !key_start_loc) return PKV_ERR_NULL;
        if ((reinterpret_cast<uintptr_t>(query_start_loc) | reinterpret_cast<uintptr_t>(key_start_loc)) & 3u)
            return PKV_ERR_ALIGNMENT;
        latent_expanded_check_kernel<<<1, kExThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    if (!out || !query || !key || !key_rope || !value || !query_start_loc || !key_start_loc) return PKV_ERR_NULL;
    constexpr int64_t kMost = int64_t(1) << 38;          // of a tensor map's strides, in elements
    if (key_head_stride < kExNope || value_head_stride < kExV || key_head_stride > kMost || value_head_stride > kMost)
        return PKV_ERR_SHAPE;
    const int64_t h = num_heads;
    if (query_token_stride < h * kExDim || query_token_stride > kMost ||
        key_token_stride < kExNope || key_token_stride > kMost || key_rope_token_stride < kLatRope ||
        key_rope_token_stride > kMost || value_token_stride < kExV || value_token_stride > kMost)
        return PKV_ERR_SHAPE;
    if ((query_token_stride % 8) || (key_token_stride % 8) || (key_head_stride % 8) || (key_rope_token_stride % 8) ||
        (value_token_stride % 8) || (value_head_stride % 8))
        return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(query) | reinterpret_cast<uintptr_t>(key) |
         reinterpret_cast<uintptr_t>(key_rope) | reinterpret_cast<uintptr_t>(value)) & 15u)
        return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(query_start_loc) | reinterpret_cast<uintptr_t>(key_start_loc)) & 3u)
        return PKV_ERR_ALIGNMENT;

    p.out = static_cast<__nv_bfloat16 *>(out);
    // the most that sum of ceil(q_r / 256) can be
    const int64_t bound = (num_tokens + static_cast<int64_t>(num_seqs) * (kExTokens - 1)) / kExTokens;
    const int64_t tiles = bound < num_tokens ? bound : num_tokens;
    if (tiles * num_heads > INT32_MAX) return PKV_ERR_SHAPE;
    p.tiles = static_cast<int32_t>(tiles);
    // Keys and values of every head at once outgrow L2 (126 MB) long before one head's
    // do: then the token tiles of a head run side by side, and its keys and values come
    // from memory once instead of once a token tile.  All heads of a rank / all ranks of a head:
    // 2048 tokens at 8192 keys of 128 heads (537 MB of keys and values) 855 / 775 us, 1024 tokens
    // there 462 / 451; 268 MB, 2048 tokens at 4096 keys of 128 heads 372 / 371, at 8192 of 64 heads 419 /
    // 429; 134 MB, 16 heads at 16384 keys 218 / 227; 33 MB, 16 heads at 4096 keys 57.7 / 65.7.  So the
    // bound is on the low side: between it and some 270 MB the order costs up to 8%.
    p.by_head = static_cast<int64_t>(num_keys) * num_heads * (kExNope + kExV) * 2 > (int64_t(64) << 20);
    p.scale_log2 = scale * 1.4426950408889634f;
    CUtensorMap qm, km, rm, vm;
    int rc = make_rows_map(&qm, query, kExDim, h, kExDim, num_tokens, query_token_stride, kExRows);
    if (!rc) rc = make_rows_map(&km, key, kExNope, h, key_head_stride, num_keys, key_token_stride, kExKeys);
    if (!rc) rc = make_rows_map(&rm, key_rope, kLatRope, 1, kLatRope, num_keys, key_rope_token_stride, kExKeys);
    if (!rc) rc = make_rows_map(&vm, value, kExV, h, value_head_stride, num_keys, value_token_stride, kExKeys / 2);
    if (rc) return rc;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    static std::mutex mu;
    static uint64_t done_mask = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (!bit || !(done_mask & bit)) {
            if (cudaFuncSetAttribute(latent_expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExSmem) !=
                cudaSuccess)
                return PKV_ERR_CUDA;
            done_mask |= bit;
        }
    }
    // Few token tiles of many keys each leave SMs idle and wait for the longest.  Then two or
    // four CTAs, a cluster, share a tile's keys.  Two where the CTAs were at most one an SM (a
    // causal chunk's tiles see half of the longest's keys on average, so a second round of
    // shorter ones still pays: 4096 tokens of 8 heads 40.6 us instead of 57.7, 2048 of 16
    // heads 29.8 instead of 32.0); four where one round holds them (256 tokens at 8192 keys of
    // 16 heads: 108 us whole, 59.8 by two, 34.8 by four; 1024 tokens of 16 heads, 64 tiles:
    // 18.0, 15.4, 22.7).  Each further CTA pays a start and an end of 6 us or so (three requests
    // of 300 to 2046 tokens, 224 tiles: 32.5 whole, 49.6 by two), and of clusters of eight only
    // 15 find a place on the 152 SMs (256 at 8192: 43.5).
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return PKV_ERR_CUDA;
    const int key_tiles = (max_key_len + kExKeys - 1) / kExKeys;
    p.split = 1;
    if (tiles * num_heads <= sms && key_tiles >= 2) p.split = 2;
    if (tiles * num_heads * 4 <= sms && key_tiles >= 4) p.split = 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * num_heads * p.split));
    cfg.blockDim = dim3(kExThreads);
    cfg.dynamicSmemBytes = kExSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, latent_expanded_kernel, qm, km, rm, vm, p) != cudaSuccess) return PKV_ERR_CUDA;
    return PKV_OK;
}
