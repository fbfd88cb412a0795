// Chunks over an int8 cache (int8_common.cuh), on the 5th-generation tensor cores: the computation of int8_decode.cu
// for requests of many rows (query token, query head of the kv head's group).
//
// With codes k_j, v_j and their blocks' scales ks, vs, for a row q scaled by a power of two 2^e into f16:
//     S_j = <q 2^e, 1152 + k_j>,   e_j = (S_j - 1152 sum q 2^e) (scale 2^-e log2(e) ks) + log2 vs
//     p'_j = 2^(e_j - m),          out = sum_j p'_j v_j / sum_j p'_j / vs
// K's codes widen to f16 as 1152 + code (a byte next to 0x64) and stay so: what that adds to S is one number a row, and
// goes with the block's factor into the constants of the softmax, of which a row has three a block of 16 keys.  V's
// codes are taken back to themselves.  m is 3 below the row's largest e_j so far, which is looked for again only where
// the weights of a tile sum to more than 6e4, so that p' fits f16 whatever the blocks' scales are, and a long tail of
// small ones is no more than 2^-28 of the largest off each.
//
// Work item: 256 rows of one request for one kv head, as two 128-row tiles that take turns on the tensor cores and
// share each 128-key tile; a persistent CTA an SM takes items largest first.  Where that would leave CTAs idle for
// longer than a join takes, the items' key tiles are one line that is cut into an equal run for each CTA; the combine
// that follows joins the pieces' sums, which are left in the workspace.
//
// Per key tile: 8 pages (a TMA box each for K and for V) land raw, four warps widen them into a ring of 16 KiB slots in
// the layout the products read, S = Q K^T from shared memory (128 x 128 x 16), softmax by four warps a row tile (a row
// per thread), P as f16 over S in tensor memory, O += P V.  Tensor memory: S of both tiles, O of both (512 columns).
//
// Warp roles (448 threads): warp 0 items, loads and the pages' scales, warp 1 issues the MMAs, warps 2, 3, 12 and 13
// widen (one on each scheduler), warps 4-7 and 8-11 are the softmax and epilogue of the two row tiles.  Every wait is
// bounded.
//
// What bounds it: the softmax warps, three warps a scheduler with the widening one.  2432 tokens behind 6144 keys of
// 32/8 heads of 128 (two rounds of whole items) take 263 us, 4100 cycles a pair of tiles where the products take 2080;
// 2046 tokens 239, in runs (the tensor pipe at 48%, issue at 47%).  Tried and slower: two threads a row, halves of 64
// keys (P V early, or the next S early: the other half's S while P V runs hides what the softmax waits for, and reads Q
// twice), an MMA warp a row tile, a pass for each row's largest score (367 us with loops unrolled: instruction fetch).
// 256 tokens at 6400 keys: 63 us, with items left whole 119.
#include <mutex>
#include <type_traits>

#include "int8_common.cuh"
#include "latent_common.cuh"

namespace pkv {

constexpr int kIpRows = 128;                          // of a row tile
constexpr int kIpKeys = 128;                          // of a key tile
constexpr int kIpPages = kIpKeys / kBlock;
constexpr int kIpSoft = 4;                            // softmax warps of a row tile
constexpr int kIpWiden = 4;                           // warps that widen
constexpr int kIpThreads = 32 * (2 + kIpWiden + 2 * kIpSoft);
constexpr int kIpSlot = 16384;                        // 64 dims of 128 rows, or 128 dims of 64 rows, as f16
constexpr int kIpSlots = 8;
constexpr int kIpScaleTiles = 8;                      // key tiles whose blocks' scales are held
constexpr int kIpReaders = 1 + kIpWiden + 2 * kIpSoft;    // of an item: MMA, widening and softmax warps

template <int HD>
struct IpCfg {
    static constexpr int kChunks = HD / 64;           // slots of a K (or V) tile, 64-dim chunks of Q
    static constexpr int kRaw = HD == 128 ? 2 : 4;    // raw K or V tiles in flight
    static constexpr int kRawBytes = kIpKeys * HD;
    static constexpr int kOffQ = 0;                   // [row tile][chunk] 16 KiB
    static constexpr int kOffRing = kOffQ + 2 * kChunks * kIpSlot;
    static constexpr int kOffRaw = kOffRing + kIpSlots * kIpSlot;
    static constexpr int kOffBar = kOffRaw + kRaw * kRawBytes;
    static constexpr int kOffItems = kOffBar + 512;
    static constexpr int kOffScales = kOffItems + 256;    // float4 {K's, log2 of V's, 1 / V's, -} [tile & 7][block]
    static constexpr int kSmem = kOffScales + kIpScaleTiles * kIpPages * 16 + 1024;   // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

enum IpBar {
    kIpItemFull = 0,     // (+ item & 3)
    kIpItemEmpty = 4,    // (+ item & 3)
    kIpRawFull = 8,      // (+ place of the raw K or V tile)
    kIpRawEmpty = 12,    // (+ place)
    kIpFull = 16,        // (+ slot)
    kIpEmpty = 24,       // (+ slot)
    kIpQFull = 32,       // (+ row tile)
    kIpSFull = 34,       // (+ row tile)
    kIpPFull = 36,       // (+ row tile)
    kIpODone = 38,       // (+ row tile)
    kIpOFree = 40,       // (+ row tile)
    kIpScFull = 42,      // (+ tile & 7)
    kIpNumBars = 50
};
static_assert(kIpNumBars * 8 + 8 <= 512, "barriers, the tensor-memory address and the tile count");

struct IpItem {
    int32_t valid, r, g, n[2], L, qs, ctx, rows_total, row0, n_pages;
    int32_t first;       // first key tile; n: key tiles from there on that each of the two row tiles sees
    int32_t place;       // where the piece's sums go, -1: the item is whole
};
static_assert(kItemSlots * sizeof(IpItem) <= 256 && kItemSlots == 4, "the item ring's place");

// The bounded waits of this kernel, their loops once in the code: five roles run side by side, and with every wait and
// loop unrolled in place instruction fetch bounds the kernel.
__device__ __noinline__ bool ip_wait_long(uint64_t *bar, uint32_t parity, int32_t *status) {
    return pf_wait(bar, parity, status);
}
__device__ __forceinline__ bool ip_wait(uint64_t *bar, uint32_t parity, int32_t *status) {
    return mbar_try_wait(bar, parity) || ip_wait_long(bar, parity, status);
}
__device__ __forceinline__ bool ip_warp_wait(uint64_t *bar, uint32_t parity, int32_t *status) {
    return __all_sync(0xffffffffu, ip_wait(bar, parity, status));
}
__device__ __noinline__ bool ip_warp_wait_tiles(uint64_t *bar, uint32_t parity, const volatile int32_t *tiles,
                                                int32_t *status) {
    return warp_wait_tiles(bar, parity, tiles, status);
}

__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// What the loads before left in flight is there, this among it.
__device__ __forceinline__ void ip_ld_wait(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}

// In the line that is cut, an item counts for as many units as it has key tiles and kIpOver more (Q, epilogue, and what
// a piece more costs); a CTA gets kIpLeast units at least.  The cut and the join cost about kIpJoin units more.
constexpr int kIpOver = 3, kIpLeast = 6, kIpJoin = 13;

template <int HD>
__global__ void __launch_bounds__(kIpThreads, 1)
    int8_prefill_kernel(const __grid_constant__ CUtensorMap kv_map, const __nv_bfloat16 *__restrict__ query,
                        const int64_t q_stride, const float2 *__restrict__ kv_scales, const PrefillParams p) {
    using Cfg = IpCfg<HD>;
    constexpr int C = Cfg::kChunks, SLOTS = kIpSlots, RAW = Cfg::kRaw;
    constexpr int PER = 2 * C;                            // slots of a key tile: K's, then V's
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kIpNumBars);
    volatile int32_t *tiles_loaded = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
    volatile IpItem *items = reinterpret_cast<volatile IpItem *>(smem + Cfg::kOffItems);
    float4 *scales = reinterpret_cast<float4 *>(smem + Cfg::kOffScales);
    const uint32_t sQ = smem_u32(smem + Cfg::kOffQ), sRing = smem_u32(smem + Cfg::kOffRing);
    const int warp = uniform(static_cast<int>(threadIdx.x) >> 5), lane = threadIdx.x & 31;

    // As the other chunk kernels: the kernel before this one (decode) writes other rows, and it started when the plan
    // and the cache write had completed, so the plan's lists are read at once, through L2; the wait on it comes at the
    // end.
    pdl_trigger();
    const WsHeader *hdr = reinterpret_cast<const WsHeader *>(p.ws);
    int32_t *status = reinterpret_cast<int32_t *>(p.ws);
    const int n_tiles = ws_ld(&hdr->n_ptiles);
    // {request, tile, key tiles, -}
    const int4 *ptiles = reinterpret_cast<const int4 *>(p.ws + ws_ld(&hdr->off_ptiles));
    const int n_items = n_tiles * p.num_kv_heads;
    // Whole items to each CTA (rounds of an item's mean, and the largest item at least), or equal runs of all items'
    // units?  32/8 heads of 128 behind 6144 keys, runs and whole: 256 tokens (32 items) 63 and 120 us, 1280 (160) 159
    // and 229, 2046 (256) 239 and 252, 2432 (304) 283 and 263; 1280 behind none 59 and 46.  Of 64 dims (a piece's sums
    // are half as large): 256 tokens 51 and 103, 1280 130 and 193, 2046 198 and 214, 2432 231 and 224; behind none 44
    // and 37, behind 2000 keys 1000 tokens 61 and 60.  From four rounds on whole items.  The plan lists tiles of one
    // size by their index, as far as runs are taken: which items are cut, and where, and so the order of their sums, is
    // the same in every call.
    bool runs = n_items <= min(kSplitItems, 3 * static_cast<int>(gridDim.x));
    int64_t all = 0;
    int ctas = gridDim.x;
    if (runs && n_items) {                            // (some hundred tiles at most)
        for (int t = lane; t < n_tiles; t += 32) all += ws_ld(ptiles + t).z + kIpOver;
        const int64_t largest = ws_ld(ptiles).z + kIpOver;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const int64_t rounds = (n_items + ctas - 1) / ctas;
        all *= p.num_kv_heads;
        runs = all / ctas + kIpJoin < max(largest, rounds * all / n_items);
        ctas = static_cast<int>(min(static_cast<int64_t>(ctas), max(static_cast<int64_t>(1), all / kIpLeast)));
    }
    if (!runs) ctas = gridDim.x;
    if (static_cast<int>(blockIdx.x) >= (runs && n_items ? ctas : n_items)) {     // uniform over the CTA
        pdl_wait();
        return;
    }
    SplitItem *cut = reinterpret_cast<SplitItem *>(p.ws + p.split.off_items) + blockIdx.x;
    if (runs && threadIdx.x == 0) {
        cut->place = -1;
        if (blockIdx.x == 0) const_cast<WsHeader *>(hdr)->split_items = ctas;
    }
    const int G = p.G;
    if (threadIdx.x < kIpNumBars) {
        const int b = threadIdx.x;
        int count = 1;
        if (b >= kIpItemEmpty && b < kIpItemEmpty + 4) count = kIpReaders;
        else if ((b >= kIpRawEmpty && b < kIpRawEmpty + 4) || (b >= kIpFull && b < kIpFull + 8)) count = kIpWiden;
        else if ((b >= kIpQFull && b < kIpQFull + 2) || (b >= kIpPFull && b < kIpPFull + 2) ||
                 (b >= kIpOFree && b < kIpOFree + 2))
            count = kIpSoft;
        mbar_init(&bars[b], count);
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kv_map);
        *tiles_loaded = 0;
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);

    if (warp == 0) {
        // ---------------- items, raw pages, scales ----------------
        bool ok = true;
        int taken = 0, gt = 0, loads = 0;             // items, key tiles, and K and V tiles of this CTA so far
        int item = blockIdx.x;                        // whole items: the next one
        int *next_item = reinterpret_cast<int *>(p.ws + offsetof(WsHeader, next_ptile_item));
        int tile = 0;                                 // runs: a tile, where its units begin, the next unit, and the end
        int64_t at = 0, u = all * blockIdx.x / ctas;
        const int64_t u0 = u, u1 = all * (blockIdx.x + 1) / ctas;
        while (runs) {                                // the tile that this run begins in
            const int units = tile + lane < n_tiles ? ws_ld(ptiles + tile + lane).z + kIpOver : 0;
            int64_t sum = static_cast<int64_t>(units) * p.num_kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t before = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += before;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, at + sum > u0);
            if (past) {
                const int f = __ffs(static_cast<int>(past)) - 1;
                at += __shfl_sync(0xffffffffu, sum - static_cast<int64_t>(units) * p.num_kv_heads, f);
                tile += f;
                break;
            }
            at += __shfl_sync(0xffffffffu, sum, 31);
            tile += 32;
        }
        for (int k = 0; ok; ++k) {
            const int slot = k & 3;
            if (k >= 4) ok = ip_warp_wait(&bars[kIpItemEmpty + slot], (k / 4 - 1) & 1, status);
            if (!ok) break;
            IpItem it{};
            int n_kv = 0, last = 0;
            int4 pt = make_int4(0, 0, 0, 0);
            it.place = -1;
            if (!runs) {
                if (item < n_items) {
                    pt = ws_ld(ptiles + item / p.num_kv_heads);
                    it.g = item % p.num_kv_heads;
                    n_kv = pt.z;
                }
            } else {
                while (u < u1 && n_kv <= 0) {         // (a run may begin with an item's end that has no key tiles)
                    pt = ws_ld(ptiles + tile);
                    const int units = pt.z + kIpOver;
                    const int64_t next = at + static_cast<int64_t>(units) * p.num_kv_heads;
                    if (u >= next) {
                        at = next, ++tile;
                        continue;
                    }
                    it.g = static_cast<int>((u - at) / units);
                    const int64_t begin = at + static_cast<int64_t>(it.g) * units;          // of this item
                    const int o0 = static_cast<int>(u - begin);
                    const int o1 = static_cast<int>(min(u1 - begin, static_cast<int64_t>(units)));
                    it.first = max(0, o0 - kIpOver);
                    n_kv = max(0, o1 - kIpOver) - it.first;
                    if (n_kv > 0 && n_kv < pt.z) {
                        it.place = 2 * static_cast<int>(blockIdx.x) + (u == u0 ? 0 : 1);
                        // the run that its last key tile is in
                        last = static_cast<int>(((begin + units) * ctas - 1) / all);
                    }
                    u = begin + o1;
                }
            }
            if (n_kv > 0) {
                it.valid = 1;
                it.r = pt.x;
                it.L = p.seq_lens[it.r];
                it.qs = p.qsl[it.r];
                const int qlen = p.qsl[it.r + 1] - it.qs;
                it.ctx = it.L - qlen;
                it.rows_total = qlen * G;
                it.row0 = pt.y * 2 * kIpRows;
                it.n_pages = (it.L + kBlock - 1) / kBlock;
                for (int i = 0; i < 2; ++i) {
                    const int end = min(it.row0 + (i + 1) * kIpRows, it.rows_total);
                    const int seen = end > it.row0 + i * kIpRows ? (it.ctx + (end - 1) / G + kIpKeys) / kIpKeys : 0;
                    it.n[i] = max(0, min(seen - it.first, n_kv));
                }
                if (it.place >= 0 && it.first == 0 && lane == 0)
                    *cut = SplitItem{it.qs, it.rows_total, it.row0, it.g * G, it.place, static_cast<int>(blockIdx.x),
                                     last - static_cast<int>(blockIdx.x) + 1, G};
            }
            if (lane == 0) {
                volatile int32_t *dst = reinterpret_cast<volatile int32_t *>(items + slot);
                const int32_t *src = reinterpret_cast<const int32_t *>(&it);
#pragma unroll
                for (int e = 0; e < static_cast<int>(sizeof(IpItem) / 4); ++e) dst[e] = src[e];
                mbar_arrive(&bars[kIpItemFull + slot]);
            }
            if (!it.valid) break;
            ++taken;
            const int32_t *bt = p.block_tables + static_cast<int64_t>(it.r) * p.max_blocks_per_seq;
            // block ids and their scales in windows of 32 pages (4 key tiles), one lane a page, the next window ahead;
            // pages past the sequence are -1 and load as zeros (outside the tensor map)
            auto blocks_of = [&](int w) -> int {
                const int page = it.first * kIpPages + w * 32 + lane;
                const int b = page < it.n_pages ? bt[page] : -1;
                if (page < it.n_pages && (b < 0 || b >= p.num_blocks)) set_status(status, PKV_ERR_DEVICE_INDEX);
                return b;
            };
            auto scales_of = [&](int b) -> float2 {
                return b >= 0 && b < p.num_blocks ? kv_scales[static_cast<int64_t>(b) * p.num_kv_heads + it.g]
                                                  : make_float2(0.f, 1.f);
            };
            int win = 0, win_next = blocks_of(0);
            float2 sc = make_float2(0.f, 1.f), sc_next = scales_of(win_next);
#pragma unroll 1
            for (int j = 0; j < n_kv && ok; ++j, ++gt) {
                if ((j & 3) == 0) {
                    win = win_next, sc = sc_next;
                    win_next = blocks_of(j / 4 + 1);
                }
                if ((j & 3) == 2) sc_next = scales_of(win_next);
                const int at = (j & 3) * kIpPages + (lane & 7);
                const int b = __shfl_sync(0xffffffffu, win, at);
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const int rs = loads % RAW;
                    if (loads >= RAW) ok = ip_warp_wait(&bars[kIpRawEmpty + rs], (loads / RAW - 1) & 1, status);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars[kIpRawFull + rs], Cfg::kRawBytes);
                        *tiles_loaded = gt + 1;
                    }
                    __syncwarp();
                    if (lane < kIpPages)
                        tma_load_5d(smem + Cfg::kOffRaw + rs * Cfg::kRawBytes + lane * (kBlock * HD), &kv_map,
                                    &bars[kIpRawFull + rs], 0, 0, side, it.g, b);
                    ++loads;
                    if (side) continue;
                    const float ks = __shfl_sync(0xffffffffu, sc.x, at);
                    float vs = __shfl_sync(0xffffffffu, sc.y, at);
                    vs = vs < kInt8LeastScale ? kInt8LeastScale : vs;
                    // a block without a scale, of either side: NaN here (an infinity is none)
                    if (!(ks < __int_as_float(0x7f800000) && vs < __int_as_float(0x7f800000)))
                        vs = __int_as_float(0x7fc00000);
                    if (lane < kIpPages)
                        scales[(gt & 7) * kIpPages + lane] = make_float4(ks, __log2f(vs), __frcp_rn(vs), 0.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[kIpScFull + (gt & 7)]);
                }
            }
            if (!runs) {
                int nxt = 0;
                if (lane == 0) nxt = static_cast<int>(gridDim.x) + atomicAdd(next_item, 1);
                item = __shfl_sync(0xffffffffu, nxt, 0);
            }
        }
        if (!ok)                                      // the copies in flight land before the CTA ends
            for (int t = max(0, loads - RAW); t < loads; ++t)
                mbar_wait_bounded(&bars[kIpRawFull + t % RAW], (t / RAW) & 1);
        // this CTA's share of the schedule
        if (lane == 0) reinterpret_cast<int32_t *>(p.ws + kStatsOffset)[blockIdx.x] = taken;
    } else if (warp == 1) {
        // ---------------- MMA issue: one elected thread ----------------
        if (elect_one()) {
            constexpr uint32_t kIdescS = idesc_f16_f32(kIpRows, kIpKeys, 0, 0);
            constexpr uint32_t kIdescO = idesc_f16_f32(kIpRows, HD, 0, 1);
            const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sRing, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sRing, 8192, 1024);       // MN-major: 64-dim chunks 8 KiB apart
            auto wait = [&](int b, uint32_t parity) { return ip_wait(&bars[b], parity, status); };
            int landed = 0;                           // slots waited for
            int cnt[2] = {0, 0}, qs[2] = {0, 0};      // key tiles, items of each row tile so far
            int gt = 0;
            auto need = [&](int s) {
                if (s < landed) return true;
                landed = s + 1;
                const bool there = wait(kIpFull + s % SLOTS, (s / SLOTS) & 1);
                tc_fence_after();
                return there;
            };
            auto issue_s = [&](int i, int t, bool frees) {
                const uint64_t a = dq + i * (C * kIpSlot >> 4);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int s = t * PER + c, slot = s % SLOTS;
                    if (!need(s)) return false;
                    const uint64_t b = dk + static_cast<uint32_t>(slot * (kIpSlot >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ss(tmem + 128u * i, a + c * (kIpSlot >> 4) + kk * 2, b + kk * 2, kIdescS,
                                    (c | kk) ? 1u : 0u);
                    if (frees) umma_commit(&bars[kIpEmpty + slot]);
                }
                umma_commit(&bars[kIpSFull + i]);
                return true;
            };
            auto issue_pv = [&](int i, int t, bool first, bool frees) {
#pragma unroll
                for (int h = 0; h < C; ++h) {
                    const int s = t * PER + C + h, slot = s % SLOTS;
                    if (!need(s)) return false;
                    const uint64_t b = dv + static_cast<uint32_t>(slot * (kIpSlot >> 4));
                    constexpr int kSteps = 8 / C;     // of 16 keys
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk)
                        umma_f16_ts(tmem + 256u + 128u * i,
                                    tmem + 128u * i + 8u * (h * kSteps + kk), b + kk * (2048 >> 4), kIdescO,
                                    (h | kk) ? 1u : (first ? 0u : 1u));
                    if (frees) umma_commit(&bars[kIpEmpty + slot]);
                }
                umma_commit(&bars[kIpODone + i]);
                return true;
            };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int slot = k & 3;
                ok = wait(kIpItemFull + slot, (k / 4) & 1);
                if (!ok) break;
                const bool valid = items[slot].valid != 0;
                const int n[2] = {items[slot].n[0], items[slot].n[1]};
                mbar_arrive(&bars[kIpItemEmpty + slot]);
                if (!valid) break;
                const int n_kv = max(n[0], n[1]);
                const bool two = n[1] > 0;            // the second row tile reads a slot last, where it sees keys
                // (it sees as many key tiles as the first, or more, where it has rows)
                // row tile i's P V of key tile j, then its S of j + 1 (over the P that was just read)
#pragma unroll 1
                for (int j = -1; j < n_kv && ok; ++j) {
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const int mine = i ? n[1] : n[0];
                        if (!ok || max(j, 0) >= mine) continue;
                        const bool frees = i == (two ? 1 : 0);
                        if (j < 0) {
                            ok = wait(kIpQFull + i, (i ? qs[1] : qs[0]) & 1);
                        } else {
                            ok = wait(kIpPFull + i, (i ? cnt[1] : cnt[0]) & 1);
                            // the item before's O has been read out
                            if (ok && j == 0 && (i ? qs[1] : qs[0]) > 0)
                                ok = wait(kIpOFree + i, ((i ? qs[1] : qs[0]) - 1) & 1);
                            if (!ok) break;
                            tc_fence_after();
                            ok = issue_pv(i, gt + j, j == 0, frees);
                            if (i) ++cnt[1];
                            else ++cnt[0];
                        }
                        if (ok && j + 1 < mine) ok = issue_s(i, gt + j + 1, frees);
                    }
                }
                gt += n_kv;
                if (n[0]) ++qs[0];
                if (two) ++qs[1];
            }
        }
        __syncwarp();
    } else if (warp < 4 || warp >= 4 + 2 * kIpSoft) {
        // ---------------- widening: each of the warps its share of every slot ----------------
        // (all wait for every release of every slot: none can meet a barrier two phases on)
        const int part = warp < 4 ? warp - 2 : warp - 2 * kIpSoft - 2;
        bool ok = true;
        int gt = 0;
        auto freed = [&](int s) {
            return s < SLOTS || ip_warp_wait(&bars[kIpEmpty + s % SLOTS], (s / SLOTS - 1) & 1, status);
        };
        auto filled = [&](int s) {                     // (the fence: for the tensor cores)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kIpFull + s % SLOTS]);
        };
        // A warp widens 8 rows x 64 dims at a time, four lanes a row, 16 dims a lane.  Of eight lanes that access
        // memory together four have row a and four row a ^ 5 (64 dims: a ^ 1): the raw rows of 128 bytes lie with their
        // 16-byte pieces permuted by the row (TMA), those of 64 bytes as they are, and the f16 rows with theirs
        // permuted by the row too, so neither the reads nor the writes meet in a bank.
        const int c = lane & 3;
        const int r8 = HD == 128 ? ((lane >> 2) & 1 ? (lane >> 3) ^ 5 : lane >> 3) : lane >> 2;
        const uint32_t from = r8 * HD + (HD == 128 ? (c ^ r8) << 4 : c << 4);     // (second 64 dims: ^ 64)
        const uint32_t to = r8 * 128 + (((2 * c) ^ r8) << 4);                     // (its second 8 dims: ^ 16)
        // groups g0 .. of 8 rows of the raw tile at src, to groups of a slot (dst0; the second 64 dims: dst1)
        constexpr int B = 4 / C;                       // groups at a time: four 16-byte loads a lane
        auto widen = [&](auto is_v, int groups, uint32_t src, int g0, uint32_t dst0, uint32_t dst1) {
            constexpr bool V = decltype(is_v)::value;
#pragma unroll 1
            for (int n = 0; n < groups; n += B) {
                uint32_t w[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int g = g0 + n + u / C;
                    const uint32_t at = src + g * 8 * HD + from;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                                 : "r"(at ^ (64u * (u % C))));
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int8x4_to_biased_f16(w[u][e], h[2 * e], h[2 * e + 1]);
                        if (V) h[2 * e] = unbias_f16(h[2 * e]), h[2 * e + 1] = unbias_f16(h[2 * e + 1]);
                    }
                    const uint32_t row = (u % C ? dst1 : dst0) + (n + u / C) * 1024 + to;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                                 "r"(h[3])
                                 : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row ^ 16u), "r"(h[4]), "r"(h[5]),
                                 "r"(h[6]), "r"(h[7])
                                 : "memory");
                }
            }
        };
        constexpr int KG = 16 / kIpWiden, VG = 16 / C / kIpWiden;        // groups a warp: of a K tile, of a slot of V
        for (int k = 0; ok; ++k) {
            const int islot = k & 3;
            ok = ip_warp_wait(&bars[kIpItemFull + islot], (k / 4) & 1, status);
            if (!ok) break;
            const bool valid = items[islot].valid != 0;
            const int n_kv = max(items[islot].n[0], items[islot].n[1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kIpItemEmpty + islot]);
            if (!valid) break;
#pragma unroll 1
            for (int j = 0; j < n_kv && ok; ++j, ++gt) {
                const int s0 = gt * PER, rk = 2 * gt % RAW, rv = rk + 1;
                const uint32_t raw = smem_u32(smem + Cfg::kOffRaw);
                ok = ip_warp_wait(&bars[kIpRawFull + rk], (2 * gt / RAW) & 1, status);
                // K: dims 64 c .. of row r in slot c
#pragma unroll 1
                for (int s = 0; s < C && ok; ++s) ok = freed(s0 + s);
                if (!ok) break;
                const uint32_t k0 = sRing + (s0 % SLOTS) * kIpSlot, k1 = sRing + ((s0 + C - 1) % SLOTS) * kIpSlot;
                widen(std::false_type(), KG, raw + rk * Cfg::kRawBytes, part * KG, k0 + part * KG * 1024,
                      k1 + part * KG * 1024);
                for (int s = 0; s < C; ++s) filled(s0 + s);
                // (the raw tile's place is loaded again behind the last of `filled`'s fences)
                if (lane == 0) mbar_arrive(&bars[kIpRawEmpty + rk]);
                ok = ip_warp_wait(&bars[kIpRawFull + rv], (2 * gt / RAW) & 1, status);
                // V: rows 64 h .. in slot h, 64-dim chunks 8 KiB apart (64 dims: one slot)
#pragma unroll 1
                for (int h = 0; h < C && ok; ++h) {
                    ok = freed(s0 + C + h);
                    if (!ok) break;
                    const uint32_t slot = sRing + ((s0 + C + h) % SLOTS) * kIpSlot + part * VG * 1024;
                    widen(std::true_type(), VG, raw + rv * Cfg::kRawBytes, 8 * h + part * VG, slot, slot + 8192);
                    filled(s0 + C + h);
                }
                if (ok && lane == 0) mbar_arrive(&bars[kIpRawEmpty + rv]);
            }
        }
    } else {
        // ---------------- softmax (a row per thread) and epilogue ----------------
        const int i = (warp - 4) / kIpSoft, quad = warp & 3;
        const int row = quad * 32 + lane;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * i;
        const uint32_t tO = tS + 256u;
        // the sign of the scale goes into the query, so that the largest score has the largest weight
        const float sl2 = fabsf(p.scale_log2), flip = p.scale_log2 < 0.f ? -1.f : 1.f;
        bool ok = true;
        float factor = 0.f, bias = 0.f;                // of this thread's row: to log2 units, and 1152 sum q times it
        int lim = INT32_MAX;                      // keys [0, lim) visible (a row that is none sees all, for nobody)
        int64_t dst = -1;                              // where its output goes
        // this thread's row of an item: into shared memory as f16, zeros past the request
        auto take_row = [&](const volatile IpItem *it) {
            const int rrow = it->row0 + i * kIpRows + row, tok = rrow / G, hh = it->g * G + (rrow - tok * G);
            const bool mine = rrow < it->rows_total;
            lim = mine ? it->ctx + tok + 1 : INT32_MAX;
            dst = mine ? (static_cast<int64_t>(it->qs + tok) * p.num_q_heads + hh) * HD : -1;
            const uint4 *qp =
                reinterpret_cast<const uint4 *>(query + (it->qs + tok) * q_stride + static_cast<int64_t>(hh) * HD);
            uint4 v[HD / 8];
#pragma unroll
            for (int c = 0; c < HD / 8; ++c) v[c] = mine ? qp[c] : make_uint4(0, 0, 0, 0);
            uint32_t a = 0;                            // the largest |q|, of the halves of the words
#pragma unroll
            for (int c = 0; c < HD / 8; ++c)
                a = __vmaxu2(a, __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu)));
            a = max(a & 0xFFFF0000u, a << 16);
            // into [2^14, 2^15): exact but for parts below 2^-24 of the row's largest
            const int ex = a ? min(126, max(-114, 141 - static_cast<int>(a >> 23))) : 0;
            const float up = __int_as_float((ex + 127) << 23) * flip;
            const uint64_t up2 = f2_pack(up, up);
            uint64_t sum2 = 0;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c) {
                uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t x2 =
                        f2_mul(f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)), up2);
                    float x0, x1;
                    f2_unpack(x2, x0, x1);
                    w[e] = pack_p<true>(x0, x1);
                    sum2 = f2_add(sum2, x2);
                }
                const uint32_t at = sQ + (i * C + (c >> 3)) * kIpSlot + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                             :
                             : "r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            }
            float s0, s1;
            f2_unpack(sum2, s0, s1);
            factor = sl2 * __int_as_float((127 - ex) << 23);
            bias = kInt8Bias * (s0 + s1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kIpQFull + i]);
        };
        int cnt = 0, gt = 0;                           // key tiles of this row tile, and of the CTA, so far
        float m = NEG_INF, l = 0.f;
        int place = -1, n = 0;
        // A piece of an item: {reference, sum} and the sums as they are, into the workspace.
        auto leave_piece = [&](int tiles) {
            // (a row tile that sees none of these keys has no part; a sum that is no number counts in any join)
            *(reinterpret_cast<float2 *>(p.ws + p.split.off_state) + static_cast<int64_t>(place) * kSplitRows +
              i * kIpRows + row) =
                make_float2(tiles ? (l != l && m == NEG_INF ? 0.f : m) : NEG_INF, l);
            if (!tiles) return true;
            if (!ip_warp_wait(&bars[kIpODone + i], (cnt - 1) & 1, status)) return false;
            tc_fence_after();
            float4 *sums = reinterpret_cast<float4 *>(p.ws + p.split.off_sums) +
                           static_cast<int64_t>(place) * (HD / 4) * kSplitRows + i * kIpRows + row;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                float v[32];
                tmem_ld32f(tO + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sums[(8 * c + e) * kSplitRows] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kIpOFree + i]);
            return true;
        };
        // (k: the item whose Q is loaded; the epilogue of the item before comes behind that)
        for (int k = 0;; ++k) {
            ok = ip_warp_wait_tiles(&bars[kIpItemFull + (k & 3)], (k / 4) & 1, tiles_loaded, status);
            if (!ok) break;
            const volatile IpItem *cur = items + (k & 3);
            const bool valid = cur->valid != 0;
            const int n_before = n, n_kv = max(cur->n[0], cur->n[1]), place_before = place;
            const int64_t dst_before = dst;
            n = valid ? cur->n[i] : 0;
            const int first = cur->first;
            // Q right away: every S of the item before has completed
            if (n) take_row(cur);
            if (place_before >= 0) {
                ok = leave_piece(n_before);
                if (!ok) break;
            } else if (n_before) {
                ok = ip_warp_wait(&bars[kIpODone + i], (cnt - 1) & 1, status);
                if (!ok) break;
                tc_fence_after();
                const float inv = l <= 0.f ? 0.f : 1.f / l;                // (NaN stays)
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    float v[32];
                    tmem_ld32f(tO + 32 * c, v);
                    tmem_ld_wait();
                    if (dst_before >= 0) {
                        uint4 *o = reinterpret_cast<uint4 *>(p.out + dst_before) + 4 * c;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = make_uint4(pack_bf16x2(v[8 * e] * inv, v[8 * e + 1] * inv),
                                              pack_bf16x2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                              pack_bf16x2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                              pack_bf16x2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                    }
                }
                // O is read: this item's first P V may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kIpOFree + i]);
            }
            place = valid ? cur->place : -1;
            __syncwarp();
            if (valid && lane == 0) mbar_arrive(&bars[kIpItemEmpty + (k & 3)]);    // (what it says is in registers)
            if (!valid) break;
            m = NEG_INF, l = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j, ++cnt) {
                ok = ip_warp_wait(&bars[kIpSFull + i], cnt & 1, status) &&
                     ip_warp_wait(&bars[kIpScFull + ((gt + j) & 7)], ((gt + j) >> 3) & 1, status);
                if (!ok) break;
                tc_fence_after();
                const float4 *sc = scales + ((gt + j) & 7) * kIpPages;
                const int key0 = (first + j) * kIpKeys;
                const bool masked = __any_sync(0xffffffffu, key0 + kIpKeys > lim);
                // three constants of block b of the tile: what S is times, what is added, what the weights' sum is
                // times
                const float least = masked ? 1e-37f : 0.f;               // (not 0 where a score may be -inf)
                auto constants = [&](int b, float &f, float &c0, float &inv) {
                    const float4 v = sc[b];
                    f = fmaxf(factor * v.x, least);
                    c0 = fmaf(-bias, f, v.y);
                    inv = v.z;
                    // (a block without a scale, in a tile of which some rows do not see all: see below.  A query that is
                    // no number makes its own row NaN, by its bias)
                    if (masked && v.y != v.y) f = 1.f, c0 = inv = 0.f;
                };
                if (masked) {
                    // keys that the row does not see: their scores become -inf where they lie.  Blocks without a scale
                    // make the sums of the rows that see some of them no number, and have any other for those that do
                    // not.
#pragma unroll 1
                    for (int c = 0; c < kIpKeys / 32; ++c) {
                        uint32_t x[32];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = key0 + 32 * c + e < lim ? x[e] : 0xFF800000u;
                        tmem_st32(tS + 32 * c, x);
#pragma unroll
                        for (int b = 2 * c; b < 2 * c + 2; ++b)
                            if (key0 + b * kBlock < lim && sc[b].y != sc[b].y) l = sc[b].y;
                    }
                    tmem_st_wait();
                }
                // The weights are taken against the reference that is there.  Where they sum to 6e4 or less none of
                // them is past f16, and the row's largest score need not be looked for; where they do not, the
                // reference moves to 3 below it.  (Where there is none, m = -inf, they sum to an infinity or to no
                // number.)
                bool slow = j == 0;
                uint32_t w[kIpKeys / 2];               // P, pairs of f16
                float all, some;                       // the weights' sum, and that of the blocks' times 1 / vs
                while (true) {
                    if (slow) {
                        float mx = NEG_INF;
#pragma unroll 1
                        for (int b = 0; b < kIpPages; b += 2) {
                            float x[32];
                            tmem_ld32f(tS + 16 * b, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float f, c0, inv, *y = x + 16 * h;
                                constants(b + h, f, c0, inv);
#pragma unroll
                                for (int e = 8; e > 0; e >>= 1)
#pragma unroll
                                    for (int d = 0; d < e; ++d) y[d] = fmaxf(y[d], y[d + e]);
                                mx = fmaxf(mx, fmaf(y[0], f, c0));
                            }
                        }
                        mx -= kInt8ChunkLift;
                        const bool grow = mx > m;      // (m = -inf at first)
                        const float alpha = grow ? fast_exp2(m - mx) : 1.f;
                        if (grow) m = mx;
                        l *= alpha;
                        if (j > 0) {
                            // O rescaled once the previous tile's product has completed
                            ok = ip_warp_wait(&bars[kIpODone + i], (cnt - 1) & 1, status);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < HD / 16; ++c) {
                                float v[16];
                                uint32_t x[16];
                                tmem_ld16f(tO + 16 * c, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(v[e] * alpha);
                                tmem_st16(tO + 16 * c, x);
                            }
                        }
                    }
                    const float ref = slow && m == NEG_INF ? 0.f : m;
                    all = some = 0.f;
                    float x[2][16];
                    tmem_ld16f(tS, x[0]);
#pragma unroll
                    for (int b = 0; b < kIpPages; ++b) {
                        float (&z)[16] = x[b & 1];
                        ip_ld_wait(z);
                        if (b + 1 < kIpPages) tmem_ld16f(tS + 16 * (b + 1), x[(b + 1) & 1]);
                        float f, c0, inv;
                        constants(b, f, c0, inv);
                        const float cb = c0 - ref;
                        const uint64_t f2 = f2_pack(f, f), c2 = f2_pack(cb, cb);
                        // (in three sweeps, each of them independent of itself: products, exponentials, sums and pairs)
                        uint64_t y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = f2_fma(f2_pack(z[2 * e], z[2 * e + 1]), f2, c2);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y0, y1;
                            f2_unpack(y[e], y0, y1);
                            z[2 * e] = fast_exp2(y0), z[2 * e + 1] = fast_exp2(y1);
                        }
                        uint64_t sum[2];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint64_t p2 = f2_pack(z[2 * e], z[2 * e + 1]);
                            sum[e & 1] = e < 2 ? p2 : f2_add(sum[e & 1], p2);
                            w[8 * b + e] = pack_p<true>(z[2 * e], z[2 * e + 1]);
                        }
                        float s0, s1;
                        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
                        s0 += s1;
                        all += s0;
                        some = fmaf(s0, inv, some);
                    }
                    if (slow) break;
                    slow = __any_sync(0xffffffffu, !(all <= kInt8ChunkMost));
                    if (!slow) break;
                }
                if (!ok) break;
                l += some;
#pragma unroll
                for (int c = 0; c < kIpKeys / 64; ++c) {
                    uint32_t x[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = w[32 * c + e];
                    tmem_st32(tS + 32 * c, x);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kIpPFull + i]);
            }
            if (!ok) break;
            gt += n_kv;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    pdl_wait();       // complete only after the kernel launched before this one
}

// ---- host side --------------------------------------------------------------------

template <int HD>
static int launch_ip(const PrefillParams &p, const CUtensorMap &map, const void *query, int64_t q_stride,
                     const float *kv_scales, int64_t grid, int dev, cudaStream_t stream) {
    static std::mutex mu;
    static uint64_t done_mask = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (!bit || !(done_mask & bit)) {
            if (cudaFuncSetAttribute(int8_prefill_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     IpCfg<HD>::kSmem) != cudaSuccess)
                return PKV_ERR_CUDA;
            done_mask |= bit;
        }
    }
    const cudaError_t e = launch_pdl(int8_prefill_kernel<HD>, dim3(static_cast<unsigned>(grid)), dim3(kIpThreads),
                                     IpCfg<HD>::kSmem, stream, map, static_cast<const __nv_bfloat16 *>(query), q_stride,
                                     reinterpret_cast<const float2 *>(kv_scales), p);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int launch_prefill_int8(const PrefillParams &p, const void *query, int64_t q_stride, const void *kv_cache,
                        const float *kv_scales, int64_t num_blocks, int32_t head_size, int64_t grid, int dev,
                        cudaStream_t stream) {
    if (grid <= 0) return PKV_OK;
    // a box is a page of one kv head, its K or V rows; rows of 128 bytes with their 16-byte pieces permuted
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    CUtensorMap map;
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(head_size), kBlock, 2, static_cast<cuuint64_t>(p.num_kv_heads),
                                static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t row = static_cast<cuuint64_t>(head_size);
    const cuuint64_t strides[4] = {row, row * kBlock, row * kBlock * 2, row * kBlock * 2 * p.num_kv_heads};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(head_size), kBlock, 1, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(kv_cache), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, head_size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return PKV_ERR_CUDA;
    return head_size == 64 ? launch_ip<64>(p, map, query, q_stride, kv_scales, grid, dev, stream)
                           : launch_ip<128>(p, map, query, q_stride, kv_scales, grid, dev, stream);
}

}  // namespace pkv
