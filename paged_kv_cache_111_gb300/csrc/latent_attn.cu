// Paged attention over a latent cache, in the latent space (the absorbed form
// of latent attention), on the 5th-generation tensor cores.
//
// Request r's i-th query token sits at position c + i (c keys before the
// step's tokens).  For every head h, with rows C_j of 576 dims read through the
// block table,
//     out[t][h][:] = sum_j softmax_j(scale <query[t][h], C_j>) C_j[0 .. 511],
//     j = 0 .. c + i:
// one row serves every head as key (576 dims) and value (its first 512), so a
// cached row is read once for up to 64 rows of queries.
//
// Work item: one row tile, (up to 64 heads) x (tokens that fit, a power of
// two), against the 64-key tiles that its last token sees.  Rows of a tile are
// token * heads + head.  Per key tile, in shared memory once:
//   S  = Q C^T    tcgen05.mma 64 x 64 x 16, 36 of them: both operands K-major
//   softmax       each of four warps reads 16 rows of S (four threads a row, 16
//                 keys each), keeps the rows' running max and sum in fp32, and
//                 writes the weights as bf16 into shared memory
//   O' += C'P'    the products transposed: tcgen05.mma 128 x rows x 16 with A =
//                 the same tile's latent dims read MN-major, B = the weights; 16
//                 of them, O' as four blocks of 128 dims (lanes) x rows (columns)
// Transposed, the 64 x 512 outputs take 256 tensor-memory columns and leave
// room for two S buffers; the straight form (rows on lanes) would leave half of
// the lanes empty and fill all 512 columns.  Heads beyond 64 are split into
// groups, and CTAs of one lane (below) read the same keys at the same time, one
// from memory and the others through L2.
//
// Split: the batch is one line of (row tile, key tile) units, request after
// request; it is cut into equal runs, one per CTA lane, so that every SM gets
// the same number of key tiles whatever the lengths (a decode of one long
// request and a batch of short ones alike).  Every CTA finds its run from the
// lengths itself; there is no plan kernel.  A row tile that falls into one run
// is written at once; one that runs across lanes leaves unnormalised partial
// sums with their maxima, merged by a second kernel.  A run holds at most two
// such partial tiles, its first and its last, so the workspace has a fixed size.
//
// The weights enter the second product as bf16: an error of at most 2^-8 of
// each weight, about that of the output's own rounding.  Sums, maxima and
// outputs are fp32.
//
// Warp roles (416 threads): warp 3 walks the run and publishes items ahead of
// the others; warp 0 loads pages by TMA (two boxes a page); warp 1 issues the S
// products and warp 8 the second ones, each as soon as its operands are there (one
// warp for both had to look for two events in turn, about 600 cycles a tile);
// warp 2 loads Q (TMA), zeroes the rows past a tile's last visible key
// (so that what an unwritten slot holds never meets a zero weight) and owns
// tensor memory; warps 4-7 are the softmax; warps 9-12 write finished tiles out
// while the softmax is at the next one.  Every wait is bounded; those that last as long as an
// item go by the tiles loaded meanwhile.
//
// What bounds it: shared memory.  A 64-key tile takes 36 x 4 KiB for S, 16 x 6 KiB for
// the second products, 72 KiB of loads and 8 of weights, 320 KiB at 128 bytes a cycle: 2560
// cycles, and 2500 to 2740 are measured.  A row tile costs 6000 cycles beside its key
// tiles, the merge 10 us a call (of four short requests 3.6).  256 requests of 16 to 4096 keys,
// 128 heads (330 MB, 62.6 GFLOP): 94 us, 3.5 TB/s, 665 TFLOP/s.  Two decodes and a 2046-token
// chunk of 16 heads (109 GFLOP): 132.5 us, 820 TFLOP/s.  Bringing Q in in two parts, or into L2 ahead
// of its item, gained nothing (94 to 96 us).
#include <mutex>
#include <type_traits>

#include "latent_common.cuh"
#include "prefill_common.cuh"

namespace pkv {

constexpr int kLaRows = 64;                                  // rows of a tile (M of the S product)
constexpr int kLaKeys = 64;                                  // keys of a tile
constexpr int kLaPages = kLaKeys / kBlock;                   // 4
constexpr int kLaStage = kLaPages * kLatPageBytes;           // 73728
constexpr int kLaStages = 2;
constexpr int kLaChunks = kLatRow / 64;                      // 9 chunks of 64 dims
constexpr int kLaQChunk = kLaRows * 128;                     // 8192: 64 dims of 64 rows
constexpr int kLaMaxCtas = 152;
constexpr int kLaMaxHeads = 1024;
constexpr int kLaThreads = 416;
constexpr int kLaItemSlots = 4;
constexpr int kLaAhead = 1;                                  // tiles between a page's way into L2 and its load
// Buffers of the rescale votes, by tile.  A softmax warp that does not rescale at tile g has
// nobody wait for its look at the votes of g, so they are overwritten only by a tile whose
// scores that look came before in any order of events: S of tile g + 3 is written to the stage
// that the second products of g + 1 have released; those wait for every softmax warp's weights
// of g + 1, and a warp is at g + 1 once it has looked at g.  Two buffers do not hold across items,
// as an item's first tile looks at no votes; three do, and four are indexed by a mask.
constexpr int kLaVotes = 4;
static_assert(kLaAhead * kLaPages <= 32, "one page a lane");

// A stage holds a tile's 64 keys in two parts, each [page][token half][chunk]
// [token % 8][64 dims] with 128-byte swizzle: part A has chunks 0-3 (dims 0 .. 255),
// part B chunks 4-8 (dims 256 .. 511 and the rotated 64).  In each part the 8-key
// groups of the tile sit at one stride, for both products.  The parts are loaded,
// waited for and released on their own: S starts on A while B is on its way, and
// A's next load starts while the products with B's dims still run.  The rotated
// chunk is not needed once S is computed: the tile's weights are written over it
// (rows of 64 query rows per key, MN-major).
constexpr int kLaChunksA = 4, kLaChunksB = kLaChunks - kLaChunksA;        // 4, 5
constexpr int kLaGroupA = kLaChunksA * 1024, kLaGroupB = kLaChunksB * 1024;
constexpr int kLaPageA = 2 * kLaGroupA, kLaPageB = 2 * kLaGroupB;         // 8192, 10240
constexpr int kLaPartA = kLaPages * kLaPageA, kLaPartB = kLaPages * kLaPageB;
static_assert(kLaPartA + kLaPartB == kLaStage, "a stage's parts");
constexpr int kLaOffW = kLaPartA + (kLaChunksB - 1) * 1024;               // weights of key group 0 in a stage

// shared memory (from a 1 KiB boundary)
constexpr int kLaOffQ = 0;
constexpr int kLaOffKV = kLaOffQ + kLaChunks * kLaQChunk;                 // 73728
constexpr int kLaOffOut = kLaOffKV + kLaStages * kLaStage;                // rows on their way out, 2 KiB a warp
constexpr int kLaOffBar = kLaOffOut + 4 * 2048;                           // 229376
constexpr int kLaOffAlpha = kLaOffBar + 304;                              // float [2][64]
constexpr int kLaOffRow = kLaOffAlpha + 512;                              // LaRows [2]
constexpr int kLaRowsBytes = 528;
constexpr int kLaOffItems = kLaOffRow + 2 * kLaRowsBytes;
constexpr int kLaSmem = kLaOffItems + 160 + 1024;                         // with alignment slack
static_assert(kLaSmem <= 227 * 1024, "shared memory of one CTA");

// tensor memory: O' block m at columns 64 m, S buffer b at 256 + 64 b
constexpr uint32_t kLaTmemCols = 512;
__device__ __forceinline__ constexpr uint32_t la_col_s(int b) { return 256u + 64u * b; }

// workspace
constexpr int64_t kLaWsStatus = 256;                                      // int32 per CTA
constexpr int64_t kLaWsDesc = 1280;                                       // int4 per CTA
constexpr int64_t kLaWsDesc0 = kLaWsDesc + kLaMaxCtas * 16;               // int4 per CTA
constexpr int64_t kLaWsMl = 8192;                                         // float [CTA][2][max, sum][64]
constexpr int64_t kLaWsO = kLaWsMl + kLaMaxCtas * 2 * 2 * kLaRows * 4;    // float [CTA][2][64 x 512]
constexpr int64_t kLaPartFloats = kLaRows * kLatent;
constexpr int64_t kLaWsBytes = kLaWsO + static_cast<int64_t>(kLaMaxCtas) * 2 * kLaPartFloats * 4;
static_assert(kLaWsStatus + kLaMaxCtas * 4 <= kLaWsDesc && kLaWsDesc0 + kLaMaxCtas * 16 <= kLaWsMl, "workspace");

struct LaParams {
    __nv_bfloat16 *out;
    const int32_t *block_tables;
    int32_t max_blocks_per_seq;
    const int32_t *seq_lens, *qsl;
    int32_t num_seqs, num_tokens, max_query_len, max_seq_len;
    int32_t heads;            // query heads
    int32_t groups;           // head groups: CTAs of a lane
    int32_t hpt, tpt;         // heads and tokens of a row tile
    int32_t tpt_shift;        // log2(tpt)
    int32_t lanes;
    const uint8_t *cache;
    int64_t num_blocks;
    float scale_log2;
    uint8_t *ws;
};

// One item of a CTA's run: key tiles [kv0, kv1) of a row tile.
struct LaItem {
    int32_t valid;
    int32_t tok0, ntok;       // its tokens in the batch
    int32_t lim0;             // keys its first token sees (each later one sees one more)
    int32_t kv0, kv1;
    int32_t n_kv;             // key tiles of the whole row tile
    int32_t slot;             // -1: complete, written to out; else the partial slot of this CTA
    int32_t r;                // request
};
static_assert(kLaItemSlots * sizeof(LaItem) + 4 <= 160, "item ring, tiles loaded");

// What the softmax warps leave for the warps that write a finished item out.
struct LaRows {
    float inv[kLaRows];       // one over the row's sum
    int32_t dst[kLaRows];     // token * heads + head, or -1
    int32_t rows, slot;       // of the item (slot: LaItem's)
};
static_assert(sizeof(LaRows) <= kLaRowsBytes && kLaRowsBytes % 16 == 0, "row records");

enum LaBar {
    kLaQFull = 0, kLaQEmpty = 1,
    kLaSFull = 2,             // S buffer b written (+ b)
    kLaSFree = 27,            // S buffer b read (+ b)
    kLaRowFull = 29,          // row record b written (+ b)
    kLaRowFree = 31,          // row record b read (+ b)
    kLaPFull = 33,            // weights and votes of a tile written (+ tile & 1)
    kLaODone = 5,             // the tile's second products completed
    kLaOReady = 8,            // the item's last ones completed
    kLaOFree = 6,             // dims 0 .. 255 of O' read out
    kLaOFree2 = 4,            // and the others
    kLaRescaled = 7,          // O' rescaled (only in tiles where some warp voted for it)
    kLaFix = 9,               // rows past the last visible key zeroed (+ stage)
    kLaItemFull = 11, kLaItemEmpty = 15,
    kLaKVFull = 19,           // a part landed (+ 2 stage + part)
    kLaKVEmpty = 23,          // a part read by its last product (+ 2 stage + part)
    kLaNumBars = 35
};
static_assert(kLaNumBars * 8 + 8 + 4 * kLaVotes <= 304, "barriers, tensor-memory address, status, votes");

// Request r's share of the line of units.
struct LaReq {
    int32_t q, L, ctx, qs;
    int32_t n_full;           // row tiles whose tokens are all there
    int64_t units;            // length of all its row tiles on the line
};

// sum of floor(x / 2^s) over x < m
__device__ __forceinline__ int64_t la_floor_sum(int64_t m, int s) {
    const int64_t d = m >> s;
    return ((d * (d - 1) / 2) << s) + d * (m - (d << s));
}

// A row tile costs, beside its key tiles, about as much time as two of them (its
// query's load, the first softmax, the outputs' way out): on the line it is two
// units longer, so that runs of many short row tiles are not the last to end.
constexpr int kLaExtra = 2;

// Units of the row tiles before tile j of a request (j <= n_full): tile i sees
// ctx + (i + 1) tpt keys, and tpt = 2^shift divides 64.
__device__ __forceinline__ int64_t la_units_before(int32_t ctx, int shift, int64_t j) {
    const int64_t b = (ctx + kLaKeys - 1) >> shift;
    return la_floor_sum(b + j + 1, 6 - shift) - la_floor_sum(b + 1, 6 - shift) + kLaExtra * j;
}
static_assert(kLaKeys == 64, "2^6 keys a tile");

__device__ __forceinline__ LaReq la_request(const LaParams &p, int r, bool &bad) {
    LaReq a;
    a.qs = __ldg(p.qsl + r);
    const int q1 = __ldg(p.qsl + r + 1);
    a.L = __ldg(p.seq_lens + r);
    a.q = q1 - a.qs;
    a.ctx = a.L - a.q;
    a.n_full = 0;
    a.units = 0;
    const bool ok = !(a.qs < 0 || a.q < 0 || q1 > p.num_tokens || a.L < a.q || a.L > p.max_seq_len ||
                      a.q > p.max_query_len || (a.L + kBlock - 1) / kBlock > p.max_blocks_per_seq);
    bad |= !ok;
    if (ok && a.q > 0) {
        a.n_full = a.q >> p.tpt_shift;
        a.units = la_units_before(a.ctx, p.tpt_shift, a.n_full);
        if (a.q & (p.tpt - 1)) a.units += (a.L + kLaKeys - 1) / kLaKeys + kLaExtra;
    }
    return a;
}

// 16 lanes x 64 columns of tensor memory: thread t gets rows t / 4 (registers
// 4 k, 4 k + 1) and t / 4 + 8 (4 k + 2, 4 k + 3), columns 8 k + 2 (t % 4) + {0, 1}.
__device__ __forceinline__ void tmem_ld_16x64f(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}

// The same of 32 columns.
__device__ __forceinline__ void tmem_ld_16x32f(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// Four 8 x 8 tiles of 16-bit values to shared memory, transposed: thread t holds
// elements (t / 4, 2 (t % 4) + {0, 1}) of each, and gives the address of column
// t % 8 of tile t / 8.
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}

// 2-D tiled store of one box from shared memory, as a bulk group of this thread.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All of this thread's bulk stores have read shared memory (or are complete).
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__global__ void __launch_bounds__(kLaThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                       const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap out_map,
                       const LaParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kLaOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kLaNumBars);
    int32_t *status = reinterpret_cast<int32_t *>(tmem_slot + 1);       // of this CTA, in shared memory
    volatile uint8_t *votes = reinterpret_cast<volatile uint8_t *>(tmem_slot + 2);    // [tile % kLaVotes][warp]
    int64_t *scan = reinterpret_cast<int64_t *>(smem + kLaOffAlpha);    // before the roles start only
    volatile LaItem *items = reinterpret_cast<volatile LaItem *>(smem + kLaOffItems);
    volatile int32_t *tiles = reinterpret_cast<volatile int32_t *>(smem + kLaOffItems + kLaItemSlots * sizeof(LaItem));
    const uint32_t sQ = smem_u32(smem + kLaOffQ), sKV = smem_u32(smem + kLaOffKV), sOut = smem_u32(smem + kLaOffOut);
    const int warp = uniform(static_cast<int>(threadIdx.x) >> 5), lane = threadIdx.x & 31;
    const int my_lane = blockIdx.x / p.groups;               // run
    const int group = blockIdx.x - my_lane * p.groups;       // head group

    if (threadIdx.x < kLaNumBars) {
        const int b = threadIdx.x;
        int count = 1;
        if (b == kLaOFree || b == kLaOFree2 || b == kLaRescaled || b == kLaSFree || b == kLaSFree + 1 || b >= kLaRowFull)
            count = 4;                                       // four warps
        else if (b >= kLaItemEmpty && b < kLaItemEmpty + kLaItemSlots) count = 12;  // loads, 2 MMA warps, Q, 4 softmax warps, 4 that write out
        mbar_init(&bars[b], count);
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&a_map);
        tma_prefetch_desc(&b_map);
        tma_prefetch_desc(&q_map);
        *status = PKV_OK;
        *tiles = 0;
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, kLaTmemCols);
        tmem_relinquish();
    }
    fence_barrier_init();

    // this CTA's run [lo, hi) of the line of units, and the request that holds lo
    bool bad = false;
    int64_t units = 0;
    const LaReq first_req = threadIdx.x < p.num_seqs ? la_request(p, threadIdx.x, bad) : LaReq{};
    units = first_req.units;
    for (int r = threadIdx.x + kLaThreads; r < p.num_seqs; r += kLaThreads) units += la_request(p, r, bad).units;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) units += __shfl_xor_sync(0xffffffffu, units, m);
    if (lane == 0) scan[warp] = units;
    const bool any_bad = __syncthreads_or(bad);
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kLaThreads / 32; ++w) total += scan[w];
    const int64_t per = max(static_cast<int64_t>(1), (total + p.lanes - 1) / p.lanes);
    const int64_t lo = min(total, my_lane * per), hi = min(total, lo + per);
    __syncthreads();
    if (threadIdx.x == 0) scan[14] = -1;
    int64_t base = 0;
    for (int r0 = 0; r0 < p.num_seqs && lo < hi; r0 += kLaThreads) {
        const int r = r0 + threadIdx.x;
        int64_t mine = first_req.units;
        bool unused = false;
        if (r0 > 0) mine = r < p.num_seqs ? la_request(p, r, unused).units : 0;
        int64_t inc = mine;                                   // inclusive scan in the warp, then over the warps
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += y;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int64_t before = base + inc - mine, all = base;
#pragma unroll
        for (int w = 0; w < kLaThreads / 32; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
        if (lo >= before && lo < before + mine) {
            scan[14] = r;
            scan[15] = lo - before;
        }
        base = all;
        __syncthreads();
        if (all > lo) break;                                  // uniform
    }
    int start_req = 0;
    int64_t start_off = 0;
    if (lo < hi) {
        start_req = static_cast<int>(scan[14]);
        start_off = scan[15];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    // everything before this call is complete from here on: the cache write, the
    // query, and the previous use of the workspace
    pdl_wait();
    pdl_trigger();                        // the merge's CTAs may take their places (they wait for this grid)
    const bool work = lo < hi;
    // for the merge kernel, {first token, tokens, lanes that it runs across, this lane among them}: the row tile
    // that starts here and ends in another lane, and the one that started in an earlier lane
    int4 *desc = reinterpret_cast<int4 *>(p.ws + kLaWsDesc) + blockIdx.x;
    int4 *desc0 = reinterpret_cast<int4 *>(p.ws + kLaWsDesc0) + blockIdx.x;

    if (warp == 3) {
        // ---------------- walk of the run: items, ahead of the other warps ----------------
        bool ok = true;
        int r = start_req;
        int64_t off = start_off, left = hi - lo, at = lo;     // at: position in the line
        int4 split = make_int4(0, 0, 0, 0), split0 = split;
        bool unused = false;
        LaReq req = work ? la_request(p, r, unused) : LaReq{};
        for (int k = 0; ok; ++k) {
            const int slot = k % kLaItemSlots;
            if (k >= kLaItemSlots)
                ok = warp_wait_tiles(&bars[kLaItemEmpty + slot], (k / kLaItemSlots - 1) & 1, tiles, status);
            if (!ok) break;
            LaItem it{};
            while (left > 0 && !it.valid) {
                while (req.units == off) {                    // the next request with rows (there is one: left > 0)
                    ++r;
                    req = la_request(p, r, unused);
                    off = 0;
                }
                // the row tile that holds `off`: largest j with units_before(j) <= off
                int lo_j = 0, hi_j = req.n_full;
                while (lo_j < hi_j) {
                    const int mid = (lo_j + hi_j + 1) >> 1;
                    if (la_units_before(req.ctx, p.tpt_shift, mid) <= off) lo_j = mid;
                    else hi_j = mid - 1;
                }
                const int64_t before = la_units_before(req.ctx, p.tpt_shift, lo_j);
                // a row tile is kLaExtra units without keys, then its key tiles
                const int64_t pos = off - before - kLaExtra;
                it.r = r;
                it.tok0 = req.qs + lo_j * p.tpt;
                it.ntok = min(p.tpt, req.q - lo_j * p.tpt);
                it.lim0 = req.ctx + lo_j * p.tpt + 1;
                it.n_kv = (it.lim0 + it.ntok - 1 + kLaKeys - 1) / kLaKeys;
                const int64_t n = min(it.n_kv - pos, left);                  // its units in this run
                it.kv0 = static_cast<int32_t>(max(static_cast<int64_t>(0), pos));
                it.kv1 = static_cast<int32_t>(pos + n);
                it.valid = it.kv1 > it.kv0;                                  // (else it starts in the next lane)
                it.slot = it.kv0 > 0 ? 0 : (it.kv1 < it.n_kv ? 1 : -1);
                if (it.valid && it.slot >= 0) {
                    const int64_t first = (at - pos) / per, last = (at - pos + it.n_kv - 1) / per;   // lanes of its key tiles
                    const int4 d = make_int4(it.tok0, it.ntok, static_cast<int>(last - first) + 1,
                                             static_cast<int>(my_lane - first));
                    if (it.slot == 1) split = d;
                    else split0 = d;
                }
                off += n, at += n, left -= n;
            }
            if (lane == 0) {
                volatile int32_t *dst = reinterpret_cast<volatile int32_t *>(items + slot);
                const int32_t *src = reinterpret_cast<const int32_t *>(&it);
#pragma unroll
                for (int e = 0; e < static_cast<int>(sizeof(LaItem) / 4); ++e) dst[e] = src[e];
                mbar_arrive(&bars[kLaItemFull + slot]);
            }
            if (!it.valid) break;
        }
        if (lane == 0) *desc = split, *desc0 = split0;
    } else if (warp == 0) {
        // ---------------- pages through the block table ----------------
        bool ok = true;
        int gt = 0;                                           // key tiles of this CTA so far
        int issued = 0;                                       // parts whose copies were issued
        struct {
            bool valid;
            int kv0, kv1, n_pages;
            const int32_t *table;
        } cur, next{};
        // block ids in windows of 32 pages (8 key tiles), a lane each, loaded a window
        // ahead, and for the next item while the current one ends
        auto window = [&](int w) -> int {
            const int page = next.kv0 * kLaPages + w * 32 + lane;
            return next.valid && page < next.n_pages ? __ldg(next.table + page) : -1;
        };
        auto fetch = [&](int k) {
            const int slot = k % kLaItemSlots;
            ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status));
            const volatile LaItem *it = items + slot;
            next.valid = ok && it->valid;
            next.kv0 = it->kv0, next.kv1 = it->kv1;
            next.n_pages = (it->lim0 + it->ntok - 1 + kBlock - 1) / kBlock;    // with a key that the last token sees
            next.table = p.block_tables + static_cast<int64_t>(it->r) * p.max_blocks_per_seq;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
        };
        // Pages are brought into L2 kLaAhead tiles before they are loaded, the first ones of
        // an item while the one before ends: two stages of shared memory are too few to
        // cover memory's latency.  (256 requests of 128 heads: 99 us without, 96 us one tile
        // ahead, 97 two, 101 four, 109 eight.)  The CTAs of a lane share the pages out.
        auto prefetch = [&](int id, bool there) {
            if (there && id >= 0 && id < p.num_blocks && lane % p.groups == group)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.cache + static_cast<int64_t>(id) *
                                                                                              kLatPageBytes),
                             "r"(kLatPageBytes)
                             : "memory");
        };
        fetch(0);
        int win_cur = window(0), win_next = window(1);
        prefetch(win_cur, next.valid && lane < min(kLaAhead, next.kv1 - next.kv0) * kLaPages);
        for (int k = 0; ok && next.valid; ++k) {
            cur = next;
            int ahead0 = -1, ahead1 = -1;                     // the next item's first windows
            for (int j = cur.kv0; j < cur.kv1 && ok; ++j, ++gt) {
                const int st = gt % kLaStages;
                const int wofs = ((j - cur.kv0) * kLaPages) % 32;
                if (j > cur.kv0 && wofs == 0) {
                    win_cur = win_next;
                    win_next = window((j - cur.kv0) * kLaPages / 32 + 1);
                }
                // pages past the end, and ids outside the cache (reported), become -1: they
                // load as zeros
                int id = __shfl_sync(0xffffffffu, win_cur, wofs + (lane & (kLaPages - 1)));
                if (id < 0 || id >= p.num_blocks) {
                    if (j * kLaPages + (lane & (kLaPages - 1)) < cur.n_pages) set_status(status, PKV_ERR_DEVICE_INDEX);
                    id = -1;
                }
                {
                    // tile j + kLaAhead: in this window or the next
                    const int w = wofs + kLaAhead * kLaPages + (lane & (kLaPages - 1));
                    const int a = __shfl_sync(0xffffffffu, win_cur, w & 31), b = __shfl_sync(0xffffffffu, win_next, w & 31);
                    prefetch(w < 32 ? a : b, lane < kLaPages && j + kLaAhead < cur.kv1);
                }
                if (j == cur.kv1 - 1) {
                    fetch(k + 1);
                    if (!ok) break;
                    ahead0 = window(0), ahead1 = window(1);
                    prefetch(ahead0, next.valid && lane < min(kLaAhead, next.kv1 - next.kv0) * kLaPages);
                }
                // each part as soon as the products of the tile two before have read it
#pragma unroll 1
                for (int part = 0; part < 2 && ok; ++part) {
                    const int b = 2 * st + part;
                    if (gt >= kLaStages)
                        ok = __all_sync(0xffffffffu,
                                        pf_wait(&bars[kLaKVEmpty + b], (gt / kLaStages - 1) & 1, status));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars[kLaKVFull + b], part ? kLaPartB : kLaPartA);
                        *tiles = gt + 1;
                    }
                    __syncwarp();
                    if (lane < kLaPages)
                        tma_load_5d(smem + kLaOffKV + st * kLaStage + (part ? kLaPartA + lane * kLaPageB : lane * kLaPageA),
                                    part ? &b_map : &a_map, &bars[kLaKVFull + b], 0, 0, part ? kLaChunksA : 0, 0, id);
                    issued = 2 * gt + part + 1;
                }
            }
            win_cur = ahead0, win_next = ahead1;
        }
        // (after a failed wait: the copies in flight land before the CTA ends)
        for (int g = max(0, issued - 2 * kLaStages); g < issued && !ok; ++g)
            mbar_wait_bounded(&bars[kLaKVFull + g % (2 * kLaStages)], (g / (2 * kLaStages)) & 1);
    } else if (warp == 1) {
        // ---------------- S products (the warp stays converged) ----------------
        constexpr uint32_t kIdescS = idesc_bf16_f32(kLaRows, kLaKeys, 0, 0);
        // queries and keys K-major (8-key groups one stride apart)
        const uint64_t dq = smem_desc_sw128(sQ, 16, 1024);
        const uint64_t dka = smem_desc_sw128(sKV, 16, kLaGroupA), dkb = smem_desc_sw128(sKV + kLaPartA, 16, kLaGroupB);
        bool ok = true;
        int gt = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k % kLaItemSlots;
            ok = warp_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status);
            if (!ok) break;
            const bool valid = uniform(static_cast<int>(items[slot].valid)) != 0;
            const int n = uniform(items[slot].kv1 - items[slot].kv0);
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
            if (!valid) break;
            ok = warp_wait(&bars[kLaQFull], k & 1, status);
            for (int j = 0; j < n && ok; ++j, ++gt) {
                const int st = gt % kLaStages, sb = gt & 1;
                const uint32_t par = (gt / kLaStages) & 1;
                // the buffer's scores of the tile two before have been read
                if (gt >= 2) ok = warp_wait(&bars[kLaSFree + sb], ((gt >> 1) - 1) & 1, status);
                if (ok) ok = warp_wait(&bars[kLaKVFull + 2 * st], par, status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t so = static_cast<uint32_t>(st * (kLaStage >> 4));
                const uint32_t d = tmem + la_col_s(sb);
                const uint64_t ba = dka + so, bb = dkb + so;
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < kLaChunksA; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ss(d, dq + c * (kLaQChunk >> 4) + kk * 2, ba + c * (1024 >> 4) + kk * 2, kIdescS,
                                        (c | kk) ? 1u : 0u);
                }
                __syncwarp();
                ok = warp_wait(&bars[kLaKVFull + 2 * st + 1], par, status);
                if (!ok) break;
                tc_fence_after();
                const bool last = j == n - 1;
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < kLaChunksB; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ss(d, dq + (kLaChunksA + c) * (kLaQChunk >> 4) + kk * 2, bb + c * (1024 >> 4) + kk * 2,
                                        kIdescS, 1u);
                    umma_commit(&bars[kLaSFull + sb]);
                    if (last) umma_commit(&bars[kLaQEmpty]);
                }
                __syncwarp();
            }
        }
    } else if (warp == 8) {
        // ---------------- second products (the warp stays converged) ----------------
        // values MN-major (64-dim chunks 1024 apart), weights MN-major
        const uint64_t dva = smem_desc_sw128(sKV, 1024, kLaGroupA), dvb = smem_desc_sw128(sKV + kLaPartA, 1024, kLaGroupB);
        const uint64_t dw = smem_desc_sw128(sKV + kLaOffW, 16, kLaGroupB);
        bool ok = true;
        int gt = 0;
        uint32_t fix_par = 0, rescales = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k % kLaItemSlots;
            ok = warp_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status);
            if (!ok) break;
            const volatile LaItem *cur = items + slot;
            const bool valid = uniform(static_cast<int>(cur->valid)) != 0;
            const int n = uniform(cur->kv1 - cur->kv0);
            const int rows = uniform(cur->ntok * p.hpt);
            const int end = uniform(cur->lim0 + cur->ntok - 1);
            const bool fix = uniform(static_cast<int>(cur->kv1 == cur->n_kv && end % kBlock)) != 0;
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
            if (!valid) break;
            // N: the tile's rows, in sixteens
            const uint32_t idesc_o = idesc_bf16_f32(128, (rows + 15) & ~15, 1, 1);
            for (int j = 0; j < n && ok; ++j, ++gt) {
                const int st = gt % kLaStages;
                ok = warp_wait(&bars[kLaPFull + (gt & 1)], (gt >> 1) & 1, status);
                if (!ok) break;
                if (fix && j == n - 1) {
                    ok = warp_wait(&bars[kLaFix + st], (fix_par >> st) & 1u, status);
                    fix_par ^= 1u << st;
                }
                if (j > 0 && uniform(*reinterpret_cast<volatile const uint32_t *>(votes + 4 * (gt % kLaVotes)))) {
                    if (ok) ok = warp_wait(&bars[kLaRescaled], rescales & 1, status);
                    ++rescales;
                }
                // the previous item's O' has been read out, half by half
                if (ok && k > 0 && j == 0) ok = warp_wait(&bars[kLaOFree], (k - 1) & 1, status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t so = static_cast<uint32_t>(st * (kLaStage >> 4));
                const uint64_t a0 = dva + so, a1 = dvb + so, w0 = dw + so;
                const uint32_t more = j > 0 ? 1u : 0u;
                const bool last = j == n - 1;
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int kk = 0; kk < kLaPages; ++kk)
                            umma_f16_ss(tmem + 64u * m, a0 + kk * (kLaPageA >> 4) + m * (2048 >> 4),
                                        w0 + kk * (kLaPageB >> 4), idesc_o, kk > 0 ? 1u : more);
                    umma_commit(&bars[kLaKVEmpty + 2 * st]);
                }
                __syncwarp();
                if (k > 0 && j == 0) {
                    ok = warp_wait(&bars[kLaOFree2], (k - 1) & 1, status);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int kk = 0; kk < kLaPages; ++kk)
                            umma_f16_ss(tmem + 128u + 64u * m, a1 + kk * (kLaPageB >> 4) + m * (2048 >> 4),
                                        w0 + kk * (kLaPageB >> 4), idesc_o, kk > 0 ? 1u : more);
                    umma_commit(&bars[kLaKVEmpty + 2 * st + 1]);
                    umma_commit(&bars[kLaODone]);
                    if (last) umma_commit(&bars[kLaOReady]);
                }
                __syncwarp();
            }
        }
    } else if (warp == 2) {
        // ---------------- Q of each item; rows past its last visible key ----------------
        bool ok = true;
        int loaded = 0, gt = 0;
        int kv1 = 0, end = 0;                                 // of the item before
        bool fix = false;
        for (int k = 0; ok; ++k) {
            const int slot = k % kLaItemSlots;
            ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status));
            if (!ok) break;
            const volatile LaItem *it = items + slot;
            const bool valid = it->valid != 0;
            const int tok0 = it->tok0, n = it->kv1 - it->kv0;
            const int next_end = it->lim0 + it->ntok - 1, next_kv1 = it->kv1;
            const bool next_fix = valid && next_kv1 == it->n_kv && next_end % kBlock;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
            // the previous item's last S has read its Q (and that tile's keys)
            if (k > 0) ok = warp_wait_tiles(&bars[kLaQEmpty], (k - 1) & 1, tiles, status);
            if (!ok) break;
            if (valid) {
                // a box is 64 dims of the group's heads of tpt tokens; tokens past the batch
                // and heads past the last load as zeros, rows that no item holds are masked
                if (lane == 0) mbar_arrive_expect_tx(&bars[kLaQFull], kLaChunks * 128 * p.hpt * p.tpt);
                __syncwarp();
                if (lane < kLaChunks)
                    tma_load_3d(smem + kLaOffQ + lane * kLaQChunk, &q_map, &bars[kLaQFull], lane * 64, group * p.hpt,
                                tok0);
                loaded = k + 1;
            }
            if (fix) {
                // zero the rows past the previous item's last visible key, in its page, while
                // the softmax works on that tile
                const int st = (gt - 1) % kLaStages;
                const int first = end % kBlock;
                const int page = (end - 1) / kBlock - (kv1 - 1) * kLaPages;
                const uint32_t base = sKV + st * kLaStage + (lane >> 3) * 1024 + (lane & 7) * 16;   // a chunk of each part
                for (int t = first; t < kBlock; ++t) {                       // (the values' dims only)
                    const uint32_t g = 2 * page + (t >> 3), a = base + (t & 7) * 128;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a + g * kLaGroupA), "r"(0u) : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a + kLaPartA + g * kLaGroupB), "r"(0u)
                                 : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kLaFix + st]);
            }
            if (!valid) break;
            gt += n;
            fix = next_fix, end = next_end, kv1 = next_kv1;
        }
        if (loaded > 0) mbar_wait_bounded(&bars[kLaQFull], (loaded - 1) & 1);    // landed before the CTA ends
    } else if (warp < 8) {
        // ---------------- softmax ----------------
        const int quad = warp - 4;
        const float NEG_INF = -__int_as_float(0x7f800000);
        float *alphas = reinterpret_cast<float *>(smem + kLaOffAlpha);
        const int rA = quad * 16 + (lane >> 2);              // this thread's rows: rA and rA + 8
        const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const float sl2 = p.scale_log2;
        const int heads_here = min(p.hpt, p.heads - group * p.hpt);
        // After this warp's weights of tile g: if some warp voted for it, O' is rescaled
        // (its columns are rows of every warp, its lanes the quadrants of every warp),
        // between the products of tile g - 1 and those of g.
        auto rescale = [&](int g) -> bool {
            if (!__all_sync(0xffffffffu, pf_wait(&bars[kLaPFull + (g & 1)], (g >> 1) & 1, status))) return false;
            const uint32_t vote = *reinterpret_cast<volatile const uint32_t *>(votes + 4 * (g % kLaVotes));
            if (!vote) return true;
            if (!__all_sync(0xffffffffu, pf_wait(&bars[kLaODone], (g - 1) & 1, status))) return false;
            tc_fence_after();
            const float *al = alphas + (g & 1) * kLaRows;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {                     // 32 rows of one 128-dim block at a time
                uint32_t v[32];
                const uint32_t a = tlane + 64u * (c >> 1) + 32u * (c & 1);
                tmem_ld32(a, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e)                  // (a warp that did not vote wrote no factors)
                    if ((vote >> (8 * (2 * (c & 1) + (e >> 4)))) & 0xffu)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * al[32 * (c & 1) + e]);
                tmem_st32(a, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaRescaled]);
            return true;
        };
        // this thread's two rows of every tile: token, head
        int row_tok[2], row_head[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            row_tok[i] = (rA + 8 * i) / p.hpt;
            row_head[i] = rA + 8 * i - row_tok[i] * p.hpt;
        }
        bool ok = true;
        int gt = 0;
        for (int k = 0;; ++k) {
            const int slot = k % kLaItemSlots;
            ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status));
            if (!ok) break;
            const volatile LaItem *cur = items + slot;
            if (!cur->valid) break;
            const int kv0 = cur->kv0, kv1 = cur->kv1, ntok = cur->ntok, lim0 = cur->lim0, tok0 = cur->tok0;
            const int part = cur->slot;
            const int rows = ntok * p.hpt, end = lim0 + ntok - 1;
            int lim[2], dst[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = row_tok[i] < ntok && row_head[i] < heads_here;
                // (a row that no head owns computes what it finds, for nobody, rather than put
                // its warp on the masked path)
                lim[i] = in ? lim0 + row_tok[i] : INT32_MAX;
                dst[i] = in ? (tok0 + row_tok[i]) * p.heads + group * p.hpt + row_head[i] : -1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
            float m_ref[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};
            // Rows of tile j that some tokens see and others do not, with an infinity or NaN among
            // their values: zeroed.  (S has been computed from them: the tokens that see one have
            // weights that are no numbers.)
            auto clear_odd_rows = [&](int j) {
                for (int part = 0; part < 2; ++part)          // (landed, as S shows; this thread has to see it)
                    pf_wait(&bars[kLaKVFull + 2 * (gt % kLaStages) + part], (gt / kLaStages) & 1, status);
                for (int t = max(lim0 - j * kLaKeys, 0); t < min(kLaKeys, end - j * kLaKeys); ++t) {
                    const uint32_t a = sKV + (gt % kLaStages) * kLaStage + (lane >> 3) * 1024 + (lane & 7) * 16 + (t & 7) * 128;
                    const uint32_t at[2] = {a + (t >> 3) * kLaGroupA, a + kLaPartA + (t >> 3) * kLaGroupB};
                    bool bad = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                     : "r"(at[h])
                                     : "memory");
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bad |= (v[e] & 0x7F80u) == 0x7F80u || (v[e] & 0x7F800000u) == 0x7F800000u;
                    }
                    if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at[h]), "r"(0u) : "memory");
                }
            };
            for (int j = kv0; j < kv1 && ok; ++j, ++gt) {
                const int sb = gt & 1;
                ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaSFull + sb], (gt >> 1) & 1, status));
                if (!ok) break;
                tc_fence_after();
                float s[32];
                tmem_ld_16x64f(tlane + la_col_s(sb), s);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kLaSFree + sb]);
                const int key0 = j * kLaKeys + 2 * (lane & 3);
                const bool masked = __any_sync(0xffffffffu, (j + 1) * kLaKeys > min(lim[0], lim[1]));
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] *= sl2;
                if (masked) {
                    // A score that this row does not see but a later one does: where it is no number,
                    // an infinity or NaN may lie in the key's row, which must not meet a weight of 0
                    // (0 x NaN).  `odd` stays 0 as long as every such score is finite.
                    float odd = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int key = key0 + (e >> 2) * 8 + (e & 1);
                        if (key >= lim[(e >> 1) & 1]) {
                            if (key < end) odd = fmaf(s[e], 0.f, odd);
                            s[e] = NEG_INF;
                        }
                    }
                    if (__any_sync(0xffffffffu, odd != 0.f)) clear_odd_rows(j);
                }
                // The reference moves on a row's first visible key, and then only when some
                // score exceeds it by 2^40: fp32 sums and bf16 weights keep their relative
                // accuracy at any common scale, and 2^40 leaves 2^87 of range.  So most tiles
                // need no row maximum, only each thread's own.
                float mx[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float a = fmaxf(s[2 * i], s[2 * i + 1]), b = fmaxf(s[4 + 2 * i], s[4 + 2 * i + 1]);
#pragma unroll
                    for (int c = 8; c < 32; c += 8) {
                        a = fmax3(a, s[c + 2 * i], s[c + 2 * i + 1]);
                        b = fmax3(b, s[c + 4 + 2 * i], s[c + 4 + 2 * i + 1]);
                    }
                    mx[i] = fmaxf(a, b);
                }
                bool grow = false;
                if (__any_sync(0xffffffffu, mx[0] > m_ref[0] + 40.f || mx[1] > m_ref[1] + 40.f)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                        const bool first = m_ref[i] == NEG_INF;
                        const bool g = !first && mx[i] > m_ref[i] + 40.f;
                        const float alpha = g ? fast_exp2(m_ref[i] - mx[i]) : 1.f;
                        if (first || g) m_ref[i] = mx[i];
                        l[i] *= alpha;
                        if ((lane & 3) == 0) alphas[sb * kLaRows + rA + 8 * i] = alpha;
                        grow |= g;
                    }
                    grow = __any_sync(0xffffffffu, grow);
                }
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float ref = m_ref[i] == NEG_INF ? 0.f : m_ref[i];
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float a = fast_exp2(s[4 * c + 2 * i] - ref), b = fast_exp2(s[4 * c + 2 * i + 1] - ref);
                        sum += a + b;
                        w[2 * c + i] = pack_bf16x2(a, b);
                    }
                    l[i] += sum;
                }
                // weights of 16 rows and 64 keys, transposed by stmatrix into rows of a key, over
                // the stage's rotated chunk (which S has read)
                const uint32_t sW = sKV + (gt % kLaStages) * kLaStage + kLaOffW;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    const int i = lane & 7, m = lane >> 3;    // key in its group; tile: group c + m / 2, rows m % 2
                    stsm_x4_trans(sW + (c + (m >> 1)) * kLaGroupB + i * 128 + (((2 * quad + (m & 1)) ^ i) << 4),
                                  w[2 * c], w[2 * c + 1], w[2 * c + 2], w[2 * c + 3]);
                }
                if (lane == 0) votes[4 * (gt % kLaVotes) + quad] = grow ? 1 : 0;
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kLaPFull + sb]);
                if (j > kv0) ok = rescale(gt);
            }
            // the rows' sums and places, for the warps that write the item out
            const int rb = k & 1;
            if (ok && k >= 2) ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaRowFree + rb], ((k >> 1) - 1) & 1, status));
            if (!ok) break;
            LaRows *rec = reinterpret_cast<LaRows *>(smem + kLaOffRow + rb * kLaRowsBytes);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            }
            if ((lane & 3) == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = rA + 8 * i;
                    rec->inv[row] = l[i] <= 0.f ? 0.f : 1.f / l[i];       // (NaN stays)
                    rec->dst[row] = dst[i];
                    if (part >= 0) {
                        float *ml = reinterpret_cast<float *>(p.ws + kLaWsMl) +
                                    (static_cast<int64_t>(blockIdx.x) * 2 + part) * 2 * kLaRows;
                        ml[row] = l[i] == l[i] ? m_ref[i] : -NEG_INF;        // (a NaN stays one in the merge)
                        ml[kLaRows + row] = l[i];
                    }
                }
            }
            if (warp == 4 && lane == 0) rec->rows = rows, rec->slot = part;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaRowFull + rb]);
        }
    } else {
        // ---------------- finished tiles to memory (warps 9-12) ----------------
        const int quad = warp & 3;
        const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t stage = sOut + quad * 2048;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k % kLaItemSlots;
            ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaItemFull + slot], (k / kLaItemSlots) & 1, status));
            if (!ok) break;
            const bool valid = items[slot].valid != 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kLaItemEmpty + slot]);
            if (!valid) break;
            const int rb = k & 1;
            ok = warp_wait_tiles(&bars[kLaRowFull + rb], (k >> 1) & 1, tiles, status);
            if (ok) ok = __all_sync(0xffffffffu, pf_wait(&bars[kLaOReady], k & 1, status));
            if (!ok) break;
            tc_fence_after();
            const LaRows *rec = reinterpret_cast<const LaRows *>(smem + kLaOffRow + rb * kLaRowsBytes);
            const int rows = rec->rows, part = rec->slot;
            // blocks of 128 dims x 32 rows, dims first
            auto half_read = [&]() {                          // dims 0 .. 255 of O' have been read out
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kLaOFree]);
            };
            auto write = [&](auto two) {                      // rows beyond the first 32, or none
                constexpr int kH = decltype(two)::value ? 2 : 1, kBlocks = 4 * kH;
                if (part >= 0) {
                    // [128-dim block][row / 4][dim][row % 4]
                    float *po = reinterpret_cast<float *>(p.ws + kLaWsO) +
                                (static_cast<int64_t>(blockIdx.x) * 2 + part) * kLaPartFloats + (quad * 32 + lane) * 4;
                    float v[2][32];                             // the next block's loads run beside the stores
                    tmem_ld32f(tlane, v[0]);
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i) {
                        tmem_ld_wait();
                        if (i == kBlocks / 2 - 1) half_read();
                        if (i + 1 < kBlocks)
                            tmem_ld32f(tlane + 64u * ((i + 1) / kH) + 32u * ((i + 1) % kH), v[(i + 1) & 1]);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            if (32 * (i % kH) + e < rows)
                                *reinterpret_cast<float4 *>(po + (i / kH * 16 + 8 * (i % kH) + e / 4) * 512) =
                                    make_float4(v[i & 1][e], v[i & 1][e + 1], v[i & 1][e + 2], v[i & 1][e + 3]);
                    }
                    return;
                }
                // 32 dims x 32 rows at a time through 2 KiB of shared memory, transposed by
                // stmatrix into rows of 64 bytes (64-byte swizzle).  The tile's rows lie one after
                // another in `out`: 32 of them leave as one TMA store (stores of the lanes would
                // queue in front of the softmax warps' shuffles), fewer by 16-byte stores.  Block
                // i + 1 is packed while block i leaves.
                float a[16], b[16];                             // dims t / 4 (+ 8), and 16 further
                uint32_t w[16];
                uint4 out[4];
                auto fetch = [&](int i) {
                    tmem_ld_16x32f(tlane + 64u * (i / kH) + 32u * (i % kH), a);
                    tmem_ld_16x32f(tlane + (16u << 16) + 64u * (i / kH) + 32u * (i % kH), b);
                };
                auto pack = [&](int i) {
                    tmem_ld_wait();
                    if (i == kBlocks / 2 - 1) half_read();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {               // rows 8 e ..
                        const float2 s = *reinterpret_cast<const float2 *>(rec->inv + 32 * (i % kH) + 8 * e + 2 * (lane & 3));
                        w[4 * e] = pack_bf16x2(a[4 * e] * s.x, a[4 * e + 1] * s.y);
                        w[4 * e + 1] = pack_bf16x2(a[4 * e + 2] * s.x, a[4 * e + 3] * s.y);
                        w[4 * e + 2] = pack_bf16x2(b[4 * e] * s.x, b[4 * e + 1] * s.y);
                        w[4 * e + 3] = pack_bf16x2(b[4 * e + 2] * s.x, b[4 * e + 3] * s.y);
                    }
                };
                fetch(0);
                pack(0);
#pragma unroll 2
                for (int i = 0; i < kBlocks; ++i) {
                    if (i + 1 < kBlocks) fetch(i + 1);
                    const int first = rec->dst[32 * (i % kH)];
                    const bool whole = first >= 0 && rec->dst[32 * (i % kH) + 31] >= 0;
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();                               // the block before has been read
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 8 * e + (lane & 7);
                        stsm_x4_trans(stage + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4), w[4 * e], w[4 * e + 1],
                                      w[4 * e + 2], w[4 * e + 3]);
                    }
                    if (whole) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&out_map, stage, 128 * (i / kH) + 32 * quad, first);
                        if (i + 1 < kBlocks) pack(i + 1);
                        continue;
                    }
                    __syncwarp();
                    int dst[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 8 * e + (lane >> 2);
                        dst[e] = rec->dst[32 * (i % kH) + row];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(out[e].x), "=r"(out[e].y), "=r"(out[e].z), "=r"(out[e].w)
                                     : "r"(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4))
                                     : "memory");
                    }
                    if (i + 1 < kBlocks) pack(i + 1);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (dst[e] >= 0)
                            *reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(dst[e]) * kLatent + 128 * (i / kH) +
                                                       quad * 32 + (lane & 3) * 8) = out[e];
                }
            };
            if (rows > 32) write(std::true_type{});
            else write(std::false_type{});
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[kLaOFree2]);
                mbar_arrive(&bars[kLaRowFree + rb]);
            }
        }
        if (lane == 0) bulk_wait();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kLaTmemCols);
    }
    if (threadIdx.x == 0) {
        int32_t s = *reinterpret_cast<volatile int32_t *>(status);
        if (s == PKV_OK && any_bad) s = PKV_ERR_DEVICE_METADATA;
        reinterpret_cast<int32_t *>(p.ws + kLaWsStatus)[blockIdx.x] = s;
        // the call's own word starts afresh, before any CTA of the merge looks at it: those only
        // add errors to it, and the first one stays
        if (blockIdx.x == 0) *reinterpret_cast<int32_t *>(p.ws) = PKV_OK;
    }
}

// Merge of the row tiles that run across lanes, and the call's status word.
// Piece i of the tile that starts in CTA c lies in CTA c + i * groups, slot 1
// for the first and 0 for the others:
//     out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
// The merge is one trip to memory that the first kernel has just written, and
// nothing else.  Two kernels, by what a call can hold:
//  - many row tiles, so that of like lengths most have two pieces and nearly every
//    lane starts one: latent_merge_kernel, a CTA for 128 dims of a lane's tile, which takes
//    the two pieces in bulk into shared memory (64 KiB a CTA, three CTAs an SM: twice
//    what registers could have in flight; 256 requests of 128 heads, 40 MB: 15 us by
//    registers) before it knows whether there is a tile to merge, and any further pieces one
//    after another (a request far longer than the others has them, and waits for them);
//  - few, so that every tile can have many pieces (a long request on an otherwise idle GPU):
//    latent_merge_few_kernel, which shares a tile of many pieces out over the CTAs
//    of its first four lanes by rows, and in each over two halves of the pieces
//    (1000 keys of one request, 16 heads: 15.4 us with one after another, 11.6 us).

// The call's status: the first error of its CTAs (beside one that a CTA of the merge itself adds).
__device__ __forceinline__ void la_collect_status(const LaParams &p, int ctas) {
    if (blockIdx.x != 0 || blockIdx.y != 0 || threadIdx.x >= 32) return;
    int32_t s = 0;
    for (int c = threadIdx.x; c < ctas; c += 32) {
        const int32_t x = reinterpret_cast<const int32_t *>(p.ws + kLaWsStatus)[c];
        s = s ? s : x;
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int32_t y = __shfl_down_sync(0xffffffffu, s, m);
        s = s ? s : y;
    }
    if (threadIdx.x == 0 && s) set_status(reinterpret_cast<int32_t *>(p.ws), s);
}

// Four rows (4 r4 ..) of one dim a thread to `out`: neighbouring lanes exchange a
// row each, 4-byte stores.  d: {first token, tokens, ..} of the tile.
__device__ __forceinline__ void la_store_rows(const LaParams &p, const int4 &d, int group, int r4, int m, int dim,
                                              const float (&y)[4]) {
    const bool odd = dim & 1;
    const int heads_here = min(p.hpt, p.heads - group * p.hpt);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? y[e] : y[e + 1], 1);
        const int row = r4 * 4 + e + (odd ? 1 : 0), tok = row / p.hpt, h = row - tok * p.hpt;
        if (row < d.y * p.hpt && h < heads_here)
            *reinterpret_cast<uint32_t *>(p.out +
                                          (static_cast<int64_t>(d.x + tok) * p.heads + group * p.hpt + h) * kLatent +
                                          m * 128 + (dim & ~1)) =
                odd ? pack_bf16x2(got, y[e + 1]) : pack_bf16x2(y[e], got);
    }
}

// f v, where a piece's factor is 0 whatever its sums hold is not used
__device__ __forceinline__ float la_weigh(float f, float v) { return f == 0.f ? 0.f : f * v; }

// 128 dims of a piece of the rows that a tile can have: at most 32 KiB
__host__ __device__ __forceinline__ uint32_t la_merge_bytes(const LaParams &p) {
    return static_cast<uint32_t>((p.hpt * p.tpt + 3) / 4) * 2048;
}
constexpr uint32_t kLaMergeExtra = 2 * kLaRows * 4 + 16;     // factors, barriers
constexpr uint32_t kLaMergeMost = 2 * kLaRows * 128 * 4 + kLaMergeExtra;

__global__ void __launch_bounds__(256) latent_merge_kernel(const LaParams p, int ctas) {
    pdl_trigger();                        // a following call may start looking at its lengths
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t bytes = la_merge_bytes(p);
    float *factor = reinterpret_cast<float *>(smem_raw + 2 * bytes);                  // [2][64]
    uint64_t *bars = reinterpret_cast<uint64_t *>(factor + 2 * kLaRows);
    if (threadIdx.x < 2) mbar_init(&bars[threadIdx.x], 1);
    fence_barrier_init();
    __syncthreads();
    pdl_wait();
    const int cta = blockIdx.x, m = blockIdx.y, dim = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int group = cta % p.groups, row = threadIdx.x;     // (of the first 64 threads)
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float *ml = reinterpret_cast<const float *>(p.ws + kLaWsMl);
    auto part_of = [&](int i) { return static_cast<int64_t>(min(cta + i * p.groups, ctas - 1)) * 2 + (i == 0 ? 1 : 0); };
    auto load = [&](int i, int b) {                          // (one thread)
        mbar_arrive_expect_tx(&bars[b], bytes);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(smem_raw + b * bytes)),
                     "l"(reinterpret_cast<const float *>(p.ws + kLaWsO) + part_of(i) * kLaPartFloats + m * kLaRows * 128),
                     "r"(bytes), "r"(smem_u32(&bars[b]))
                     : "memory");
    };
    if (threadIdx.x == 0) load(0, 0), load(1, 1);
    float m0 = NEG_INF, l0 = 0.f, m1 = NEG_INF, l1 = 0.f;
    if (row < kLaRows) {
        const float *a = ml + part_of(0) * 2 * kLaRows + row, *b = ml + part_of(1) * 2 * kLaRows + row;
        m0 = a[0], l0 = a[kLaRows], m1 = b[0], l1 = b[kLaRows];
    }
    const int4 d = reinterpret_cast<const int4 *>(p.ws + kLaWsDesc)[cta];
    la_collect_status(p, ctas);
    const int pieces = d.z, rows = d.y * p.hpt;
    if (pieces < 2) {                                        // the loads land before the CTA ends
        if (threadIdx.x == 0) mbar_wait_bounded(&bars[0], 0), mbar_wait_bounded(&bars[1], 0);
        return;
    }
    float M = fmaxf(m0, m1), inv = 0.f;
    if (row < kLaRows) {
        for (int i = 2; i < pieces; ++i) M = fmaxf(M, ml[part_of(i) * 2 * kLaRows + row]);
        const float w0 = m0 == NEG_INF ? 0.f : fast_exp2(m0 - M), w1 = m1 == NEG_INF ? 0.f : fast_exp2(m1 - M);
        float L = la_weigh(w0, l0) + la_weigh(w1, l1);
        for (int i = 2; i < pieces; ++i) {
            const float mi = ml[part_of(i) * 2 * kLaRows + row];
            L += la_weigh(mi == NEG_INF ? 0.f : fast_exp2(mi - M), ml[part_of(i) * 2 * kLaRows + kLaRows + row]);
        }
        inv = L <= 0.f ? 0.f : 1.f / L;                      // (NaN stays)
        factor[row] = w0 * inv;
        factor[kLaRows + row] = w1 * inv;
    }
    // (the factors are there too; and every thread takes the same way)
    bool ok = __syncthreads_and(mbar_wait_bounded(&bars[0], 0) && mbar_wait_bounded(&bars[1], 0));
    float4 acc[8];                                           // rows 32 half + 4 q ..
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int r4 = half * 8 + q;
        if (r4 * 4 >= rows) break;
        const float4 a = *reinterpret_cast<const float4 *>(smem_raw + (r4 * 128 + dim) * 16);
        const float4 b = *reinterpret_cast<const float4 *>(smem_raw + bytes + (r4 * 128 + dim) * 16);
        const float4 f = *reinterpret_cast<const float4 *>(factor + r4 * 4);
        const float4 g = *reinterpret_cast<const float4 *>(factor + kLaRows + r4 * 4);
        acc[q] = make_float4(la_weigh(f.x, a.x) + la_weigh(g.x, b.x), la_weigh(f.y, a.y) + la_weigh(g.y, b.y),
                             la_weigh(f.z, a.z) + la_weigh(g.z, b.z), la_weigh(f.w, a.w) + la_weigh(g.w, b.w));
    }
#pragma unroll 1
    for (int i = 2; i < pieces && ok; ++i) {                 // further pieces, one after another
        __syncthreads();
        if (threadIdx.x == 0) {
            fence_proxy_async_smem();
            load(i, 0);
        }
        if (row < kLaRows) {
            const float mi = ml[part_of(i) * 2 * kLaRows + row];
            factor[row] = mi == NEG_INF ? 0.f : fast_exp2(mi - M) * inv;
        }
        ok = __syncthreads_and(mbar_wait_bounded(&bars[0], (i - 1) & 1));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r4 = half * 8 + q;
            if (r4 * 4 >= rows) break;
            const float4 a = *reinterpret_cast<const float4 *>(smem_raw + (r4 * 128 + dim) * 16);
            const float4 f = *reinterpret_cast<const float4 *>(factor + r4 * 4);
            acc[q].x += la_weigh(f.x, a.x), acc[q].y += la_weigh(f.y, a.y);
            acc[q].z += la_weigh(f.z, a.z), acc[q].w += la_weigh(f.w, a.w);
        }
    }
    if (!ok) {
        set_status(reinterpret_cast<int32_t *>(p.ws), PKV_ERR_DEVICE_TIMEOUT);
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int r4 = half * 8 + q;
        if (r4 * 4 >= rows) break;
        const float y[4] = {acc[q].x, acc[q].y, acc[q].z, acc[q].w};
        la_store_rows(p, d, group, r4, m, dim, y);
    }
}

// Pieces from which a tile is shared out: 16 heads, one request of 512 keys (8 pieces): 10.5 us shared
// out, 11.6 not; 20000 keys (152): 21.8 and 55.9.  From four on (16 requests of 4000 keys, 128 heads, five
// or six pieces each): 43.6 where eight give 39.6.
constexpr int kLaMany = 8;

// blockIdx.y: 128 dims x 16 rows; a thread takes one dim of eight rows.
__global__ void __launch_bounds__(256) latent_merge_few_kernel(const LaParams p, int ctas) {
    pdl_trigger();
    pdl_wait();
    la_collect_status(p, ctas);
    constexpr int kQ = 2;                                             // groups of four rows a thread
    const int cta = blockIdx.x, group = cta % p.groups;
    const int m = blockIdx.y >> 2, dim = threadIdx.x & 127, half = threadIdx.x >> 7;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float *ml = reinterpret_cast<const float *>(p.ws + kLaWsMl);
    const float *o = reinterpret_cast<const float *>(p.ws + kLaWsO) + dim * 4;
    const int4 d = reinterpret_cast<const int4 *>(p.ws + kLaWsDesc)[cta];
    const int4 d0 = reinterpret_cast<const int4 *>(p.ws + kLaWsDesc0)[cta];
    {
        const int r4 = (blockIdx.y & 3) * 4 + half * kQ;
        float4 mx[kQ], ls[kQ], acc[kQ], m1[kQ], l1[kQ], a1[kQ];
        auto load = [&](int64_t part, float4 (&a)[kQ], float4 (&b)[kQ], float4 (&c)[kQ]) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                a[q] = *reinterpret_cast<const float4 *>(ml + part * 2 * kLaRows + (r4 + q) * 4);
                b[q] = *reinterpret_cast<const float4 *>(ml + part * 2 * kLaRows + kLaRows + (r4 + q) * 4);
                c[q] = *reinterpret_cast<const float4 *>(o + part * kLaPartFloats + (m * 16 + r4 + q) * 512);
            }
        };
        // two softmax states into one; a state that saw no key has m = -inf, and whatever its sums hold is not used
        auto join = [&](float &m0, float &l0, float &a0, float m1, float l1, float a1) {
            const float M = fmaxf(m0, m1);
            const float w0 = m0 == NEG_INF ? 0.f : fast_exp2(m0 - M), w1 = m1 == NEG_INF ? 0.f : fast_exp2(m1 - M);
            l0 = la_weigh(w0, l0) + la_weigh(w1, l1);
            a0 = la_weigh(w0, a0) + la_weigh(w1, a1);
            m0 = M;
        };
        load(static_cast<int64_t>(cta) * 2 + 1, mx, ls, acc);
        load(static_cast<int64_t>(min(cta + p.groups, ctas - 1)) * 2, m1, l1, a1);
        if (d.z >= 2 && d.z < kLaMany && r4 * 4 < d.y * p.hpt) {      // (whole warps)
#pragma unroll 1
            for (int i = 1;;) {
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    join(mx[q].x, ls[q].x, acc[q].x, m1[q].x, l1[q].x, a1[q].x);
                    join(mx[q].y, ls[q].y, acc[q].y, m1[q].y, l1[q].y, a1[q].y);
                    join(mx[q].z, ls[q].z, acc[q].z, m1[q].z, l1[q].z, a1[q].z);
                    join(mx[q].w, ls[q].w, acc[q].w, m1[q].w, l1[q].w, a1[q].w);
                }
                if (++i >= d.z) break;
                load(static_cast<int64_t>(cta + i * p.groups) * 2, m1, l1, a1);
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const float v[4] = {acc[q].x, acc[q].y, acc[q].z, acc[q].w}, l[4] = {ls[q].x, ls[q].y, ls[q].z, ls[q].w};
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = l[e] <= 0.f ? 0.f : v[e] / l[e];
                la_store_rows(p, d, group, r4 + q, m, dim, y);
            }
        }
    }

    __shared__ float4 factor[kLaMaxCtas];                             // of a piece, for four rows
    __shared__ float4 other[128];
    auto many = [&](const int4 &d) {
        const int first = cta - d.w * p.groups, pieces = d.z;
        const int r4 = (blockIdx.y & 3) * 4 + d.w;
        if (d.z < kLaMany || d.w >= 4 || r4 * 4 >= d.y * p.hpt) return;   // (the whole CTA)
        auto part_of = [&](int i) { return static_cast<int64_t>(first + i * p.groups) * 2 + (i == 0 ? 1 : 0); };
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (warp < 4) {                                               // a row a warp
            const float *row = ml + r4 * 4 + warp;
            float M = NEG_INF, L = 0.f;
            for (int i = lane; i < pieces; i += 32) M = fmaxf(M, row[part_of(i) * 2 * kLaRows]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            for (int i = lane; i < pieces; i += 32) {
                const float mi = row[part_of(i) * 2 * kLaRows];
                const float w = mi == NEG_INF ? 0.f : fast_exp2(mi - M);
                if (w != 0.f) L = fmaf(w, row[part_of(i) * 2 * kLaRows + kLaRows], L);
                reinterpret_cast<float *>(factor + i)[warp] = w;
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
            const float inv = L <= 0.f ? 0.f : 1.f / L;
            for (int i = lane; i < pieces; i += 32) reinterpret_cast<float *>(factor + i)[warp] *= inv;
        }
        __syncthreads();
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int i = half; i < pieces; i += 2) {
            const float4 v = *reinterpret_cast<const float4 *>(o + part_of(i) * kLaPartFloats + (m * 16 + r4) * 512);
            const float4 f = factor[i];
            y[0] += la_weigh(f.x, v.x), y[1] += la_weigh(f.y, v.y);
            y[2] += la_weigh(f.z, v.z), y[3] += la_weigh(f.w, v.w);
        }
        if (half) other[dim] = make_float4(y[0], y[1], y[2], y[3]);
        __syncthreads();
        if (!half) {
            const float4 v = other[dim];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
            la_store_rows(p, d, group, r4, m, dim, y);
        }
        __syncthreads();                                              // (the other tile's turn)
    };
    many(d);
    many(d0);
}

// ---- host side --------------------------------------------------------------------

// {64 dims, 8 tokens, 9 chunks, 2 halves, blocks}: a box {64, 8, chunks, 2, 1} is
// that many chunks of one page.
static int make_latent_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int chunks) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    const cuuint64_t dims[5] = {64, 8, kLaChunks, 2, static_cast<cuuint64_t>(num_blocks)};
    const cuuint64_t strides[4] = {kLatRowBytes, 128, 8 * kLatRowBytes, kLatPageBytes};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(chunks), 2, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(cache), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

// {512 dims, token x head rows} of the output: a box is 32 dims of 32 rows.
static int make_latent_out_map(CUtensorMap *map, void *out, int64_t rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    const cuuint64_t dims[2] = {kLatent, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {kLatent * 2};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t es[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

// {576 dims, heads, tokens}: a box is 64 dims of hpt heads of tpt tokens.
static int make_latent_query_map(CUtensorMap *map, const void *query, int64_t q_stride, const LaParams &p) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return PKV_ERR_CUDA;
    const cuuint64_t dims[3] = {kLatRow, static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.num_tokens)};
    const cuuint64_t strides[2] = {kLatRowBytes, static_cast<cuuint64_t>(q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.hpt), static_cast<cuuint32_t>(p.tpt)};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(query), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // namespace pkv

extern "C" int pkv_latent_paged_attn(void *out, const void *query, int64_t query_token_stride,
                                     const void *latent_cache, int64_t num_blocks, const int32_t *block_tables,
                                     int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                     const int32_t *query_start_loc, int32_t num_seqs, int32_t num_tokens,
                                     int32_t max_query_len, int32_t max_seq_len, int32_t num_heads,
                                     int32_t block_size, float scale, void *workspace, size_t workspace_bytes,
                                     size_t *workspace_needed, void *stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || max_seq_len < 0 || max_blocks_per_seq < 0 ||
        num_heads <= 0 || num_blocks <= 0)
        return PKV_ERR_SHAPE;
    if (block_size != kBlock || num_heads > kLaMaxHeads) return PKV_ERR_UNSUPPORTED;
    if (num_blocks > INT32_MAX || static_cast<int64_t>(num_tokens) * num_heads > INT32_MAX) return PKV_ERR_SHAPE;
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return PKV_ERR_SHAPE;
    if (workspace_needed) *workspace_needed = kLaWsBytes;
    if (num_seqs == 0) {
        if (num_tokens) return PKV_ERR_SHAPE;
        // no request: of the call's results there is the status word alone (without a workspace
        // this is the size query)
        if (workspace && workspace_bytes >= static_cast<size_t>(kLaWsBytes) &&
            cudaMemsetAsync(workspace, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return PKV_ERR_CUDA;
        return PKV_OK;
    }
    if (max_query_len > max_seq_len || max_seq_len > INT32_MAX - 128) return PKV_ERR_SHAPE;
    if ((static_cast<int64_t>(max_seq_len) + kBlock - 1) / kBlock > max_blocks_per_seq) return PKV_ERR_SHAPE;
    if (!workspace || workspace_bytes < static_cast<size_t>(kLaWsBytes)) return PKV_ERR_WORKSPACE;
    if (!block_tables || !seq_lens || !query_start_loc || !latent_cache) return PKV_ERR_NULL;
    if (num_tokens > 0 && (!out || !query)) return PKV_ERR_NULL;
    if (query_token_stride < static_cast<int64_t>(num_heads) * kLatRow) return PKV_ERR_SHAPE;
    if (query_token_stride >= (int64_t(1) << 38)) return PKV_ERR_SHAPE;
    if (query_token_stride % 8) return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(query) |
         reinterpret_cast<uintptr_t>(latent_cache)) & 15u)
        return PKV_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
         reinterpret_cast<uintptr_t>(query_start_loc)) & 3u)
        return PKV_ERR_ALIGNMENT;

    LaParams p;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.seq_lens = seq_lens, p.qsl = query_start_loc;
    p.num_seqs = num_seqs, p.num_tokens = num_tokens;
    p.max_query_len = max_query_len, p.max_seq_len = max_seq_len;
    p.heads = num_heads;
    p.groups = (num_heads + kLaRows - 1) / kLaRows;
    p.hpt = (num_heads + p.groups - 1) / p.groups;
    p.tpt = 1;
    if (p.groups == 1)
        while (2 * p.tpt * p.hpt <= kLaRows && p.tpt < max_query_len) p.tpt *= 2;
    p.tpt_shift = 0;
    while ((1 << p.tpt_shift) < p.tpt) ++p.tpt_shift;
    p.cache = static_cast<const uint8_t *>(latent_cache);
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.ws = static_cast<uint8_t *>(workspace);

    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return PKV_ERR_CUDA;
    p.lanes = (sms < kLaMaxCtas ? sms : kLaMaxCtas) / p.groups;
    // no more lanes than the bounds leave units for
    const int64_t most = static_cast<int64_t>(num_seqs) * ((max_query_len + p.tpt - 1) / p.tpt);     // row tiles
    if (most < p.lanes) {                          // (the product of loose bounds can pass 64 bits)
        const int64_t units = most * ((max_seq_len + kLaKeys - 1) / kLaKeys + kLaExtra);
        if (units < p.lanes) p.lanes = units > 1 ? static_cast<int32_t>(units) : 1;
    }
    const int ctas = p.lanes * p.groups;
    CUtensorMap am, bm, qm, om;
    int rc = make_latent_map(&am, latent_cache, num_blocks, kLaChunksA);
    if (!rc) rc = make_latent_map(&bm, latent_cache, num_blocks, kLaChunksB);
    if (rc) return rc;
    if (num_tokens > 0) {
        rc = make_latent_query_map(&qm, query, query_token_stride, p);
        if (!rc) rc = make_latent_out_map(&om, out, static_cast<int64_t>(num_tokens) * num_heads);
        if (rc) return rc;
    } else {
        qm = om = am;                              // no rows: not used
    }
    static std::mutex mu;
    static uint64_t done_mask = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (!bit || !(done_mask & bit)) {
            if (cudaFuncSetAttribute(latent_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLaSmem) !=
                    cudaSuccess ||
                cudaFuncSetAttribute(latent_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLaMergeMost) !=
                    cudaSuccess)
                return PKV_ERR_CUDA;
            done_mask |= bit;
        }
    }
    if (launch_pdl(latent_attn_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kLaThreads), kLaSmem,
                   static_cast<cudaStream_t>(stream), am, bm, qm, om, p) != cudaSuccess)
        return PKV_ERR_CUDA;
    // All tiles can have many pieces only where they are few; and of few rows there is little to
    // bring in in bulk.  1000 keys, 128 heads (76 lanes), calls merged few / in bulk: 4 requests 18.1 /
    // 30.4 us, 8: 21.9 / 24.8, 16: 24.9 / 25.7, 19: 26.4 / 26.6, 24: 28.1 / 27.2, 48: 37.8 / 33.9, 76 and
    // more within 4%; 64 heads (152 lanes), 30: 27.5 / 28.0, 39: 29.8 / 29.3, 76: 38.7 / 35.4.  256 requests
    // of 16 rows 66.1 / 71.9, 32: 71.4 / 74.3, 33: 73.7 / 75.8, 40: 74.6 / 74.2, 48: 76.6 / 74.6, 64: 81.1 /
    // 75.8.
    const bool bulk = most > p.lanes / 4 && p.hpt * p.tpt > 32;
    const dim3 lanes(static_cast<unsigned>(ctas), bulk ? 4 : 16);
    if ((bulk ? launch_pdl(latent_merge_kernel, lanes, dim3(256), 2 * la_merge_bytes(p) + kLaMergeExtra,
                           static_cast<cudaStream_t>(stream), p, ctas)
              : launch_pdl(latent_merge_few_kernel, lanes, dim3(256), 0, static_cast<cudaStream_t>(stream), p, ctas)) !=
        cudaSuccess)
        return PKV_ERR_CUDA;
    return PKV_OK;
}
