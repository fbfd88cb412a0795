// How a decode kernel plans a small call by itself (decode.cu, int8_decode.cu), in place of the plan kernel.
#pragma once

#include "attn_internal.cuh"

namespace pkv {

// ---- the decode kernel's own plan ---------------------------------------------
//
// For a call that decode_self_plan_ok admits (every request a split row, a
// batch small enough that every warp takes at most two chunks) no plan kernel
// runs.  Every CTA plans the whole call in shared memory (the space its rings
// take later) with the plan kernel's decisions (request_valid, the automatic
// split size, split_geometry), lists chunks in request order, and takes its
// warps' chunks from that list.  The grid's last CTA takes no chunks: it
// writes what the combine and the caller read (header, status, split tokens),
// beside the other CTAs' work rather than before it.

// One chunk of a warp: request, split, page range, the request's splits and
// first partial row.
struct SelfChunk {
    int r, k, pb, npages, n_split, pbase;
};

struct SelfPlanShared {
    unsigned long long total_pages;
    int bad, fits;
    int4 warp_tot[kDecodeWarps];
    int4 tot;
};

// The plan of the call in `scr` (8 * num_seqs + 1 ints) and the chunks of
// this warp (round 0 and round 1 of the snake order); returns the number of
// items (chunks x kv heads), 0 when the metadata does not fit the workspace.
template <int NW>
__device__ int decode_self_plan(const AttnParams &p, int *scr, SelfPlanShared &sh, SelfChunk (&mine)[2]) {
    const int S = p.num_seqs, tid = threadIdx.x, nthr = NW * 32;
    const int lane = tid & 31, warp = tid >> 5;
    int *s_qsl = scr, *s_len = scr + S + 1, *s_cb = s_len + S, *s_nc = s_cb + S, *s_ps = s_nc + S;
    int *s_pg = s_ps + S, *s_pb = s_pg + S, *s_sb = s_pb + S;
    for (int r = tid; r <= S; r += nthr) s_qsl[r] = __ldg(p.qsl + r);
    for (int r = tid; r < S; r += nthr) s_len[r] = __ldg(p.seq_lens + r);
    if (tid == 0) {
        sh.total_pages = 0;
        sh.bad = 0;
    }
    __syncthreads();
    // total key pages (sets the automatic split size), and the metadata check
    unsigned long long pages = 0;
    int bad = tid == 0 && s_qsl[0] != 0;
    for (int r = tid; r < S; r += nthr) {
        const int q0 = s_qsl[r], q1 = s_qsl[r + 1], L = s_len[r];
        if (!request_valid(q0, q1, L, p.num_tokens, p.max_seq_len, p.max_query_len, p.max_blocks_per_seq)) bad = 1;
        else if (q1 > q0) pages += static_cast<unsigned long long>(div_up(L, kBlock));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) pages += __shfl_xor_sync(0xffffffffu, pages, o);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        if (pages) atomicAdd(&sh.total_pages, pages);
        if (bad) sh.bad = 1;
    }
    __syncthreads();
    const int pps = auto_pages_per_split(sh.total_pages, p.num_kv_heads, p.total_warps);
    // per request: chunks, pages per split, partial rows and split tokens; each
    // thread a contiguous range of requests, one block scan for the bases
    const int per_thr = div_up(S, nthr);
    const int r_begin = min(S, tid * per_thr), r_end = min(S, r_begin + per_thr);
    int4 cnt = make_int4(0, 0, 0, 0);
    for (int r = r_begin; r < r_end; ++r) {
        const int q0 = s_qsl[r], q1 = s_qsl[r + 1], L = s_len[r];
        const int q = q1 - q0;
        int n = 0, ps = 0, span = 0;
        if (q > 0 && request_valid(q0, q1, L, p.num_tokens, p.max_seq_len, p.max_query_len, p.max_blocks_per_seq)) {
            span = div_up(L, kBlock);
            const int2 sg = split_geometry(span, pps, 0, kMaxSplits);
            ps = sg.x;
            n = sg.y;
        }
        s_nc[r] = n;
        s_ps[r] = ps;
        s_pg[r] = span;
        cnt.x += n;
        if (n > 1) {
            cnt.y += q * p.num_q_heads * n;
            cnt.z += q;
        }
    }
    int4 inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, inc.x, o), b = __shfl_up_sync(0xffffffffu, inc.y, o);
        const int c = __shfl_up_sync(0xffffffffu, inc.z, o);
        if (lane >= o) {
            inc.x += a;
            inc.y += b;
            inc.z += c;
        }
    }
    if (lane == 31) sh.warp_tot[warp] = inc;
    __syncthreads();
    if (tid == 0) {
        int4 acc = make_int4(0, 0, 0, 0);
        for (int w = 0; w < NW; ++w) {
            const int4 t = sh.warp_tot[w];
            sh.warp_tot[w] = acc;
            acc.x += t.x;
            acc.y += t.y;
            acc.z += t.z;
        }
        sh.tot = acc;
        sh.fits = acc.x <= p.lay.max_chunks && acc.y <= p.lay.max_prow && acc.z <= p.num_tokens;
        if (!sh.fits) sh.bad = 1;
    }
    __syncthreads();
    {
        const int4 wb = sh.warp_tot[warp];
        int cb = wb.x + inc.x - cnt.x, pb = wb.y + inc.y - cnt.y, sb = wb.z + inc.z - cnt.z;
        for (int r = r_begin; r < r_end; ++r) {
            const int n = s_nc[r];
            s_cb[r] = cb;
            s_pb[r] = pb;
            s_sb[r] = sb;
            cb += n;
            if (n > 1) {
                const int q = s_qsl[r + 1] - s_qsl[r];
                pb += q * p.num_q_heads * n;
                sb += q;
            }
        }
    }
    __syncthreads();
    const int n_items = sh.fits ? sh.tot.x * p.num_kv_heads : 0;
    // this warp's chunks: items wid and 2 W - 1 - wid (the snake order of the
    // loop), W the warps of every CTA but the last
    const int W = (gridDim.x - 1) * NW, wid = blockIdx.x * NW + warp;
#pragma unroll
    for (int round = 0; round < 2; ++round) {
        const int item = round ? 2 * W - 1 - wid : wid;
        SelfChunk c{-1, 0, 0, 0, 1, 0};
        if (wid < W && item < n_items) {
            const int ch = item / p.num_kv_heads;
            // the request of chunk ch: the last with chunk base <= ch, past any
            // request without chunks
            int lo = 0, hi = S - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cb[mid] <= ch) lo = mid;
                else hi = mid - 1;
            }
            while (lo < S - 1 && s_nc[lo] == 0) ++lo;
            c.r = lo;
            c.k = ch - s_cb[lo];
            c.pb = c.k * s_ps[lo];
            c.npages = min(s_pg[lo], c.pb + s_ps[lo]) - c.pb;
            c.n_split = s_nc[lo] > 1 ? s_nc[lo] : 1;
            c.pbase = s_nc[lo] > 1 ? s_pb[lo] : 0;
        }
        mine[round] = c;
    }
    return n_items;
}

// The same plan made by one warp alone, in registers, for a batch of at most
// 32 x kWarpPlanPer requests: lane l holds requests [l per, (l + 1) per), the
// page total and the bases come from warp shuffles, and the owner of each of
// the warp's chunks is found by a ballot over the lanes' chunk ranges.  No
// block barrier and no shared memory: a chunk CTA's warps go from the
// metadata read to their first page loads on their own.  Decisions and
// bases are those of decode_self_plan (the grid's last CTA still makes that
// one, for the header and the split tokens).
constexpr int kWarpPlanPer = 2;

static __device__ int decode_warp_plan(const AttnParams &p, SelfChunk (&mine)[2], int W, int wid) {
    const int S = p.num_seqs, lane = threadIdx.x & 31;
    const int per = div_up(S, 32);
    const int r0 = min(S, lane * per), r1 = min(S, r0 + per);
    int q0a[kWarpPlanPer], qa[kWarpPlanPer], La[kWarpPlanPer];
#pragma unroll
    for (int i = 0; i < kWarpPlanPer; ++i) {
        const int r = r0 + i;
        const bool in = i < per && r < r1;
        q0a[i] = in ? __ldg(p.qsl + r) : 0;
        qa[i] = in ? __ldg(p.qsl + r + 1) : 0;       // q1 for now
        La[i] = in ? __ldg(p.seq_lens + r) : 0;
    }
    // total key pages of the valid requests (the automatic split size)
    unsigned long long pages = 0;
    bool valid[kWarpPlanPer];
#pragma unroll
    for (int i = 0; i < kWarpPlanPer; ++i) {
        const bool in = i < per && r0 + i < r1;
        valid[i] = in && request_valid(q0a[i], qa[i], La[i], p.num_tokens, p.max_seq_len, p.max_query_len,
                                       p.max_blocks_per_seq);
        qa[i] -= q0a[i];                                 // query tokens
        if (valid[i] && qa[i] > 0) pages += static_cast<unsigned long long>(div_up(La[i], kBlock));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) pages += __shfl_xor_sync(0xffffffffu, pages, o);
    const int pps = auto_pages_per_split(pages, p.num_kv_heads, p.total_warps);
    // per request: chunks, pages per split, page span; per lane: chunks,
    // partial rows, split tokens
    int na[kWarpPlanPer], psa[kWarpPlanPer], spa[kWarpPlanPer];
    int4 cnt = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kWarpPlanPer; ++i) {
        int n = 0, ps = 0, span = 0;
        if (valid[i] && qa[i] > 0) {
            span = div_up(La[i], kBlock);
            const int2 sg = split_geometry(span, pps, 0, kMaxSplits);
            ps = sg.x;
            n = sg.y;
        }
        na[i] = n;
        psa[i] = ps;
        spa[i] = span;
        cnt.x += n;
        if (n > 1) {
            cnt.y += qa[i] * p.num_q_heads * n;
            cnt.z += qa[i];
        }
    }
    int4 inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, inc.x, o), b = __shfl_up_sync(0xffffffffu, inc.y, o);
        const int c = __shfl_up_sync(0xffffffffu, inc.z, o);
        if (lane >= o) {
            inc.x += a;
            inc.y += b;
            inc.z += c;
        }
    }
    const int tot_x = __shfl_sync(0xffffffffu, inc.x, 31), tot_y = __shfl_sync(0xffffffffu, inc.y, 31);
    const int tot_z = __shfl_sync(0xffffffffu, inc.z, 31);
    const bool fits = tot_x <= p.lay.max_chunks && tot_y <= p.lay.max_prow && tot_z <= p.num_tokens;
    const int n_items = fits ? tot_x * p.num_kv_heads : 0;
    const int cb0 = inc.x - cnt.x, pb0 = inc.y - cnt.y;      // this lane's first chunk and partial row
#pragma unroll
    for (int round = 0; round < 2; ++round) {
        const int item = round ? 2 * W - 1 - wid : wid;
        SelfChunk c{-1, 0, 0, 0, 1, 0};
        if (wid < W && item < n_items) {                     // uniform over the warp
            const int ch = item / p.num_kv_heads;
            const unsigned owners = __ballot_sync(0xffffffffu, cb0 <= ch && ch < cb0 + cnt.x);
            const int owner = __ffs(owners) - 1;
            int cb = cb0, pb = pb0;
            bool done = false;
#pragma unroll
            for (int i = 0; i < kWarpPlanPer; ++i) {
                if (!done && ch < cb + na[i]) {
                    done = true;
                    c.r = r0 + i;
                    c.k = ch - cb;
                    c.pb = c.k * psa[i];
                    c.npages = min(spa[i], c.pb + psa[i]) - c.pb;
                    c.n_split = na[i] > 1 ? na[i] : 1;
                    c.pbase = na[i] > 1 ? pb : 0;
                }
                cb += na[i];
                if (na[i] > 1) pb += qa[i] * p.num_q_heads * na[i];
            }
            c.r = __shfl_sync(0xffffffffu, c.r, owner);
            c.k = __shfl_sync(0xffffffffu, c.k, owner);
            c.pb = __shfl_sync(0xffffffffu, c.pb, owner);
            c.npages = __shfl_sync(0xffffffffu, c.npages, owner);
            c.n_split = __shfl_sync(0xffffffffu, c.n_split, owner);
            c.pbase = __shfl_sync(0xffffffffu, c.pbase, owner);
        }
        mine[round] = c;
    }
    return n_items;
}

// The last CTA of a self-planned call: the header, status and split tokens
// the plan kernel would have written (after every earlier kernel on the
// stream is complete), then the header's epoch is bumped.  (The request table
// is the plan kernel's record for its own decode launches; a self-planned
// call does not read it.)
template <int NW>
__device__ void decode_self_plan_publish(const AttnParams &p, const int *scr, const SelfPlanShared &sh) {
    const int S = p.num_seqs, tid = threadIdx.x, nthr = NW * 32;
    const int *s_qsl = scr, *s_len = scr + S + 1, *s_cb = s_len + S, *s_nc = s_cb + S;
    const int *s_pb = s_nc + 2 * S + S, *s_sb = s_pb + S;
    WsHeader *hdr = reinterpret_cast<WsHeader *>(p.ws);
    int4 *stoks = reinterpret_cast<int4 *>(p.ws + p.lay.off_stoks);
    const bool fits = sh.fits != 0;
    for (int i = tid; i < 2 * kStatsCtas; i += nthr) reinterpret_cast<int32_t *>(p.ws + kStatsOffset)[i] = 0;
    (void)s_len;
    (void)s_cb;
    for (int r = tid; r < S; r += nthr) {
        const int n = fits ? s_nc[r] : 0;
        const int q0 = s_qsl[r];
        const int q = s_qsl[r + 1] - q0;
        if (n > 1)
            for (int i = 0; i < q; ++i)
                stoks[s_sb[r] + i] = make_int4(q0 + i, s_pb[r] + i * p.num_q_heads * n, n, 0);
    }
    if (tid == 0) {
        hdr->status = sh.bad ? PKV_ERR_DEVICE_METADATA : PKV_OK;
        hdr->magic = kMagic;
        hdr->n_chunks = fits ? sh.tot.x : 0;
        hdr->num_tokens = p.num_tokens;
        hdr->num_q_heads = p.num_q_heads;
        hdr->head_size = p.head_size;
        hdr->num_seqs = S;
        hdr->pages_per_split = auto_pages_per_split(sh.total_pages, p.num_kv_heads, p.total_warps);
        hdr->n_ptiles = 0;
        hdr->n_crows = 0;
        hdr->prefix_blocks = 0;
        hdr->prefix_parts = 0;
        hdr->next_ptile_item = 0;
        hdr->next_prefix_item = 0;
        hdr->n_split_tokens = fits ? sh.tot.z : 0;
        hdr->split_items = 0;
        hdr->off_req = p.lay.off_req;
        hdr->off_stoks = p.lay.off_stoks;
        hdr->off_chunks = p.lay.off_chunks;
        hdr->off_ptiles = p.lay.off_ptiles;
        hdr->off_crows = p.lay.off_crows;
        hdr->off_part_lse = p.lay.off_part_lse;
        hdr->off_part_o = p.lay.off_part_o;
        hdr->max_chunks = p.lay.max_chunks;
        hdr->max_ptiles = p.lay.max_ptiles;
        hdr->max_crows = p.lay.max_crows;
        hdr->max_prow = p.lay.max_prow;
        hdr->prow_used = sh.tot.y;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) atomicAdd(&hdr->epoch, 1);
}

}  // namespace pkv
