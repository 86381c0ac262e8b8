// Page bookkeeping of a paged KV cache ("Multi-Token Prediction &
// Draft-Model-Free Speculative Decoding", section "Production Deployment
// Guidelines": the cache is held in non-contiguous physical blocks): block
// tables and slot maps from request lengths, and the append of new K/V rows
// to their slots.
#include <cooperative_groups.h>

#include "kernels.h"

namespace medusa {

namespace {

constexpr int kPlanThreads = 1024;

// inclusive scan of one value per thread over the block; `total` gets the
// block's sum.  s_warp: 33 entries of shared memory.
__device__ long block_scan(long x, long* s_warp, long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's readers are done
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(kFull, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    total = s_warp[31];
    return x + (warp > 0 ? s_warp[warp - 1] : 0);
}

// The whole plan in one launch of one thread-block cluster (a single CTA for
// few tokens).  Every CTA scans the B lengths for itself (row starts, released
// pages, grown pages: three prefix sums in shared memory), so slots need no
// table entry that this launch writes: a token's page is an old table entry,
// or an entry of the free stack, or a page released in this call.  The
// cluster barrier separates the last read of the state (owned, free_count,
// which the outputs may alias) from its first write.  Latency-bound: two
// launches (a one-CTA plan, then a grid of slots) would cost a second launch
// and a table round trip through memory.  64 sequences decoding: 6.4 us, 300 with
// up to 700 new tokens each: 9.5 us.
__global__ void __launch_bounds__(kPlanThreads) kv_page_plan_kernel(const PagePlanArgs a) {
    extern __shared__ int s_dyn[];
    int* s_row = s_dyn;             // [B + 1] first packed row of each sequence
    int* s_owned = s_row + a.B + 1;  // [B] pages owned before the call
    int* s_off = s_owned + a.B;     // [B] first growth unit; -1: not served (refused or released)
    int* s_rel = s_off + a.B;       // [B + 1] first released page
    __shared__ long s_warp[32];
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    int bad = 0;
    int fc = a.free_count[0];
    if (fc < 0 || fc > a.num_pages) {
        bad |= MEDUSA_STATUS_BAD_LENGTH;
        fc = fc < 0 ? 0 : a.num_pages;
    }
    auto new_rows = [&](int b) {  // -1: ended; what is below that counts as no new row
        const int n = a.new_len[b];
        return n < -1 ? 0 : n;
    };
    // pass 1: rows and released pages
    long rows0 = 0, rel0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long rows = 0, rel = 0;
        if (b < a.B) {
            const int n = new_rows(b);
            int own = a.owned[b];
            if (a.new_len[b] < -1) bad |= MEDUSA_STATUS_BAD_LENGTH;
            if (own < 0 || own > a.max_pages) {
                bad |= MEDUSA_STATUS_BAD_LENGTH;
                own = own < 0 ? 0 : a.max_pages;
            }
            s_owned[b] = own;
            rows = n > 0 ? n : 0;
            rel = n < 0 ? own : 0;
        }
        long t_rows, t_rel;
        const long i_rows = block_scan(rows, s_warp, t_rows);
        const long i_rel = block_scan(rel, s_warp, t_rel);
        if (b < a.B) {
            s_row[b] = (int)min(rows0 + i_rows - rows, (long)a.max_tokens);
            s_rel[b] = (int)min(rel0 + i_rel - rel, (long)a.num_pages);
        }
        rows0 += t_rows;
        rel0 += t_rel;
    }
    if (rows0 > a.max_tokens) bad |= MEDUSA_STATUS_BAD_LENGTH;
    // the stack cannot hold more than every page: an owned page counted twice
    if (rel0 > a.num_pages - fc) bad |= MEDUSA_STATUS_BAD_PAGE;
    const int nrel = (int)min(rel0, (long)(a.num_pages - fc));
    const int avail = fc + nrel;
    if (tid == 0) {
        s_row[a.B] = (int)min(rows0, (long)a.max_tokens);
        s_rel[a.B] = (int)min(rel0, (long)a.num_pages);
    }
    // pass 2: growth, in sequence order; a sequence is served when the pages
    // up to and including its own fit
    long grow0 = 0, used = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long grow = 0;
        bool fits = false;
        if (b < a.B) {
            const int n = new_rows(b), p = a.prefix_len[b];
            if (n >= 0 && p < 0) bad |= MEDUSA_STATUS_BAD_PREFIX;
            if (n >= 0 && p >= 0) {
                const long want = ((long)p + n + a.room + a.page_size - 1) / a.page_size;
                fits = want <= a.max_pages;
                if (fits && want > s_owned[b]) grow = want - s_owned[b];
                if (!fits) bad |= MEDUSA_STATUS_CACHE_OVERFLOW;
            }
        }
        long t_grow, t_used;
        const long i_grow = block_scan(grow, s_warp, t_grow) + grow0;
        const bool served = fits && (grow == 0 || i_grow <= avail);
        if (fits && !served) bad |= MEDUSA_STATUS_CACHE_OVERFLOW;
        (void)block_scan(served ? grow : 0, s_warp, t_used);
        // (what refused sequences before it would have taken may pass 32 bits; a
        // sequence served behind them takes nothing)
        if (b < a.B) s_off[b] = served ? (int)min(i_grow - grow, 0x7fffffffL) : -1;
        grow0 += t_grow;
        used += t_used;
    }
    cl.sync();  // every CTA has read owned and free_count; s_* of this CTA complete
    // entry i of the free stack as it is after the releases
    auto stack_page = [&](int i) -> int {
        if (i < fc) return a.free_list[i];
        const int r = i - fc;  // released page r: of the last sequence whose first one is <= r
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_rel[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        return a.block_table[(long)lo * a.max_pages + (r - s_rel[lo])];
    };
    auto valid = [&](int page) { return page >= 0 && page < a.num_pages; };
    // table entries, pushed pages and per-sequence outputs: a warp per sequence
    for (int b = rank + C * warp; b < a.B; b += C * (kPlanThreads / 32)) {
        const int own = s_owned[b], off = s_off[b], n = new_rows(b);
        if (n == -1) {
            for (int i = lane; i < own; i += 32) {
                const int page = a.block_table[(long)b * a.max_pages + i];
                if (!valid(page)) bad |= MEDUSA_STATUS_BAD_PAGE;
                if (s_rel[b] + i < nrel) a.free_list[fc + s_rel[b] + i] = page;
            }
        } else if (off >= 0) {
            const int want = (int)(((long)a.prefix_len[b] + n + a.room + a.page_size - 1) / a.page_size);
            for (int i = own + lane; i < want; i += 32) {
                int page = stack_page(avail - 1 - (off + i - own));
                if (!valid(page)) {
                    bad |= MEDUSA_STATUS_BAD_PAGE;
                    page = -1;
                }
                a.block_table[(long)b * a.max_pages + i] = page;
            }
            if (lane == 0) a.owned_out[b] = want > own ? want : own;
        }
        if (lane == 0) {
            a.row_start[b] = s_row[b];
            if (n == -1) a.owned_out[b] = 0;
            else if (off < 0) a.owned_out[b] = own;
        }
    }
    if (rank == 0 && tid == 0) {
        a.row_start[a.B] = s_row[a.B];
        a.free_count_out[0] = avail - (int)used;
    }
    // slots of the packed new rows
    const int total = s_row[a.B];
    for (int t = rank * kPlanThreads + tid; t < a.max_tokens; t += C * kPlanThreads) {
        long slot = -1;
        if (t < total) {
            int lo = 0, hi = a.B - 1;  // the last sequence whose first row is <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_row[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int off = s_off[lo];
            if (off >= 0) {
                const long pos = (long)a.prefix_len[lo] + (t - s_row[lo]);
                const int blk = (int)(pos / a.page_size), own = s_owned[lo];
                const int page = blk < own ? a.block_table[(long)lo * a.max_pages + blk]
                                           : stack_page(avail - 1 - (off + blk - own));
                if (valid(page)) slot = (long)page * a.page_size + pos % a.page_size;
                else bad |= MEDUSA_STATUS_BAD_PAGE;
            }
        }
        a.slot_map[t] = slot;
    }
    if (bad) set_status(a.status, bad);
}

// Rows to slots: a block takes 256 / vecs (token, head) rows at a time, a
// thread one 16-byte piece of K and of V of each, kRowsAhead rows in flight
// before their stores.  A thread's piece is fixed, so the only divisions are
// one by Hkv and one by page_size per row, in 32 bits (a row has 128 bytes at
// least: 2^31 rows or 2^32 slots are more than a GPU holds, and the entry point
// refuses them).  Bound by memory, every byte read once and written once: 32768
// tokens of 8 heads of 128 (268.7 MB) in 42.7 us, 6294 GB/s; 48.5 us with 64-bit
// divisions per piece.
constexpr int kRowsAhead = 4;
template <int kVecs>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a) {
    constexpr int kRows = 256 / kVecs;
    const uint8_t* k = (const uint8_t*)a.k;
    const uint8_t* v = (const uint8_t*)a.v;
    uint8_t* kp = (uint8_t*)a.k_pages;
    uint8_t* vp = (uint8_t*)a.v_pages;
    const long n_slots = (long)a.num_pages * a.page_size, total = (long)a.N * a.Hkv;
    const int c = threadIdx.x % kVecs;
    int bad = 0;
    const long r0 = (long)blockIdx.x * (kRows * kRowsAhead) + threadIdx.x / kVecs;
    uint4 kr[kRowsAhead], vr[kRowsAhead];
    long dst[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
        const long r = r0 + j * kRows;
        dst[j] = -1;
        if (r >= total) continue;
        const uint32_t t = (uint32_t)r / (uint32_t)a.Hkv, g = (uint32_t)r - t * (uint32_t)a.Hkv;
        const long slot = a.slot_map[t];
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1) bad = MEDUSA_STATUS_BAD_PAGE;
            continue;
        }
        const uint32_t page = (uint32_t)slot / (uint32_t)a.page_size;
        const uint32_t off = (uint32_t)slot - page * (uint32_t)a.page_size;
        dst[j] = (((long)page * a.Hkv + (long)g) * a.page_size + (long)off) * (kVecs * 16) + c * 16;
        const long src = (long)g * (kVecs * 16) + c * 16;
        kr[j] = ld_nc(k + (long)t * a.k_stride + src);
        vr[j] = ld_nc(v + (long)t * a.v_stride + src);
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j)
        if (dst[j] >= 0) {
            *reinterpret_cast<uint4*>(kp + dst[j]) = kr[j];
            *reinterpret_cast<uint4*>(vp + dst[j]) = vr[j];
        }
    if (bad) set_status(a.status, bad);
}

template <int kVecs>
void append_launch(const KvAppendArgs& a, cudaStream_t st) {
    const long total = (long)a.N * a.Hkv, per = 256 / kVecs * kRowsAhead;
    const long blocks = (total + per - 1) / per;
    kv_append_kernel<kVecs><<<(unsigned)blocks, 256, 0, st>>>(a);
}

}  // namespace

size_t page_plan_smem(int B) { return (size_t)(4 * B + 2) * sizeof(int); }

cudaError_t page_plan_launch(const PagePlanArgs& a, cudaStream_t st) {
    int ctas = (a.max_tokens + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
    ctas = ctas < 1 ? 1 : ctas > 8 ? 8 : ctas;
    cudaError_t e = cudaFuncSetAttribute(kv_page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)page_plan_smem(kMaxPlanSeqs));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = page_plan_smem(a.B);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_page_plan_kernel, a);
}

cudaError_t kv_append_launch(const KvAppendArgs& a, cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    switch (a.D * a.esize / 16) {  // 16-byte pieces of a head's row
        case 8: append_launch<8>(a, st); break;    // 64 bf16
        case 16: append_launch<16>(a, st); break;  // 128 bf16, 64 fp32
        default: append_launch<32>(a, st); break;  // 128 fp32
    }
    return cudaGetLastError();
}

}  // namespace medusa
