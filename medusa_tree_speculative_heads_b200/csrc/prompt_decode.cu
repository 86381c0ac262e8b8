// Attention of a few new tokens per sequence over a paged cache (bf16,
// head_dim 64/128, at most 16 query rows per (sequence, kv-head): plain
// decoding, short verification chunks).
//
// Such a call reads every K/V byte of the prefixes once for a handful of
// rows, so it is bound by HBM and by how evenly the bytes are spread over the
// SMs, not by arithmetic: a 128-row tcgen05 tile would be almost empty, and
// mma.sync m16n8k16 keeps up with a share of HBM many times over.  The work
// is laid out flat: the 64-key chunks of all (sequence, kv-head) pairs, end to
// end, are cut into equal runs, one per CTA (two CTAs per SM), whatever the
// lengths are; a pair counts kPairCost chunks more than it has, for its start
// and end.  A CTA's run covers the end of one pair, whole pairs, and the
// beginning of another; whole pairs are written out directly, the others as
// normalised fp32 partials that a second launch merges in run order.
// Warp 0 of a CTA streams the run by TMA: the rows of Q of each pair into two
// slots, K and V into a ring that runs on across pairs.  Warps 1-4 take 16
// keys of a chunk each for S = Q K^T, agree on the rows' running maximum
// through shared memory, put P there (bf16: 2^-8 relative, as the operands
// are; the fp32 sums l take it unrounded), and take a quarter of the output
// columns each for O += P V; O stays in registers and is complete at the end
// of a pair.  One sequence of 131072 tokens, 8 kv-heads of 128 (537 MB): 91 us,
// 5.9 TB/s (tcgen05 tiles with split keys: 143 us); 8 sequences of up to 8192
// tokens (84 MB): 23 to 25 us, of which some 10 us are two launches, the walk to a
// CTA's first pair and the merge.
#include "prompt_common.cuh"
#include "tc.cuh"
#include "tma.h"

namespace medusa {

namespace {

constexpr int kDR = 16;                      // query rows of a pair (mma M)
constexpr int kDC = 64;                      // keys per chunk
constexpr int kDW = 4;                       // consumer warps
constexpr int kDThreads = 32 * (1 + kDW);
constexpr int kDCtasPerSm = 2;
constexpr int kPairCost = 2;                 // what a pair's start and end cost, in chunks
constexpr int kPStride = kDC * 2 + 16;       // bytes of a row of P (ldmatrix rows on distinct banks)
template <int D> constexpr int d_stages() { return D == 128 ? 3 : 6; }

struct DecodeArgs {
    CUtensorMap mq;      // q as (D, Hq, N), box (64, G, 16 / G)
    CUtensorMap mk, mv;  // the pools as (D, page_size, num_pages * Hkv), box (64, page_rows, 1)
    PromptArgs p;
    float* part_o;       // [2 * grid][kDR][D]
    float* part_lse2;    // [2 * grid][kDR]
    int G, page_rows;
    float scale_log2;
    uint64_t wait_ns;
};

__device__ __forceinline__ int decode_chunks(const PromptSeq& s) { return s.n > 0 ? (s.p + s.n + kDC - 1) / kDC : 0; }
// units of one kv-head of a sequence
__device__ __forceinline__ int decode_units(const PromptSeq& s) { return s.n > 0 ? decode_chunks(s) + kPairCost : 0; }

// units of the sequences before b, and of all; one warp
__device__ inline long units_before(const PromptArgs& p, int b, long* total) {
    const int lane = threadIdx.x & 31;
    long before = 0, all = 0;
    for (int i = lane; i < p.B; i += 32) {
        const long c = (long)decode_units(prompt_seq(p, i)) * p.Hkv;
        all += c;
        if (i < b) before += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(kFull, before, o);
        all += __shfl_xor_sync(kFull, all, o);
    }
    *total = all;
    return before;
}
// run i of n: units [total * i / n, total * (i + 1) / n), none of them empty
__device__ __forceinline__ int runs_used(long total, int n) { return total < n ? (int)total : n; }
__device__ __forceinline__ long run_start(long total, int i, int n) { return total * i / n; }
// the run that holds unit u
__device__ __forceinline__ int run_of(long total, long u, int n) {
    int i = (int)(u * n / total);
    while (run_start(total, i + 1, n) <= u) ++i;
    while (run_start(total, i, n) > u) --i;
    return i;
}

// A warp's walk over the pairs of its CTA's run.  The lengths of 32 sequences
// at a time are kept one per lane.
struct DecodeWalk {
    const PromptArgs& p;
    long u, u1;          // the current segment's first unit, the run's end
    int b, g, nch, taken;
    int c_lo, c_hi;      // the segment's chunks
    int r0, n, pos;      // the sequence
    int block;
    PromptSeq mine;

    __device__ DecodeWalk(const PromptArgs& args) : p(args), block(-1) {}
    __device__ void load() {
        if (b >> 5 != block) {
            block = b >> 5;
            const int i = block * 32 + (threadIdx.x & 31);
            mine.r0 = mine.n = mine.p = 0;
            if (i < p.B) mine = prompt_seq(p, i);
        }
        r0 = __shfl_sync(kFull, mine.r0, b & 31);
        n = __shfl_sync(kFull, mine.n, b & 31);
        pos = __shfl_sync(kFull, mine.p, b & 31);
        nch = n > 0 ? (pos + n + kDC - 1) / kDC : 0;
    }
    __device__ void segment(int off) {  // of the pair, from its unit `off` on
        taken = (int)min((long)(nch + kPairCost - off), u1 - u);
        c_lo = max(0, off - kPairCost);
        c_hi = max(0, off + taken - kPairCost);
    }
    // unit u lies in sequence b0, whose first unit is `base`
    __device__ bool start(long first, long end, int b0, long base) {
        u = first;
        u1 = end;
        b = b0;
        load();
        const int off = (int)(u - base);
        g = off / (nch + kPairCost);
        segment(off % (nch + kPairCost));
        return c_lo < c_hi || next();
    }
    __device__ bool next() {
        do {
            u += taken;
            if (u >= u1) return false;
            if (++g == p.Hkv) {
                g = 0;
                do {
                    ++b;
                    load();
                } while (nch == 0);
            }
            segment(0);
        } while (c_lo == c_hi);
        return true;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// barrier of the consumer warps
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kDW * 32) : "memory"); }

template <int D>
struct DecodeSmem {
    static constexpr int kSub = kDC * 128;          // [64 keys x 64 elements]
    static constexpr int kKV = (D / 64) * kSub;     // a chunk of K (or of V)
    static constexpr int kQ = (D / 64) * kDR * 128; // the rows of a pair
    uint8_t ring[d_stages<D>()][2][kKV];
    uint8_t q[2][kQ];
    uint8_t p[kDR * kPStride];
    uint64_t full[d_stages<D>()], empty[d_stages<D>()], q_full[2], q_empty[2];
    float mx[kDW][kDR], l[kDW][kDR];
    long unit[2];
    int found, dirty[2];
};

template <int D>
__global__ void __launch_bounds__(kDThreads, kDCtasPerSm) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using Smem = DecodeSmem<D>;
    constexpr int NSUB = D / 64, ST = d_stages<D>(), kSub = Smem::kSub;
    constexpr int NT = D / 8 / kDW;       // 8-column output tiles of a warp
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);

    const PromptArgs& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_addr(smem_raw) & 1023u) {  // never expected (uniform over the grid)
        if (threadIdx.x == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
        return;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        // the run and the sequence that holds its first unit
        long total;
        (void)units_before(p, 0, &total);
        const int n = runs_used(total, gridDim.x);
        const long u0 = (int)blockIdx.x < n ? run_start(total, blockIdx.x, n) : total;
        long base = 0;
        int found = -1;
        for (int b0 = 0; b0 < p.B && found < 0; b0 += 32) {
            long c = b0 + lane < p.B ? (long)decode_units(prompt_seq(p, b0 + lane)) * p.Hkv : 0;
            long inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long y = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(kFull, base + inc > u0);
            if (hit) {
                const int src = __ffs(hit) - 1;
                found = b0 + src;
                base += __shfl_sync(kFull, inc - c, src);
            } else {
                base += __shfl_sync(kFull, inc, 31);
            }
        }
        if (lane == 0) {
            sm.found = found;
            sm.unit[0] = base;   // first unit of that sequence
            sm.unit[1] = total;
            sm.dirty[0] = sm.dirty[1] = 0;
        }
        if (blockIdx.x == 0)
            for (int b = lane; b < p.B; b += 32)
                if (const int bad = prompt_seq(p, b).bad) set_status(p.status, bad);
    } else if (threadIdx.x == 32) {
        tma_prefetch_desc(&a.mq);
        tma_prefetch_desc(&a.mk);
        tma_prefetch_desc(&a.mv);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kDW);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.q_empty[s], kDW);
        }
        mbar_fence_init();
    }
    __syncthreads();
    const long total = sm.unit[1];
    const int n_runs = runs_used(total, gridDim.x);
    if ((int)blockIdx.x >= n_runs) return;
    DecodeWalk walk(p);
    bool more = walk.start(run_start(total, blockIdx.x, n_runs), run_start(total, blockIdx.x + 1, n_runs), sm.found,
                           sm.unit[0]);
    const int G = a.G;
    int it = 0, seg = 0;  // chunk and pair of the run
    bool ok = true;
    if (warp == 0) {
        // ---------------- producer ----------------
        // A lane looks up a box of page_rows keys; the boxes of the chunk after the
        // one being issued are looked up meanwhile, across pairs too.  The warp
        // runs converged and one elected lane issues (a copy per lane goes through
        // the lanes one after the other, some 100 cycles each).
        const int pr = a.page_rows, nbox = kDC / pr;
        const bool lead = elect_one();
        int c = more ? walk.c_lo : 0;
        auto look_up = [&](int& y, int& z) {  // (row in the page, page * Hkv + kv-head), z < 0: not loaded
            const int pos = c * kDC + lane * pr;
            y = 0;
            z = -1;
            if (lane >= nbox || pos >= walk.pos + walk.n) return;
            const int page = p.block_table[(long)walk.b * p.max_pages + pos / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                set_status(p.status, MEDUSA_STATUS_BAD_PAGE);
                return;
            }
            y = pos % p.page_size;
            z = page * p.Hkv + walk.g;
        };
        int y = 0, z = -1, qrow = 0, qhead = 0;
        bool first = true;  // the chunk is its pair's first in this run
        // A slot may be filled again when its readers are done and its last copy has
        // landed.  The one implies the other, unless a wait expired and they passed
        // the slot over: its barrier then must not be armed for a second copy.
        auto free_slot = [&](uint64_t* empty, uint64_t* full, int parity) {
            return __all_sync(kFull, mbar_wait(empty, parity, a.wait_ns)) &&
                   __all_sync(kFull, mbar_wait(full, parity, a.wait_ns));
        };
        if (more) look_up(y, z);
        while (more && ok) {
            const int s = it % ST, cy = y, cz = z;
            const bool cfirst = first;
            qrow = walk.r0;
            qhead = walk.g * G;
            first = false;
            if (++c >= walk.c_hi) {
                more = walk.next();
                c = walk.c_lo;
                first = true;
            }
            if (more) look_up(y, z);
            if (cfirst) {
                const int qs = seg & 1;
                if (seg >= 2 && !free_slot(&sm.q_empty[qs], &sm.q_full[qs], ((seg >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (lead) {
                    mbar_arrive_expect_tx(&sm.q_full[qs], (uint32_t)(kDR / G * G * 128 * NSUB));
#pragma unroll
                    for (int x = 0; x < NSUB; ++x)
                        tma_load_3d(sm.q[qs] + x * kDR * 128, &a.mq, x * 64, qhead, qrow, &sm.q_full[qs]);
                }
                __syncwarp();
                ++seg;
            }
            const unsigned loads = __ballot_sync(kFull, cz >= 0);
            if (it >= ST && !free_slot(&sm.empty[s], &sm.full[s], ((it / ST) - 1) & 1)) {
                ok = false;
                break;
            }
            if (lead) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(__popc(loads) * 2 * NSUB * pr * 128));
            for (int x = 0; x < nbox; ++x) {
                const int by = __shfl_sync(kFull, cy, x), bz = __shfl_sync(kFull, cz, x);
                if (bz < 0) continue;
                if (lead) {
#pragma unroll
                    for (int u = 0; u < 2 * NSUB; ++u)
                        tma_load_3d(sm.ring[s][u / NSUB] + (u % NSUB) * kSub + x * pr * 128, u < NSUB ? &a.mk : &a.mv,
                                    (u % NSUB) * 64, by, bz, &sm.full[s]);
                }
                __syncwarp();
            }
            ++it;
        }
        if (!ok && lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
        // drain: no copy may still be landing when the CTA exits
        for (int i = max(0, it - ST); i < it; ++i) mbar_wait(&sm.full[i % ST], (i / ST) & 1);
        for (int i = max(0, seg - 2); i < seg; ++i) mbar_wait(&sm.q_full[i & 1], (i >> 1) & 1);
        return;
    }
    // ---------------- consumers ----------------
    const int w = warp - 1, r0 = lane >> 2, r1 = r0 + 8, cc = lane & 3;
    // ldmatrix rows of this lane: matrix lane / 8, row lane % 8
    const int mi = lane >> 3, mr = lane & 7;
    const int a_row = (mi & 1) * 8 + mr, a_ch = mi >> 1;           // A (Q, P): row, 16-byte column
    const int k_key = w * 16 + (mi >> 1) * 8 + mr, k_ch = mi & 1;  // K: key, 16-byte column
    const int v_key = (mi & 1) * 8 + mr, v_ch = w * NT + (mi >> 1);  // V: key of a 16-key step, 16-byte column
    const uint32_t sp = smem_addr(sm.p);
    for (; more; more = walk.next(), ++seg) {
        const int rows = walk.n * G, keys = walk.pos + walk.n;
        const int p0 = r0 < rows ? walk.pos + r0 / G : -1, p1 = r1 < rows ? walk.pos + r1 / G : -1;  // positions
        uint32_t q[D / 16][4];
        {
            if (ok) ok = __all_sync(kFull, mbar_wait(&sm.q_full[seg & 1], (seg >> 1) & 1, a.wait_ns));
            const uint32_t sq = smem_addr(sm.q[seg & 1]);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int ch = 2 * ks + a_ch;
                ldsm4(sq + (ch >> 3) * kDR * 128 + a_row * 128 + (((ch & 7) ^ mr) << 4), q[ks]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_empty[seg & 1]);
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // l: of this warp's keys
        for (int c = walk.c_lo; c < walk.c_hi; ++c, ++it) {
            const int s = it % ST;
            // (after an expired wait the chunks are passed over, barriers and all)
            if (ok) ok = __all_sync(kFull, mbar_wait(&sm.full[s], (it / ST) & 1, a.wait_ns));
            const uint32_t sk = smem_addr(sm.ring[s][0]), sv = smem_addr(sm.ring[s][1]);
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t kb[4];
                const int ch = 2 * ks + k_ch;
                ldsm4(sk + (ch >> 3) * kSub + k_key * 128 + (((ch & 7) ^ mr) << 4), kb);
                mma16816(sc[0], q[ks], kb[0], kb[1]);
                mma16816(sc[1], q[ks], kb[2], kb[3]);
            }
            const int key0 = c * kDC + w * 16;
            // columns of the lane: keys key0 + 8 n + 2 cc + {0, 1}
            float mx[2] = {-INFINITY, -INFINITY};
            const bool part = c * kDC + kDC > walk.pos + 1;  // some row does not see some of the chunk's keys
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 8 * n + 2 * cc + (e & 1);
                    if (part && key > (e < 2 ? p0 : p1)) sc[n][e] = -INFINITY;
                    mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
                if (cc == 0) sm.mx[w][h ? r1 : r0] = mx[h];
            }
            consumers_sync();  // the warps' maxima are there, P and V of the last chunk are read
            if (w == 0 && lane == 0) sm.dirty[(it + 1) & 1] = 0;
            float al[2];
            bool raised = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h ? r1 : r0;
                const float top =
                    fmaxf(fmaxf(sm.mx[0][r], sm.mx[1][r]), fmaxf(sm.mx[2][r], sm.mx[3][r])) * a.scale_log2;
                al[h] = 1.f;
                if (top > m[h] + 8.f) {  // a new reference only when the maximum rises by more than 2^8
                    al[h] = exp2_sfu(m[h] - top);
                    m[h] = top;
                    raised = true;
                }
            }
            const float mu0 = m[0] == -INFINITY ? 0.f : m[0], mu1 = m[1] == -INFINITY ? 0.f : m[1];
            float rs[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float pv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pv[e] = exp2_sfu(fmaf(sc[n][e], a.scale_log2, e < 2 ? -mu0 : -mu1));
                    rs[e >> 1] += pv[e];
                }
                const int col = (w * 16 + 8 * n + 2 * cc) * 2;
                *reinterpret_cast<uint32_t*>(sm.p + r0 * kPStride + col) = pack_bf16(pv[0], pv[1]);
                *reinterpret_cast<uint32_t*>(sm.p + r1 * kPStride + col) = pack_bf16(pv[2], pv[3]);
            }
            l[0] = l[0] * al[0] + rs[0];
            l[1] = l[1] * al[1] + rs[1];
            if (__any_sync(kFull, raised)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= al[0];
                    o[n][1] *= al[0];
                    o[n][2] *= al[1];
                    o[n][3] *= al[1];
                }
            }
            if (part) {
                // V rows that some row does not see: what is not finite is cleared (0 * NaN must
                // not reach such a row), and added below to the rows that see it
                uint8_t* vt = sm.ring[s][1] + w * 16 * 128;
                bool dirty = false;
#pragma unroll
                for (int e = lane; e < 16 * NSUB * 8; e += 32) {
                    const int row = e / (NSUB * 8), x = e % (NSUB * 8);
                    uint4* at = reinterpret_cast<uint4*>(vt + (x >> 3) * kSub + row * 128 + (x & 7) * 16);
                    const uint4 v = *at;
                    const uint32_t b0 = nonfinite2(v.x), b1 = nonfinite2(v.y);
                    const uint32_t b2 = nonfinite2(v.z), b3 = nonfinite2(v.w);
                    if (key0 + row >= keys) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (b0 | b1 | b2 | b3) {
                        *at = make_uint4(clear2(v.x, b0), clear2(v.y, b1), clear2(v.z, b2), clear2(v.w, b3));
                        dirty = true;
                    }
                }
                if (dirty) sm.dirty[it & 1] = 1;
                fence_proxy_async_shared();  // the slot's next copy comes after these writes
            }
            consumers_sync();  // P (and a cleared V) is there
#pragma unroll
            for (int ks = 0; ks < kDC / 16; ++ks) {
                uint32_t pa[4];
                ldsm4(sp + a_row * kPStride + (2 * ks + a_ch) * 16, pa);
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t vb[4];
                    const int ch = v_ch + n;
                    ldsm4_t(sv + (ch >> 3) * kSub + (ks * 16 + v_key) * 128 + (((ch & 7) ^ mr) << 4), vb);
                    mma16816(o[n], pa, vb[0], vb[1]);
                    mma16816(o[n + 1], pa, vb[2], vb[3]);
                }
            }
            if (part && *reinterpret_cast<volatile int*>(&sm.dirty[it & 1])) {
                const int end = min(keys, c * kDC + kDC);
                for (int key = c * kDC; key < end; ++key) {
                    const int page = p.block_table[(long)walk.b * p.max_pages + key / p.page_size];
                    if (page < 0 || page >= p.num_pages) continue;
                    const __nv_bfloat16* vr = (const __nv_bfloat16*)p.v +
                                              (((long)page * p.Hkv + walk.g) * p.page_size + key % p.page_size) * D;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t v2 = *reinterpret_cast<const uint32_t*>(vr + (w * NT + n) * 8 + 2 * cc);
                        const float f0 = bf16lo(v2), f1 = bf16hi(v2);
                        if (!isfinite(f0) && key <= p0) o[n][0] += f0;
                        if (!isfinite(f1) && key <= p0) o[n][1] += f1;
                        if (!isfinite(f0) && key <= p1) o[n][2] += f0;
                        if (!isfinite(f1) && key <= p1) o[n][3] += f1;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[s]);
        }
        // ---- the pair's sums over the four warps, and its rows ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFull, l[h], 1);
            l[h] += __shfl_xor_sync(kFull, l[h], 2);
            if (cc == 0) sm.l[w][h ? r1 : r0] = l[h];
        }
        consumers_sync();  // (the next pair's sums come after more barriers)
        const bool whole = walk.c_lo == 0 && walk.c_hi == walk.nch;
        // a pair's beginning ends this run (slot 1); its middle or end starts it (slot 0)
        const int slot = 2 * blockIdx.x + (walk.c_lo == 0 ? 1 : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h ? r1 : r0;
            if (r >= rows) continue;
            const float L = (sm.l[0][r] + sm.l[1][r]) + (sm.l[2][r] + sm.l[3][r]);
            const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;  // a NaN sum stays NaN
            if (whole) {
                const long orow = (long)(walk.r0 + r / G) * p.Hq + walk.g * G + r % G;
                __nv_bfloat16* dst = (__nv_bfloat16*)p.out + orow * D + w * NT * 8 + 2 * cc;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<uint32_t*>(dst + n * 8) = pack_bf16(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                if (p.lse && w == 0 && cc == 0)
                    p.lse[orow] = L == 0.f ? -INFINITY : (m[h] + log2f(L)) * 0.69314718055994531f;
            } else {
                float* dst = a.part_o + ((long)slot * kDR + r) * D + w * NT * 8 + 2 * cc;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                if (w == 0 && cc == 0) a.part_lse2[slot * kDR + r] = L == 0.f ? -INFINITY : m[h] + log2f(L);
            }
        }
    }
    if (!ok && lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
}

// Merge of the pairs that several runs share: a block per (kv-head, sequence,
// row).  Warp w takes partials w, w + 4, ... in order, its lanes the columns;
// the four sums are added in order.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    decode_merge_kernel(const __grid_constant__ DecodeArgs a, int grid) {
    constexpr int PL = D / 32;
    __shared__ float s_acc[kMergeWarps][D], s_w[kMergeWarps];
    const PromptArgs& p = a.p;
    const int g = blockIdx.x, b = blockIdx.y, r = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PromptSeq sq = prompt_seq(p, b);
    const int nch = decode_chunks(sq), rows = sq.n * a.G;
    long total;
    // the pair's first unit with a chunk
    const long u0 = units_before(p, b, &total) + (long)g * (nch + kPairCost) + kPairCost;
    const int n_runs = runs_used(total, grid);
    const int first = nch ? run_of(total, u0, n_runs) : 0, last = nch ? run_of(total, u0 + nch - 1, n_runs) : 0;
    // every block waits for the runs, so this launch never ends before them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (first == last || r >= rows) return;  // (a pair of one run was written by it)
    auto slot = [&](int i) { return (long)(2 * i + (i == first ? 1 : 0)) * kDR + r; };
    float M = -INFINITY;
    for (int i = first + lane; i <= last; i += 32) M = fmaxf(M, a.part_lse2[slot(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    float acc[PL], wsum = 0.f;
#pragma unroll
    for (int e = 0; e < PL; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = first + warp; i <= last; i += kMergeWarps) {
        const float w = exp2_sfu(a.part_lse2[slot(i)] - mu);
        const float* src = a.part_o + slot(i) * D + lane * PL;
        wsum += w;
#pragma unroll
        for (int e = 0; e < PL; ++e) acc[e] = fmaf(w, src[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < PL; ++e) s_acc[warp][lane * PL + e] = acc[e];
    if (lane == 0) s_w[warp] = wsum;
    __syncthreads();
    const float L = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const long orow = (long)(sq.r0 + r / a.G) * p.Hq + g * a.G + r % a.G;
    const int col = threadIdx.x;
    if (col < D) {
        const float x = (s_acc[0][col] + s_acc[1][col]) + (s_acc[2][col] + s_acc[3][col]);
        ((__nv_bfloat16*)p.out)[orow * D + col] = __float2bfloat16_rn(x * inv);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

template <int D>
constexpr size_t decode_smem() {
    return sizeof(DecodeSmem<D>);
}
static_assert(kDCtasPerSm * (decode_smem<128>() + 1024) <= 233472, "two CTAs per SM");
static_assert(kDCtasPerSm * (decode_smem<64>() + 1024) <= 233472, "two CTAs per SM");

template <int D>
cudaError_t decode_launch_d(const DecodeArgs& a, int runs, cudaStream_t st) {
    auto kern = decode_kernel<D>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)decode_smem<D>());
    if (e != cudaSuccess) return e;
    prefer_max_smem(kern);
    kern<<<runs, kDThreads, decode_smem<D>(), st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the merge may be scheduled while the runs finish; it waits for them itself
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.p.Hkv, a.p.B, a.p.max_new * a.G);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D>, a, runs);
}

}  // namespace

bool decode_supported(int B, int max_new, int Hq, int Hkv, int page_size, medusa_dtype dt) {
    return dt == MEDUSA_BF16 && attn_tc_page_ok(page_size) && (long)max_new * (Hq / Hkv) <= kDR && B <= 65535;
}

size_t decode_workspace_size(int D) { return (size_t)2 * kDCtasPerSm * num_sms() * kDR * (D + 1) * 4; }

cudaError_t decode_launch(const PromptArgs& x, cudaStream_t st) {
    DecodeArgs a;
    a.p = x;
    a.G = x.Hq / x.Hkv;
    a.page_rows = x.page_size < kDC ? x.page_size : kDC;
    const uint64_t D = x.D, ps = x.page_size, NP = (uint64_t)x.num_pages * x.Hkv;
    const uint64_t qdims[3] = {D, (uint64_t)x.Hq, (uint64_t)x.N}, qstrides[2] = {D * 2, (uint64_t)x.q_stride * 2};
    const uint32_t qbox[3] = {64, (uint32_t)a.G, (uint32_t)(kDR / a.G)};
    if (!make_tmap_bf16(&a.mq, x.q, 3, qdims, qstrides, qbox)) return cudaErrorInvalidValue;
    const uint64_t dims[3] = {D, ps, NP}, strides[2] = {D * 2, ps * D * 2};
    const uint32_t box[3] = {64, (uint32_t)a.page_rows, 1};
    if (!make_tmap_bf16(&a.mk, x.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!make_tmap_bf16(&a.mv, x.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    a.scale_log2 = x.scale * 1.4426950408889634f;
    a.wait_ns = wait_limit_ns();
    // a CTA per run, two per SM, but no more runs than there can be chunks
    const long chunks = ((long)x.max_prefix + x.max_new + kDC - 1) / kDC;
    const long units = (long)(x.B < x.N ? x.B : x.N) * x.Hkv * (chunks + kPairCost);
    const long most = (long)kDCtasPerSm * num_sms();
    const int runs = (int)(units < most ? (units < 1 ? 1 : units) : most);
    a.part_o = (float*)x.ws;
    a.part_lse2 = a.part_o + (size_t)2 * runs * kDR * D;
    return x.D == 128 ? decode_launch_d<128>(a, runs, st) : decode_launch_d<64>(a, runs, st);
}

}  // namespace medusa
