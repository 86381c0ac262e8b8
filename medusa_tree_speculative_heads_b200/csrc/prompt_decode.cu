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
// lengths are.  A CTA's run covers the end of one pair, whole pairs, and the
// beginning of another; whole pairs are written out directly, the others as
// normalised fp32 partials that a second launch merges in run order.
// Warp 0 of a CTA streams its chunks by TMA into a ring that runs on across
// pairs; warps 1-4 take 16 keys of every chunk each: S = Q K^T and O += P V
// with Q, P and O in registers, K and V by ldmatrix from the swizzled tiles,
// a running maximum and sum per row (fp32), merged over the four warps in
// shared memory at the end of a pair.  P is rounded to bf16 (2^-8 relative, as
// the operands are); l sums it unrounded.
#include "prompt_common.cuh"
#include "tc.cuh"
#include "tma.h"

namespace medusa {

namespace {

constexpr int kDR = 16;                      // query rows of a pair (mma M)
constexpr int kDC = 64;                      // keys per chunk
constexpr int kDW = 4;                       // consumer warps, 16 keys each
constexpr int kDThreads = 32 * (1 + kDW);
constexpr int kDCtasPerSm = 2;
template <int D> constexpr int d_stages() { return D == 128 ? 3 : 6; }

struct DecodeArgs {
    CUtensorMap mk, mv;  // the pools as (D, page_size, num_pages * Hkv), box (64, page_rows, 1)
    PromptArgs p;
    float* part_o;       // [2 * grid][kDR][D]
    float* part_lse2;    // [2 * grid][kDR]
    int G, page_rows;
    float scale_log2;
    uint64_t wait_ns;
};

__device__ __forceinline__ int decode_chunks(const PromptSeq& s) { return s.n > 0 ? (s.p + s.n + kDC - 1) / kDC : 0; }

// units (chunks of one kv-head) of the sequences before b; one warp
__device__ inline long units_before(const PromptArgs& p, int b, long* total) {
    const int lane = threadIdx.x & 31;
    long before = 0, all = 0;
    for (int i = lane; i < p.B; i += 32) {
        const long c = (long)decode_chunks(prompt_seq(p, i)) * p.Hkv;
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
// run of a CTA: units [total * i / n, total * (i + 1) / n) of n runs, none of
// them empty
__device__ __forceinline__ int runs_used(long total, int n) { return total < n ? (int)total : n; }
__device__ __forceinline__ long run_start(long total, int i, int n) { return total * i / n; }
// the CTA whose run holds unit u
__device__ __forceinline__ int run_of(long total, long u, int n) {
    int i = (int)(u * n / total);
    while (run_start(total, i + 1, n) <= u) ++i;
    while (run_start(total, i, n) > u) --i;
    return i;
}

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
__device__ __forceinline__ float d_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t d_pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
// barrier of the consumer warps
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kDW * 32) : "memory"); }

template <int D>
__global__ void __launch_bounds__(kDThreads, kDCtasPerSm) decode_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int NSUB = D / 64, ST = d_stages<D>();
    constexpr int kSub = kDC * 128;       // [64 keys x 64 elements]
    constexpr int kKV = NSUB * kSub;      // a chunk of K (or of V)
    constexpr int NT = D / 8;             // output column tiles
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem;                                              // [ST][K, V]
    float* s_merge = reinterpret_cast<float*>(ring + ST * 2 * kKV);    // [2][kDR][D]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_merge + 2 * kDR * D);
    uint64_t* empty = full + ST;
    float* s_ml = reinterpret_cast<float*>(empty + ST);                // [kDW][kDR][2]
    volatile int* s_run = reinterpret_cast<volatile int*>(s_ml + kDW * kDR * 2);
    volatile long* s_unit = reinterpret_cast<volatile long*>(s_run + 2);

    const PromptArgs& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_addr(smem) & 1023u) {  // never expected (uniform over the grid)
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
            long c = b0 + lane < p.B ? (long)decode_chunks(prompt_seq(p, b0 + lane)) * p.Hkv : 0;
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
            s_run[0] = found;
            s_unit[0] = base;   // first unit of that sequence
            s_unit[1] = total;
        }
        if (blockIdx.x == 0)
            for (int b = lane; b < p.B; b += 32)
                if (const int bad = prompt_seq(p, b).bad) set_status(p.status, bad);
    } else if (threadIdx.x == 32) {
        tma_prefetch_desc(&a.mk);
        tma_prefetch_desc(&a.mv);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kDW);
        }
        mbar_fence_init();
    }
    __syncthreads();
    const long total = s_unit[1];
    const int n_runs = runs_used(total, gridDim.x);
    if ((int)blockIdx.x >= n_runs) return;
    const long u0 = run_start(total, blockIdx.x, n_runs), u1 = run_start(total, blockIdx.x + 1, n_runs);

    // walk over the run: one step per (sequence, kv-head) segment
    int b = s_run[0];
    PromptSeq sq = prompt_seq(p, b);
    int nch = decode_chunks(sq);
    int g = (int)((u0 - s_unit[0]) / nch), c_lo = (int)((u0 - s_unit[0]) % nch);
    long u = u0;
    auto advance = [&](int taken) {  // to the next segment
        u += taken;
        c_lo = 0;
        if (++g == p.Hkv) {
            g = 0;
            if (u < u1)
                do {
                    sq = prompt_seq(p, ++b);
                    nch = decode_chunks(sq);
                } while (nch == 0);
        }
    };

    int it = 0;  // chunk of the run
    bool ok = true;
    if (warp == 0) {
        // ---------------- producer ----------------
        const int pr = a.page_rows, nbox = kDC / pr;
        const int box = lane % nbox, part = lane / nbox, sub = part % NSUB, kv = part / NSUB;
        const bool mine = part < 2 * NSUB;
        while (u < u1 && ok) {
            const int c_hi = (int)min((long)nch, c_lo + (u1 - u));
            const int keys = sq.p + sq.n;
            auto page_of = [&](int c) -> int {
                const int pos = c * kDC + box * pr;
                if (!mine || c >= c_hi || pos >= keys) return -1;
                const int page = p.block_table[(long)b * p.max_pages + pos / p.page_size];
                if (page >= 0 && page < p.num_pages) return page;
                set_status(p.status, MEDUSA_STATUS_BAD_PAGE);
                return -1;
            };
            int next = page_of(c_lo);
            for (int c = c_lo; c < c_hi; ++c, ++it) {
                const int page = next, s = it % ST;
                next = page_of(c + 1);
                const unsigned loads = __ballot_sync(kFull, page >= 0);
                if (it >= ST && !__all_sync(kFull, mbar_wait(&empty[s], ((it / ST) - 1) & 1, a.wait_ns))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(__popc(loads) * pr * 128));
                __syncwarp();
                if (page >= 0)
                    tma_load_3d(ring + s * 2 * kKV + kv * kKV + sub * kSub + box * pr * 128, kv ? &a.mv : &a.mk,
                                sub * 64, (c * kDC + box * pr) % p.page_size, page * p.Hkv + g, &full[s]);
            }
            advance(c_hi - c_lo);
        }
        if (!ok && lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
        // drain: no copy may still be landing when the CTA exits
        for (int i = max(0, it - ST); i < it; ++i) mbar_wait(&full[i % ST], (i / ST) & 1);
        return;
    }
    // ---------------- consumers ----------------
    const int w = warp - 1, r0 = lane >> 2, r1 = r0 + 8, cc = lane & 3;
    const int G = a.G;
    // ldmatrix rows of this lane: matrix lane / 8, row lane % 8
    const int mi = lane >> 3, mr = lane & 7;
    const int k_key = w * 16 + (mi >> 1) * 8 + mr, k_ch = mi & 1;  // K: (keys, 16-byte column) of the matrix
    const int v_key = w * 16 + (mi & 1) * 8 + mr, v_ch = mi >> 1;  // V
    while (u < u1) {
        const int c_hi = (int)min((long)nch, c_lo + (u1 - u));
        const int rows = sq.n * G;
        const int p0 = r0 < rows ? sq.p + r0 / G : -1, p1 = r1 < rows ? sq.p + r1 / G : -1;  // positions of the rows
        uint32_t q[D / 16][4];
        {
            const __nv_bfloat16* qb = (const __nv_bfloat16*)p.q + (long)g * G * D + 2 * cc;
            const __nv_bfloat16* q0 = qb + (long)(sq.r0 + r0 / G) * p.q_stride + (r0 % G) * D;
            const __nv_bfloat16* q1 = qb + (long)(sq.r0 + r1 / G) * p.q_stride + (r1 % G) * D;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                q[ks][0] = p0 >= 0 ? *reinterpret_cast<const uint32_t*>(q0 + ks * 16) : 0u;
                q[ks][1] = p1 >= 0 ? *reinterpret_cast<const uint32_t*>(q1 + ks * 16) : 0u;
                q[ks][2] = p0 >= 0 ? *reinterpret_cast<const uint32_t*>(q0 + ks * 16 + 8) : 0u;
                q[ks][3] = p1 >= 0 ? *reinterpret_cast<const uint32_t*>(q1 + ks * 16 + 8) : 0u;
            }
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int c = c_lo; c < c_hi; ++c, ++it) {
            const int s = it % ST;
            if (ok) ok = __all_sync(kFull, mbar_wait(&full[s], (it / ST) & 1, a.wait_ns));
            if (!ok) continue;
            const uint32_t sk = smem_addr(ring + s * 2 * kKV), sv = sk + kKV;
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
            const bool part = key0 + 16 > sq.p + 1;  // some row does not see some of the warp's keys
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 8 * n + 2 * cc + (e & 1);
                    if (part && key > (e < 2 ? p0 : p1)) sc[n][e] = -INFINITY;
                    mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
                }
            float al[2];
            bool raised = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
                mx[h] *= a.scale_log2;
                const bool raise = mx[h] > m[h] + 8.f;  // a new reference only when it rises by more than 2^8
                al[h] = 1.f;
                if (raise) {
                    al[h] = d_exp2(m[h] - mx[h]);
                    m[h] = mx[h];
                    raised = true;
                }
            }
            uint32_t pa[4];
            float rs[2] = {0.f, 0.f};
            {
                const float mu0 = m[0] == -INFINITY ? 0.f : m[0], mu1 = m[1] == -INFINITY ? 0.f : m[1];
                float pv[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pv[n][e] = d_exp2(fmaf(sc[n][e], a.scale_log2, e < 2 ? -mu0 : -mu1));
                        rs[e >> 1] += pv[n][e];
                    }
                pa[0] = d_pack(pv[0][0], pv[0][1]);
                pa[1] = d_pack(pv[0][2], pv[0][3]);
                pa[2] = d_pack(pv[1][0], pv[1][1]);
                pa[3] = d_pack(pv[1][2], pv[1][3]);
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
                // not reach such a row) and added to the rows that see it
                const int keys = sq.p + sq.n;
                uint8_t* vt = ring + s * 2 * kKV + kKV + w * 16 * 128;
                bool dirty = false;
                for (int e = lane; e < 16 * NSUB * 8; e += 32) {
                    const int row = e / (NSUB * 8), x = e % (NSUB * 8);
                    const uint4 v = *reinterpret_cast<const uint4*>(vt + (x >> 3) * kSub + row * 128 + (x & 7) * 16);
                    dirty |= key0 + row < keys && (nonfinite2(v.x) | nonfinite2(v.y) | nonfinite2(v.z) | nonfinite2(v.w));
                }
                if (__any_sync(kFull, dirty)) {
                    for (int row = 0; row < 16 && key0 + row < keys; ++row)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t v2 = *reinterpret_cast<const uint32_t*>(
                                vt + (n >> 3) * kSub + row * 128 + (((n & 7) ^ (row & 7)) << 4) + 4 * cc);
                            if (nonfinite2(v2)) {
                                const float f0 = bf16lo(v2), f1 = bf16hi(v2);
                                const int key = key0 + row;
                                if (!isfinite(f0) && key <= p0) o[n][0] += f0;
                                if (!isfinite(f1) && key <= p0) o[n][1] += f1;
                                if (!isfinite(f0) && key <= p1) o[n][2] += f0;
                                if (!isfinite(f1) && key <= p1) o[n][3] += f1;
                            }
                        }
                    __syncwarp();
                }
                for (int e = lane; e < 16 * NSUB * 8; e += 32) {
                    const int row = e / (NSUB * 8), x = e % (NSUB * 8);
                    uint4* at = reinterpret_cast<uint4*>(vt + (x >> 3) * kSub + row * 128 + (x & 7) * 16);
                    uint4 v = *at;
                    if (key0 + row >= keys) v = make_uint4(0u, 0u, 0u, 0u);
                    *at = make_uint4(clear2(v.x, nonfinite2(v.x)), clear2(v.y, nonfinite2(v.y)),
                                     clear2(v.z, nonfinite2(v.z)), clear2(v.w, nonfinite2(v.w)));
                }
                // the slot's next copy is by the async proxy, after these writes
                fence_proxy_async_shared();
                __syncwarp();
            }
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t vb[4];
                const int ch = n + v_ch;
                ldsm4_t(sv + (ch >> 3) * kSub + v_key * 128 + (((ch & 7) ^ mr) << 4), vb);
                mma16816(o[n], pa, vb[0], vb[1]);
                mma16816(o[n + 1], pa, vb[2], vb[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        // ---- merge of the four warps: common maximum, then two rounds of adding ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFull, l[h], 1);
            l[h] += __shfl_xor_sync(kFull, l[h], 2);
            if (cc == 0) {
                s_ml[(w * kDR + (h ? r1 : r0)) * 2] = m[h];
                s_ml[(w * kDR + (h ? r1 : r0)) * 2 + 1] = l[h];
            }
        }
        consumers_sync();
        float M[2], L[2], f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            M[h] = -INFINITY;
            L[h] = 0.f;
            const float* ml = s_ml + (h ? r1 : r0) * 2;
#pragma unroll
            for (int x = 0; x < kDW; ++x) M[h] = fmaxf(M[h], ml[x * kDR * 2]);
            const float mu = M[h] == -INFINITY ? 0.f : M[h];
#pragma unroll
            for (int x = 0; x < kDW; ++x) L[h] += ml[x * kDR * 2 + 1] * d_exp2(ml[x * kDR * 2] - mu);
            f[h] = d_exp2(m[h] - mu);
        }
        auto put = [&](float* dst) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(dst + r0 * D + n * 8 + 2 * cc) = make_float2(o[n][0], o[n][1]);
                *reinterpret_cast<float2*>(dst + r1 * D + n * 8 + 2 * cc) = make_float2(o[n][2], o[n][3]);
            }
        };
        auto add = [&](const float* src) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 x = *reinterpret_cast<const float2*>(src + r0 * D + n * 8 + 2 * cc);
                const float2 y = *reinterpret_cast<const float2*>(src + r1 * D + n * 8 + 2 * cc);
                o[n][0] += x.x;
                o[n][1] += x.y;
                o[n][2] += y.x;
                o[n][3] += y.y;
            }
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            o[n][0] *= f[0];
            o[n][1] *= f[0];
            o[n][2] *= f[1];
            o[n][3] *= f[1];
        }
        if (w >= 2) put(s_merge + (w - 2) * kDR * D);
        consumers_sync();
        if (w < 2) add(s_merge + w * kDR * D);
        consumers_sync();
        if (w == 1) put(s_merge);
        consumers_sync();
        if (w == 0) {
            add(s_merge);
            if (!ok && lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
            const bool whole = c_lo == 0 && c_hi == nch;
            // a pair's beginning ends this run (slot 1); its middle or end starts it (slot 0)
            const int slot = 2 * blockIdx.x + (c_lo == 0 ? 1 : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h ? r1 : r0;
                if (r >= rows) continue;
                const float inv = L[h] > 0.f ? 1.f / L[h] : L[h] == 0.f ? 0.f : L[h];
                if (whole) {
                    const long orow = (long)(sq.r0 + r / G) * p.Hq + g * G + r % G;
                    __nv_bfloat16* dst = (__nv_bfloat16*)p.out + orow * D + 2 * cc;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<uint32_t*>(dst + n * 8) = d_pack(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                    if (p.lse && cc == 0)
                        p.lse[orow] = L[h] == 0.f ? -INFINITY : (M[h] + log2f(L[h])) * 0.69314718055994531f;
                } else {
                    float* dst = a.part_o + ((long)slot * kDR + r) * D + 2 * cc;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                    if (cc == 0) a.part_lse2[slot * kDR + r] = L[h] == 0.f ? -INFINITY : M[h] + log2f(L[h]);
                }
            }
        }
        consumers_sync();  // s_ml and s_merge are free again
        advance(c_hi - c_lo);
    }
}

// Merge of the pairs that several runs share, in run order: a block per
// (kv-head, sequence), a warp per row.
template <int D>
__global__ void __launch_bounds__(256) decode_merge_kernel(const __grid_constant__ DecodeArgs a, int grid) {
    const PromptArgs& p = a.p;
    const int g = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PromptSeq sq = prompt_seq(p, b);
    const int nch = decode_chunks(sq), rows = sq.n * a.G;
    long total;
    const long u0 = units_before(p, b, &total) + (long)g * nch;
    const int n_runs = runs_used(total, grid);
    const int first = nch ? run_of(total, u0, n_runs) : 0, last = nch ? run_of(total, u0 + nch - 1, n_runs) : 0;
    // every block waits for the runs, so this launch never ends before them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (first == last || warp >= rows) return;  // (a pair of one run was written by it)
    constexpr int PL = D / 32;
    auto slot = [&](int i) { return 2 * i + (i == first ? 1 : 0); };
    for (int r = warp; r < rows; r += 8) {
        float M = -INFINITY;
        for (int i = first + lane; i <= last; i += 32) M = fmaxf(M, a.part_lse2[slot(i) * kDR + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        const float mu = M == -INFINITY ? 0.f : M;
        float acc[PL], wsum = 0.f;
#pragma unroll
        for (int e = 0; e < PL; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int i = first; i <= last; ++i) {
            const float w = d_exp2(a.part_lse2[slot(i) * kDR + r] - mu);
            const float* src = a.part_o + ((long)slot(i) * kDR + r) * D + lane * PL;
            wsum += w;
#pragma unroll
            for (int e = 0; e < PL; ++e) acc[e] = fmaf(w, src[e], acc[e]);
        }
        const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
        const long orow = (long)(sq.r0 + r / a.G) * p.Hq + g * a.G + r % a.G;
        uint32_t* dst = reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.out + orow * D + lane * PL);
#pragma unroll
        for (int e = 0; e < PL; e += 2) dst[e / 2] = d_pack(acc[e] * inv, acc[e + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[orow] = wsum == 0.f ? -INFINITY : (M + log2f(wsum)) * 0.69314718055994531f;
    }
}

template <int D>
constexpr size_t decode_smem() {
    return (size_t)d_stages<D>() * 2 * kDC * D * 2 + 2 * kDR * D * 4 + 2 * d_stages<D>() * 8 + kDW * kDR * 8 + 8 + 16 + 8;
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
    cfg.gridDim = dim3(a.p.Hkv, a.p.B);
    cfg.blockDim = dim3(256);
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
    const uint64_t dims[3] = {D, ps, NP}, strides[2] = {D * 2, ps * D * 2};
    const uint32_t box[3] = {64, (uint32_t)a.page_rows, 1};
    if (!make_tmap_bf16(&a.mk, x.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!make_tmap_bf16(&a.mv, x.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    a.scale_log2 = x.scale * 1.4426950408889634f;
    a.wait_ns = wait_limit_ns();
    // a CTA per run, two per SM, but no more runs than there can be chunks
    const long units = (long)(x.B < x.N ? x.B : x.N) * x.Hkv * (((long)x.max_prefix + x.max_new + kDC - 1) / kDC);
    const long most = (long)kDCtasPerSm * num_sms();
    const int runs = (int)(units < most ? (units < 1 ? 1 : units) : most);
    a.part_o = (float*)x.ws;
    a.part_lse2 = a.part_o + (size_t)2 * runs * kDR * D;
    return x.D == 128 ? decode_launch_d<128>(a, runs, st) : decode_launch_d<64>(a, runs, st);
}

}  // namespace medusa
