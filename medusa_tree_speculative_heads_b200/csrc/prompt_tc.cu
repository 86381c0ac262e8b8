// Causal attention of packed new rows on the 5th-generation tensor cores
// (bf16, head_dim 64/128): whole prompts over packed K/V, and chunks of new
// tokens over a paged cache.
//
// One CTA takes two 128-row query tiles of one (sequence, kv-head) -- rows are
// token-major, row = token * G + (query head of the group), so the G heads of
// a token share every K/V element; T = 128 / G tokens per tile -- and a run of
// 128-key chunks.  Per tile and chunk:
//   S  = Q K^T     tcgen05.mma M=128 N=128 K=D
//   P  = exp2(S * scale * log2 e - m), masked; bf16, over S's columns in TMEM
//   O += P V       tcgen05.mma M=128 N=D K=128 (A = P from TMEM, V MN-major)
// with the reference m and the sum l of each row in the fp32 registers of its
// softmax thread.  P is rounded to bf16 (2^-8 relative, as the operands are);
// l sums it unrounded.
//
// Any m gives the same result as long as nothing overflows, so no maximum is
// taken after the first chunk: the sum of a chunk's weights bounds them.  When
// it exceeds 2^8, m is raised by its logarithm, and O in TMEM rescaled, before
// the next chunk; when the sum of a part of the chunk exceeds 2^32 (or is not a
// number) the chunk's maximum is taken after all, m raised at once, and the
// part's weights are computed again.  (Taking the maximum of 128 scores first
// cost 400 of a chunk's 4200 cycles.)
//
// Warps: 0 and 3 producers (TMA: Q and K, V), 1 and 2 MMA issue of tiles 0 and
// 1 (1 also TMEM allocation), 4-7 softmax of tile 0, 8-11 of tile 1.  All 512
// TMEM columns are in use (2 x 128 of S, 2 x 128 of O), so a tile alternates
// between its softmax and its products; tile 1 starts a softmax later, so that
// one tile's softmax runs beside the other's products (both in step: 15%
// slower).  P is handed over in two parts, so that PV runs while the last
// exponentials are taken.  64-key chunks with two S buffers let QK run ahead,
// but a product with N = 64 takes 50 cycles against 64 with N = 128 (its A
// operand costs the same shared-memory reads), and the kernel came out no
// faster; two threads per row, turns at the exponentials, and a polynomial on
// the FMA pipe for a part of them (22 cycles a value of a warp, the SFU's 8)
// were all slower.
//
// Bound: a chunk costs each tile 2 x 512 tensor cycles (D = 128) and 128 x 128
// exponentials, 1024 cycles of the SM's 16 per clock.  One tile alone takes
// 3300 cycles a chunk (softmax 1650, products 1024, two hand-overs of some 200
// to 300), both together 4300: each slows the other's exponentials and
// products.  One prompt of 32768 tokens, 32/8 heads of 128: 7.7 to 8.4 ms, 1.05
// to 1.15 PFLOP/s (6.84 ms, 1.29 PFLOP/s, after some seconds of idling, before the
// clock drops under the power cap); 2048 tokens 46 us; 16 prompts of up to 4096,
// 240 us.
//
// What a CTA does once costs it some 9000 cycles beside 3700 per chunk: up to 5000
// to its first S (launch, tile, and some 512 copied lines of 128 bytes for the Q
// and K of the first product, served in the order of their issue, so they come
// first), 4000 from its last product on (half of it 64 KB through the SM's write
// path).  Finding its tile among several sequences costs 3000 cycles more; a
// large grid gets its tiles from a launch of its own, which this one starts under.
// Tried and slower: persistent CTAs that load across tiles (their loop over
// chunks is 5 to 10% slower, one ring stage less costs another 2%), the first
// copies issued before the block's first barrier (2%), an epilogue of rolled
// loops (2%).
//
// The visible keys of a row are 0 .. its position, so only the chunks that
// reach past the tile's first position need a mask.  In those, V elements
// that are not finite are cleared in shared memory (0 * NaN must not reach a
// row that does not see the key) and added back, from global memory, to the
// rows that do see them.
// Every pipeline wait is bounded and sets MEDUSA_STATUS_TIMEOUT on expiry.
#include "prompt_common.cuh"
#include "tc.cuh"
#include "tma.h"

namespace medusa {

namespace {

constexpr int kPW = 12;             // warps: 0 and 3 producers, 1 and 2 MMA, 4-11 softmax
constexpr int kPM = kPromptTcRows;  // rows of a query tile
constexpr int kParts = 3;           // most chunks that some row of a CTA sees in part: its 256 tokens and a first chunk
constexpr int kPC = kPromptTcKeys;  // keys per chunk
constexpr int kPParts = 2;          // parts of P
// K and V chunks share one ring (K0 V0 K1 V1 ...)
template <int D> constexpr int p_stages() { return D == 128 ? 5 : 8; }

struct PromptTcArgs {
    CUtensorMap mq;  // q as (D, Hq, N), box (64, G, T)
    CUtensorMap mk;  // packed: k as (D, Hkv, N), box (64, 1, 128); paged: the pool as
    CUtensorMap mv;  //   (D, page_size, num_pages * Hkv), box (64, page_rows, 1)
    PromptArgs p;
    SplitBuf buf;
    int G, T, page_rows;
    FastDiv div_2T, div_G;
    const int4* table;  // the grid's tiles, two entries of four each (NULL: every CTA finds its own)
    float scale_log2;
    uint64_t wait_ns;
};

// two fp32 values in one 64-bit register: the FMA pipe takes both at once
__device__ __forceinline__ uint64_t f2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a condition whose code belongs out of the way of the hot path
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

// MN-major operand as TMA writes a (64 MN x rows K) box with a 128-byte
// swizzle: 8 K-rows of 128 bytes per 1024-byte group; `lbo`: byte distance to
// the next 64-element MN block
__device__ __forceinline__ uint64_t p_mnmajor_desc(uint32_t addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// The tiles of a grid, a warp each: {b, t, r0, n}, {p}.
__global__ void __launch_bounds__(256) prompt_table_kernel(const __grid_constant__ PromptTcArgs a, int4* table,
                                                           int tiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int idx = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (idx >= tiles) return;
    const PromptTile t = prompt_tile(a.p, 2 * a.T, a.div_2T, idx);
    if ((threadIdx.x & 31) != 0) return;
    table[2 * idx] = make_int4(t.b, t.t, t.s.r0, t.s.n);
    table[2 * idx + 1] = make_int4(t.s.p, 0, 0, 0);
}

template <int D, bool kTestWaits>
__global__ void __launch_bounds__(kPW * 32, 1) prompt_tc_kernel(const __grid_constant__ PromptTcArgs a) {
    const uint64_t wait_ns = kTestWaits ? a.wait_ns : kWaitLimitNs;
    constexpr int NSUB = D / 64;
    constexpr int kQSub = kPM * 128, kQTile = NSUB * kQSub;  // [128 rows x 64 elements] block, a Q tile
    constexpr int kSub = kPC * 128, kTile = NSUB * kSub;     // [128 keys x 64 elements] block, a chunk of K or V
    constexpr int ST = p_stages<D>();
    constexpr uint32_t kIdescQK = idesc_bf16_f32(kPM, kPC);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kPM, D) | (1u << 16);  // B (V) MN-major
    constexpr uint32_t kTmemCols = 512;        // S: 128 columns per tile, O: D columns at 256 and 384
    // 1024-byte aligned when the kernel has no static shared memory (checked)
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sQ = smem;
    uint8_t* sKV = sQ + 2 * kQTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + ST * kTile);
    uint64_t* q_full = bars;           // [2]
    uint64_t* kv_full = q_full + 2;    // [ST]
    uint64_t* kv_empty = kv_full + ST;
    uint64_t* s_full = kv_empty + ST;  // [2]
    uint64_t* p_full = s_full + 2;     // [2][kPParts]
    uint64_t* o_full = p_full + 2 * kPParts;  // [2] one phase per part of a PV product
    uint64_t* o_last = o_full + 2;     // [2] a single phase: the tile's last PV
    uint64_t* v_clean = o_last + 2;    // [kParts] V of the chunks that some row sees in part is cleared
    uint64_t* stagger = v_clean + kParts;  // tile 0's first softmax is done
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stagger + 1);
    volatile int* s_tile = reinterpret_cast<volatile int*>(tmem_slot + 1);  // b, t, r0, n, p, dirty, chunks of K and V issued

    const PromptArgs& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x % p.Hkv, C = gridDim.y, split = blockIdx.y;
    const int T = a.T, G = a.G;
    if (C > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge of splits
    if (smem_addr(smem) & 1023u) {  // never expected (uniform over the grid)
        if (threadIdx.x == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
        return;
    }
    if (warp == 0) {
        if (!a.table) {
            const PromptTile t = prompt_tile(p, 2 * T, a.div_2T, blockIdx.x / p.Hkv);
            if (lane == 0) {
                s_tile[0] = t.b;
                s_tile[1] = t.t;
                s_tile[2] = t.s.r0;
                s_tile[3] = t.s.n;
                s_tile[4] = t.s.p;
            }
        }
        if (lane == 0) s_tile[5] = 0;
        if (blockIdx.x == 0 && split == 0)
            for (int b = lane; b < p.B; b += 32)
                if (const int bad = prompt_seq(p, b).bad) set_status(p.status, bad);
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
    } else if (threadIdx.x == 64) {
        tma_prefetch_desc(&a.mq);
        tma_prefetch_desc(&a.mk);
        tma_prefetch_desc(&a.mv);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&s_full[i], 1);
            for (int x = 0; x < kPParts; ++x) mbar_init(&p_full[i * kPParts + x], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_last[i], 1);
        }
        for (int i = 0; i < kParts; ++i) mbar_init(&v_clean[i], 4);
        mbar_init(stagger, 4);
        mbar_fence_init();
    }
    int4 found;
    int first;
    if (a.table) {  // written by the launch before, which this one may have started under
        asm volatile("griddepcontrol.wait;" ::: "memory");
        found = __ldcg(a.table + 2 * (blockIdx.x / p.Hkv));
        first = __ldcg(a.table + 2 * (blockIdx.x / p.Hkv) + 1).x;
    }
    tc_fence_before();
    sync_block();
    tc_fence_after();
    if (!a.table) {
        found = make_int4(s_tile[0], s_tile[1], s_tile[2], s_tile[3]);
        first = s_tile[4];
    }
    const uint32_t tmem = *tmem_slot;
    const int b = found.x;
    const struct {
        int r0, n, p;
    } sq = {found.z, found.w, first};
    const int tok0 = found.y * 2 * T;
    const int ntok = b < 0 ? 0 : min(2 * T, sq.n - tok0);
    const int pos0 = sq.p + tok0;                       // the first row's position
    const int keys = pos0 + ntok;                       // seen by the last row
    const int nch = b < 0 ? 0 : (keys + kPC - 1) / kPC;  // chunks of the longer tile
    const int c0 = C == 1 ? 0 : nch * split / C, c1 = C == 1 ? nch : nch * (split + 1) / C;
    // chunks of each tile within this split
    auto count = [&](int tile) {
        const int n = min(T, ntok - tile * T);
        if (n <= 0) return 0;
        return max(0, min(c1, (pos0 + tile * T + n + kPC - 1) / kPC) - c0);
    };
    const int cnt0 = count(0), cnt1 = count(1), cmax = max(cnt0, cnt1);
    const bool paged = p.block_table != nullptr;

    // Waits of the MMA and softmax warps: after one has expired the chunks are
    // passed through without waiting (the results mean nothing), so that every
    // barrier still meets its threads.  Each lane polls for itself.
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
        if (rare(ok && (kTestWaits || !mbar_try_wait(bar, parity)))) ok = mbar_wait(bar, parity, wait_ns);
        __syncwarp();
    };
    if (warp < 4) {
        // Registers: 384 threads are launched with 168 each; the softmax warps take
        // the others' share (88 + 2 * 208 = 3 * 168).
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0 || warp == 3) {
            // ---------------- producers: K (and Q), V ----------------
            // Like the MMA warps these run converged and one elected lane issues: a
            // copy per lane goes through the lanes one after the other, some 100
            // cycles each, and 16-row pages make 16 copies of a chunk of K.
            if (cmax > 0) {
                const bool lead = elect_one();
                const int kv = warp == 3;
                auto load_q = [&](int tile) {
                    if ((tile == 0 ? cnt0 : cnt1) > 0 && lead) {
                        mbar_arrive_expect_tx(&q_full[tile], (uint32_t)(T * G * 128 * NSUB));
#pragma unroll
                        for (int sub = 0; sub < NSUB; ++sub)
                            tma_load_3d(sQ + tile * kQTile + sub * kQSub, &a.mq, sub * 64, g * G,
                                        sq.r0 + tok0 + tile * T, &q_full[tile]);
                    }
                    __syncwarp();
                };
                // Copies are served in the order of their issue, and filling Q and the
                // ring takes some 3400 cycles: the Q and K of the first product come
                // first, and V waits for them (2048 tokens 46.7 -> 45 us).
                if (kv == 0) load_q(0);
                else asm volatile("bar.sync 2, 64;" ::: "memory");
                // a chunk's boxes of page_rows (packed: all 128) keys; a lane looks one up
                const int pr = paged ? a.page_rows : kPC, nbox = kPC / pr;
                const CUtensorMap* map = kv ? &a.mv : &a.mk;
                // (row in the page or packed row, page * Hkv + kv-head or kv-head); z < 0: not loaded
                auto look_up = [&](int j, int& y, int& z) {
                    const int pos = (c0 + j) * kPC + lane * pr;
                    y = 0;
                    z = -1;
                    if (lane >= nbox || j >= cmax || pos >= keys) return;
                    if (!paged) {
                        y = sq.r0 + pos;
                        z = g;
                        return;
                    }
                    const int page = p.block_table[(long)b * p.max_pages + pos / p.page_size];
                    if (page >= 0 && page < p.num_pages) {
                        y = pos % p.page_size;
                        z = page * p.Hkv + g;
                    } else {
                        set_status(p.status, MEDUSA_STATUS_BAD_PAGE);
                    }
                };
                int next_y, next_z, issued = 0;
                look_up(0, next_y, next_z);
                for (int j = 0; j < cmax; ++j) {
                    const int y = next_y, z = next_z, i = 2 * j + kv, s = i % ST;
                    look_up(j + 1, next_y, next_z);  // one chunk ahead: in flight during this chunk's wait
                    const unsigned loads = __ballot_sync(kFull, z >= 0);
                    // The stage's last copy has landed when its readers are done, unless a wait
                    // expired and they passed it over: a barrier then must not be armed
                    // for a second copy on top of the first.
                    const int last = ((i / ST) - 1) & 1;
                    if (i >= ST && !(__all_sync(kFull, mbar_wait(&kv_empty[s], last, wait_ns)) &&
                                     __all_sync(kFull, mbar_wait(&kv_full[s], last, wait_ns)))) {
                        if (lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
                        break;
                    }
                    if (lead) mbar_arrive_expect_tx(&kv_full[s], (uint32_t)(__popc(loads) * NSUB * pr * 128));
                    ++issued;
                    for (int x = 0; x < nbox; ++x) {
                        const int by = __shfl_sync(kFull, y, x), bz = __shfl_sync(kFull, z, x);
                        if (bz < 0) continue;
                        if (lead) {
#pragma unroll
                            for (int sub = 0; sub < NSUB; ++sub)
                                tma_load_3d(sKV + s * kTile + sub * kSub + x * pr * 128, map, sub * 64,
                                            paged ? by : bz, paged ? bz : by, &kv_full[s]);
                        }
                        __syncwarp();
                    }
                    if (j == 0 && kv == 0) {
                        load_q(1);
                        asm volatile("bar.arrive 2, 64;" ::: "memory");
                    }
                }
                // drain: no copy may still be landing when the CTA exits
                if (kv == 0 && cnt0 > 0) mbar_wait(&q_full[0], 0);
                if (kv == 0 && cnt1 > 0) mbar_wait(&q_full[1], 0);
                if (lane == 0) s_tile[6 + kv] = issued;
                asm volatile("bar.sync 1, 64;" ::: "memory");  // the two producers
                const int others = s_tile[7 - kv];
                for (int j = max(0, issued - ST); j < issued; ++j) {
                    const int i = 2 * j + kv, next = i + ST;  // (a stage that was used again had landed)
                    if (next >> 1 >= ((next & 1) == kv ? issued : others)) mbar_wait(&kv_full[i % ST], (i / ST) & 1);
                }
            }
        } else if (warp < 3) {
            // ---------------- MMA issuer of a tile ----------------
            // A warp per tile, so that the waits of one do not hold up the other's
            // products.  The whole warp runs the loop, so that descriptors and
            // addresses stay in uniform registers; one elected lane issues.
            const int tile = warp - 1;
            const int n = __shfl_sync(kFull, tile ? cnt1 : cnt0, 0), other = __shfl_sync(kFull, tile ? cnt0 : cnt1, 0);
            if (n > 0) {
                const bool lead = elect_one();
                const uint32_t tm = __shfl_sync(kFull, tmem, 0);
                // a stage is free after one arrival for each tile (two of the only one that uses it)
                auto release = [&](int s, int j) {
                    tc_commit(&kv_empty[s]);
                    if (j >= other) tc_commit(&kv_empty[s]);
                };
                const uint64_t qd = sw128_kmajor_desc(smem_addr(sQ) + tile * kQTile);
                const uint64_t kd = sw128_kmajor_desc(smem_addr(sKV));
                const uint64_t vd = p_mnmajor_desc(smem_addr(sKV), kSub);
                const uint32_t t_s = tm + tile * kPC, t_o = tm + 256 + tile * 128;
                auto issue_qk = [&](int j) {
                    const int i = 2 * j, s = i % ST;
                    wait(&kv_full[s], (i / ST) & 1);
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int sub = 0; sub < NSUB; ++sub)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_bf16(t_s, qd + (uint64_t)((sub * kQSub) >> 4) + 2 * ks,
                                            kd + (uint64_t)((s * kTile + sub * kSub) >> 4) + 2 * ks, kIdescQK,
                                            (sub | ks) != 0);
                        // completes after this tile's products so far: its last PV too
                        tc_commit(&s_full[tile]);
                        release(s, j);
                    }
                    __syncwarp();
                };
                wait(&q_full[tile], 0);
                issue_qk(0);
                for (int j = 0; j < n; ++j) {
                    const int i = 2 * j + 1, s = i % ST;
                    const uint64_t bd = vd + (uint64_t)((s * kTile) >> 4);
                    auto pv = [&](int ks) {  // 16 keys: 8 columns of P, two 1024-byte groups of V
                        tc_mma_bf16_ts(t_o, t_s + ks * 8, bd + (uint64_t)(2048 >> 4) * ks, kIdescPV, (j | ks) != 0);
                    };
                    wait(&kv_full[s], (i / ST) & 1);
                    const int part = c0 + j - (pos0 + 1) / kPC;
                    if (part >= 0) wait(&v_clean[part], 0);
#pragma unroll
                    for (int x = 0; x < kPParts; ++x) {
                        constexpr int kSteps = kPC / 16 / kPParts;
                        wait(&p_full[tile * kPParts + x], j & 1);
                        tc_fence_after();
                        if (lead) {
#pragma unroll
                            for (int ks = 0; ks < kSteps; ++ks) pv(x * kSteps + ks);
                            tc_commit(&o_full[tile]);
                        }
                        __syncwarp();
                    }
                    if (lead) {
                        release(s, j);
                        if (j + 1 == n) tc_commit(&o_last[tile]);
                    }
                    __syncwarp();
                    if (j + 1 < n) issue_qk(j + 1);  // over P: the products run in issue order
                }
                if (!ok) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
                mbar_wait(&o_last[tile], 0);  // every product issued has finished writing TMEM
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------- softmax ----------------
        const int tile = warp >= 8 ? 1 : 0, cnt = tile ? cnt1 : cnt0;
        const int lr = (warp & 3) * 32 + lane;  // TMEM lane = row of the tile
        const int row_tok = div_by(lr, a.div_G), row_head = lr - row_tok * G;
        const int tok = tile * T + row_tok;
        const bool row_ok = lr < T * G && tok < ntok;
        const int pos = row_ok ? pos0 + tok : -1;  // a row of no token sees no key
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + tile * kPC, to = lane_base + 256 + tile * 128;
        const uint64_t sc2 = f2(a.scale_log2, a.scale_log2);
        float m = -INFINITY, l = 0.f;
        bool pending = false;  // the last weights were large: m is to be raised by `rise`
        float rise = 0.f;
        auto raise = [&](int done) {  // after `done` parts of PV products
            const float alpha = pending ? exp2_sfu(-rise) : 1.f;
            if (pending) m += rise;
            pending = false;
            l *= alpha;
            if (done == 0) return;
            wait(&o_full[tile], (done - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t ro[1][16];
                tmem_ld16_async(to + c * 16, ro[0]);
                tmem_wait_ld(ro);
#pragma unroll
                for (int e = 0; e < 16; ++e) ro[0][e] = __float_as_uint(__uint_as_float(ro[0][e]) * alpha);
                tmem_st16(to + c * 16, ro[0]);
            }
        };
        for (int j = 0; j < cnt; ++j) {
            const int key0 = (c0 + j) * kPC;
            // the first tile to use a chunk that some row sees only in part clears its V
            if (rare(key0 + kPC > pos0 + 1 && (tile == 0 || j >= cnt0))) {
                const int i = 2 * j + 1, s = i % ST;
                wait(&kv_full[s], (i / ST) & 1);
                uint8_t* row = sKV + s * kTile + lr * 128;  // a thread per key
#pragma unroll 8
                for (int x = 0; x < NSUB * 8; ++x) {
                    uint4* at = reinterpret_cast<uint4*>(row + (x >> 3) * kSub + ((x + lr) & 7) * 16);
                    if (key0 + lr >= keys) {  // no row sees this key: whatever is there
                        *at = make_uint4(0u, 0u, 0u, 0u);
                        continue;
                    }
                    const uint4 w = *at;
                    const uint32_t b0 = nonfinite2(w.x), b1 = nonfinite2(w.y);
                    const uint32_t b2 = nonfinite2(w.z), b3 = nonfinite2(w.w);
                    if (b0 | b1 | b2 | b3) {
                        *at = make_uint4(clear2(w.x, b0), clear2(w.y, b1), clear2(w.z, b2), clear2(w.w, b3));
                        s_tile[5] = 1;
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_clean[c0 + j - (pos0 + 1) / kPC]);
            }
            if (tile == 1 && j == 0 && cnt0 > 2) wait(stagger, 0);  // (few chunks: no time to make up for it)
            wait(&s_full[tile], j & 1);
            tc_fence_after();
            uint32_t raw[kPC / 16][16];
#pragma unroll
            for (int c = 0; c < kPC / 16; ++c) tmem_ld16_async(ts + c * 16, raw[c]);
            tmem_wait_ld(raw);
            const int lim = pos - key0;  // visible: c <= lim
            if (rare(__any_sync(kFull, lim < kPC - 1))) {
#pragma unroll
                for (int c = 0; c < kPC; ++c)
                    raw[c >> 4][c & 15] = c <= lim ? raw[c >> 4][c & 15] : 0xff800000u;
            }
            auto row_max = [&] {
                float m4[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) m4[c] = __uint_as_float(raw[0][c]);
#pragma unroll
                for (int c = 4; c < kPC; ++c) m4[c & 3] = fmaxf(m4[c & 3], __uint_as_float(raw[c >> 4][c & 15]));
                return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
            };
            // the first chunk with a score above -inf sets the reference (O and l are still 0)
            if (rare(__any_sync(kFull, m == -INFINITY && lim >= 0))) {
                const float mx = row_max();
                if (m == -INFINITY) m = mx;
            }
            if (rare(__any_sync(kFull, pending))) raise(j * kPParts);
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < kPParts; ++x) {
                constexpr int kPairs = kPC / 2 / kPParts;
                uint32_t pk[kPairs / 16][16];
                float part;
                for (int again = 0;; ++again) {
                    const float mu = m == -INFINITY ? 0.f : m;
                    const uint64_t mu2 = f2(-mu, -mu);
                    uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const int k = 2 * (x * kPairs + e);
                        const uint64_t t = fma2(f2(__uint_as_float(raw[k >> 4][k & 15]),
                                                   __uint_as_float(raw[k >> 4][(k & 15) + 1])), sc2, mu2);
                        float p0, p1;
                        split2(t, p0, p1);
                        p0 = exp2_sfu(p0);
                        p1 = exp2_sfu(p1);
                        s2[e & 1] = add2(s2[e & 1], f2(p0, p1));
                        pk[e >> 4][e & 15] = pack_bf16(p0, p1);
                    }
                    float s0, s1;
                    split2(add2(s2[0], s2[1]), s0, s1);
                    part = s0 + s1;
                    // far above the reference, or not a number
                    if (!rare(__any_sync(kFull, !(part <= 4294967296.f))) || again) break;
                    const float mx = row_max();
                    pending = mx > m;
                    rise = mx - m;
                    if (pending) sum *= exp2_sfu(-rise);
                    raise(j * kPParts + x);
                }
                l += part;
                sum += part;
#pragma unroll
                for (int c = 0; c < kPairs / 16; ++c) tmem_st16(ts + x * kPairs + c * 16, pk[c]);
                tmem_wait_st();  // P (and a rescaled O) in TMEM before the products read it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[tile * kPParts + x]);
            }
            if (tile == 0 && j == 0 && lane == 0) mbar_arrive(stagger);
            pending = sum > 256.f;
            rise = __log2f(sum);
        }
        if (cnt > 0) wait(&o_last[tile], 0);
        ok = __all_sync(kFull, ok);
        if (!ok && lane == 0) set_status(p.status, MEDUSA_STATUS_TIMEOUT);
        tc_fence_after();
        if (ok && b >= 0) {
            float o[D];
            if (cnt > 0) {
#pragma unroll
                for (int c = 0; c < D / 16; c += 4) {
                    uint32_t ro[4][16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) tmem_ld16_async(to + (c + x) * 16, ro[x]);
                    tmem_wait_ld(ro);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[(c + x) * 16 + e] = __uint_as_float(ro[x][e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < D; ++e) o[e] = 0.f;
            }
            // The clearing of a chunk precedes every product on it (of either
            // tile: v_clean), so a flag raised for this tile's chunks is visible here.
            if (s_tile[5] && row_ok) {
                const int lo = max(c0 * kPC, (pos0 + 1) / kPC * kPC), hi = min(pos + 1, c1 * kPC);
                for (int key = lo; key < hi; ++key) {
                    const __nv_bfloat16* vr;
                    if (paged) {
                        const int page = p.block_table[(long)b * p.max_pages + key / p.page_size];
                        if (page < 0 || page >= p.num_pages) continue;
                        vr = (const __nv_bfloat16*)p.v +
                             (((long)page * p.Hkv + g) * p.page_size + key % p.page_size) * D;
                    } else {
                        vr = (const __nv_bfloat16*)p.v + (long)(sq.r0 + key) * p.v_stride + g * D;
                    }
#pragma unroll
                    for (int e = 0; e < D; e += 8) {
                        const uint4 w = ld_nc(vr + e);
                        if (nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w)) {
                            float f[8];
                            Elt<__nv_bfloat16>::unpack(w, f);
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if (!isfinite(f[x])) o[e + x] += f[x];
                        }
                    }
                }
            }
            // Rows go through the tile's Q (every product on it is done), 256 bytes of
            // each at a time, so that the warp's stores are whole rows: a store per
            // thread into its own row would touch 32 lines each.
            const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // a NaN sum stays NaN
            const long row0 = (long)(sq.r0 + tok0 + tile * T) * p.Hq + g * G;  // of TMEM lane 0
            if (row_ok) {
                const long orow = row0 + (long)row_tok * p.Hq + row_head;
                const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
                if (C > 1) a.buf.lse2[(long)split * p.N * p.Hq + orow] = lse2;
                else if (p.lse) p.lse[orow] = lse2 * 0.69314718055994531f;
            }
            uint8_t* stage = sQ + tile * kQTile + (warp & 3) * 32 * (2 * D);  // 32 rows of 2 D bytes
            constexpr int kRowVecs = 2 * D / 16;
            auto put = [&](int x, uint4 v) {
                *reinterpret_cast<uint4*>(stage + lane * (2 * D) + ((x ^ lane) & (kRowVecs - 1)) * 16) = v;
            };
            auto store = [&](uint8_t* base, long row_bytes, int off) {
                __syncwarp();
#pragma unroll 4
                for (int x = 0; x < kRowVecs; ++x) {
                    constexpr int kRows = 32 / kRowVecs;  // rows of a store
                    const int r = x * kRows + lane / kRowVecs, c = lane % kRowVecs, q = (warp & 3) * 32 + r;
                    const int t = div_by(q, a.div_G);
                    if (t < T && tile * T + t < ntok)
                        *reinterpret_cast<uint4*>(base + (row0 + (long)(t * p.Hq + q - t * G)) * row_bytes + off +
                                                  c * 16) =
                            *reinterpret_cast<const uint4*>(stage + r * (2 * D) + ((c ^ r) & (kRowVecs - 1)) * 16);
                }
                __syncwarp();
            };
            if (C > 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int x = 0; x < kRowVecs; ++x) {
                        const int e = h * (D / 2) + 4 * x;
                        put(x, make_uint4(__float_as_uint(o[e] * inv), __float_as_uint(o[e + 1] * inv),
                                          __float_as_uint(o[e + 2] * inv), __float_as_uint(o[e + 3] * inv)));
                    }
                    store((uint8_t*)(a.buf.o + (long)split * p.N * p.Hq * D), D * 4, h * (2 * D));
                }
            } else {
#pragma unroll
                for (int x = 0; x < kRowVecs; ++x)
                    put(x, make_uint4(pack_bf16(o[8 * x] * inv, o[8 * x + 1] * inv),
                                      pack_bf16(o[8 * x + 2] * inv, o[8 * x + 3] * inv),
                                      pack_bf16(o[8 * x + 4] * inv, o[8 * x + 5] * inv),
                                      pack_bf16(o[8 * x + 6] * inv, o[8 * x + 7] * inv)));
                store((uint8_t*)p.out, D * 2, 0);
            }
        }
    }
    // every role is done: no product in flight, no copy landing
    tc_fence_before();
    sync_block();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
constexpr size_t prompt_tc_smem() {
    const int bars = 2 + 2 * p_stages<D>() + 7 + 2 * kPParts + kParts;
    return (size_t)(2 * kPM + p_stages<D>() * kPC) * D * 2 + bars * 8 + 48;
}
static_assert(prompt_tc_smem<128>() <= 232448 && prompt_tc_smem<64>() <= 232448, "shared memory of a CTA");

}  // namespace

bool prompt_tc_supported(int page_size, medusa_dtype dt) {
    return dt == MEDUSA_BF16 && (page_size == 0 || attn_tc_page_ok(page_size));
}

size_t prompt_table_bytes(long tiles) { return (size_t)tiles * 2 * sizeof(int4); }

cudaError_t prompt_tc_launch(const PromptArgs& x, long tiles, int splits, const SplitBuf& buf, void* table,
                             cudaStream_t st) {
    PromptTcArgs a;
    const uint64_t D = x.D, Hq = x.Hq, Hkv = x.Hkv, N = x.N;
    a.G = x.Hq / x.Hkv;
    a.T = kPM / a.G;
    a.div_2T = fast_div(2 * a.T);
    a.div_G = fast_div(a.G);
    {
        const uint64_t dims[3] = {D, Hq, N}, strides[2] = {D * 2, (uint64_t)x.q_stride * 2};
        const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.T};
        if (!make_tmap_bf16(&a.mq, x.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (x.block_table) {
        a.page_rows = x.page_size < 64 ? x.page_size : 64;
        const uint64_t ps = x.page_size, NP = (uint64_t)x.num_pages * Hkv;
        const uint64_t dims[3] = {D, ps, NP}, strides[2] = {D * 2, ps * D * 2};
        const uint32_t box[3] = {64, (uint32_t)a.page_rows, 1};
        if (!make_tmap_bf16(&a.mk, x.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
        if (!make_tmap_bf16(&a.mv, x.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
        a.page_rows = kPC;
        const uint64_t dims[3] = {D, Hkv, N};
        const uint64_t ks[2] = {D * 2, (uint64_t)x.k_stride * 2}, vs[2] = {D * 2, (uint64_t)x.v_stride * 2};
        const uint32_t box[3] = {64, 1, (uint32_t)kPC};
        if (!make_tmap_bf16(&a.mk, x.k, 3, dims, ks, box)) return cudaErrorInvalidValue;
        if (!make_tmap_bf16(&a.mv, x.v, 3, dims, vs, box)) return cudaErrorInvalidValue;
    }
    a.p = x;
    a.buf = buf;
    a.scale_log2 = x.scale * 1.4426950408889634f;
    a.wait_ns = wait_limit_ns();
    const bool test = a.wait_ns != kWaitLimitNs;
    void (*kern)(PromptTcArgs) = x.D == 128 ? (test ? prompt_tc_kernel<128, true> : prompt_tc_kernel<128, false>)
                                            : (test ? prompt_tc_kernel<64, true> : prompt_tc_kernel<64, false>);
    const size_t smem = x.D == 128 ? prompt_tc_smem<128>() : prompt_tc_smem<64>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    a.table = (const int4*)table;
    if (table) {
        prompt_table_kernel<<<(unsigned)((tiles + 7) / 8), 256, 0, st>>>(a, (int4*)table, (int)tiles);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * x.Hkv), splits);
    cfg.blockDim = dim3(kPW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = table ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace medusa
