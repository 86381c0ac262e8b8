// Causal attention of packed new rows: whole prompts over their own packed
// K/V, and chunks of new tokens (one token: plain decoding) over a paged
// cache that already holds the chunk's K/V.  This file chooses the kernel and
// holds the CUDA-core one (fp32, and the bf16 shapes the others do not take)
// and the merge of key splits.
//
// For a new token i of sequence b (position p_b + i) and query head h with
// kv-head g = h / (Hq / Hkv):
//     O[h] = sum_{j <= p_b + i} softmax_j(scale <q[h], k_j[g]>) v_j[g]
// by one pass over the keys with a running maximum and sum in fp32.
#include "prompt_common.cuh"

namespace medusa {

namespace {

constexpr int kSimtThreads = 256;

// One CTA takes M = 16 * MI rows (row = token * G + query head of the group)
// of one (sequence, kv-head) and one split of its key chunks.  A 16 x 16 grid
// of threads: thread (ty, tx) holds scores of rows ty + 16 i and keys tx + 16
// j, then output columns 4 tx + 64 c of the same rows, so that a row's maximum
// and sum stay within half a warp.  Tiles are fp32 in shared memory (rows
// padded by 4 floats: 16-byte reads of consecutive rows fall on distinct
// banks); P overlays K.  Bound by latency and by shared-memory reads: a chunk
// takes 6.4 us at 64 columns and 12.8 at 128 (16 rows, up to two CTAs per SM; 64
// rows: 11 and 19).  Three sequences of up to 149 tokens, 4 heads of 64: 11.6 us; 12
// sequences decoding over up to 312 cached tokens, one head of 128: 14.5 us.
template <typename E, int D, int MI>
__global__ void __launch_bounds__(kSimtThreads, 2)
    prompt_simt_kernel(const PromptArgs a, const SplitBuf buf, int T, FastDiv div_T) {
    constexpr int M = 16 * MI, LD = D + 4, LP = kSimtKeys + 4, V4 = Elt<E>::kVec;
    extern __shared__ __align__(16) float sm[];
    float* sQ = sm;
    float* sK = sQ + M * LD;
    float* sV = sK + kSimtKeys * LD;
    float* sP = sK;  // K is read before P is written
    __shared__ PromptTile s_tile;
    __shared__ long s_row[2][kSimtKeys];  // where the keys of this and the next chunk are; < 0: nowhere
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int g = blockIdx.x % a.Hkv, C = gridDim.y, split = blockIdx.y;
    if (C > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge of splits
    if (tid < 32) {
        const PromptTile t = prompt_tile(a, T, div_T, blockIdx.x / a.Hkv);
        if (tid == 0) {
            s_tile = t;
            if (blockIdx.x == 0 && split == 0)
                for (int b = 0; b < a.B; ++b)
                    if (const int bad = prompt_seq(a, b).bad) set_status(a.status, bad);
        }
    }
    __syncthreads();
    const int b = s_tile.b;
    if (b < 0) return;
    const PromptSeq sq = s_tile.s;
    const int G = a.Hq / a.Hkv, tok0 = s_tile.t * T;
    const int ntok = min(T, sq.n - tok0), rows = ntok * G;
    const int keys = sq.p + tok0 + ntok;  // the tile's last token sees [0, keys)
    const int nch = (keys + kSimtKeys - 1) / kSimtKeys;
    const int c0 = (int)((long)nch * split / C), c1 = (int)((long)nch * (split + 1) / C);

    auto load_row = [&](float* dst, const E* src, int c) {  // 16 bytes of a row, widened
        float f[V4];
        Elt<E>::unpack(ld_nc(src + c * V4), f);
#pragma unroll
        for (int i = 0; i < V4; i += 4)
            *reinterpret_cast<float4*>(dst + c * V4 + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    };
    auto zero_row = [&](float* dst, int c) {
#pragma unroll
        for (int i = 0; i < V4; i += 4)
            *reinterpret_cast<float4*>(dst + c * V4 + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    };
    constexpr int CV = D / V4;  // 16-byte pieces per row
    for (int e = tid; e < M * CV; e += kSimtThreads) {
        const int r = e / CV, c = e % CV;
        if (r < rows)
            load_row(sQ + r * LD,
                     (const E*)a.q + (long)(sq.r0 + tok0 + r / G) * a.q_stride + (long)(g * G + r % G) * D, c);
        else zero_row(sQ + r * LD, c);
    }
    int pos[MI];  // the position of each of the thread's rows
    float m[MI], l[MI], o[MI][D / 16];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        pos[i] = sq.p + tok0 + (ty + 16 * i) / G;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    const float scale2 = a.scale * 1.4426950408889634f;
    int bad = 0;
    // A row of the pools or of packed K/V, by the thread of its key, a chunk ahead: the
    // lookup and the loads that depend on it would wait one after the other.
    const long k_stride = a.block_table ? D : a.k_stride, v_stride = a.block_table ? D : a.v_stride;
    const E* const kb = (const E*)a.k + (a.block_table ? 0 : g * D);
    const E* const vb = (const E*)a.v + (a.block_table ? 0 : g * D);
    auto locate = [&](int ch) {
        const int key = ch * kSimtKeys + tid;
        if (tid >= kSimtKeys) return;
        long row = -1;
        if (ch < c1 && key < keys) {
            if (a.block_table) {
                const int page = a.block_table[(long)b * a.max_pages + key / a.page_size];
                if (page >= 0 && page < a.num_pages) row = ((long)page * a.Hkv + g) * a.page_size + key % a.page_size;
                else bad = MEDUSA_STATUS_BAD_PAGE;
            } else {
                row = sq.r0 + key;
            }
        }
        s_row[ch & 1][tid] = row;
    };
    locate(c0);
    for (int ch = c0; ch < c1; ++ch) {
        const int k0 = ch * kSimtKeys, nk = min(kSimtKeys, keys - k0);  // keys that some row sees
        const long* at = s_row[ch & 1];
        __syncthreads();  // P and V of the previous chunk are read
        auto load = [&](float* dst, const E* src, long stride) {  // all of a thread's loads before its stores
            constexpr int kEach = kSimtKeys * CV / kSimtThreads;
            uint4 w[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int e = tid + i * kSimtThreads, r = e / CV, c = e % CV;
                w[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at[r] >= 0) w[i] = ld_nc(src + at[r] * stride + c * V4);
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int e = tid + i * kSimtThreads, r = e / CV, c = e % CV;
                float f[V4];
                Elt<E>::unpack(w[i], f);
#pragma unroll
                for (int x = 0; x < V4; x += 4)
                    *reinterpret_cast<float4*>(dst + r * LD + c * V4 + x) =
                        make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
            }
        };
        load(sK, kb, k_stride);
        load(sV, vb, v_stride);
        locate(ch + 1);
        __syncthreads();
        float s[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qv[MI], kv[4];
#pragma unroll
            for (int i = 0; i < MI; ++i) qv[i] = *reinterpret_cast<const float4*>(sQ + (ty + 16 * i) * LD + d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * j < nk) kv[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (16 * j >= nk) continue;
                    s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                    s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                    s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                    s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                }
        }
        __syncthreads();  // K is read: P may overlay it
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = tx + 16 * j;
                s[i][j] = k0 + r <= pos[i] && at[r] >= 0 ? s[i][j] * scale2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
            const float mn = fmaxf(m[i], mx);
            const float mu = mn == -INFINITY ? 0.f : mn;
            const float al = exp2f(m[i] - mu);
            float rs = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - mu);
                sP[(ty + 16 * i) * LP + tx + 16 * j] = p;
                rs += p;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) rs += __shfl_xor_sync(kFull, rs, w);
            l[i] = l[i] * al + rs;
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= al;
        }
        __syncthreads();
        const bool diag = k0 + kSimtKeys > sq.p + tok0 + 1;  // some row does not see some key
        for (int k = 0; k < nk; k += 4) {
            float4 pv[MI];
#pragma unroll
            for (int i = 0; i < MI; ++i) pv[i] = *reinterpret_cast<const float4*>(sP + (ty + 16 * i) * LP + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                float4 vv[D / 64];
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    vv[c] = *reinterpret_cast<const float4*>(sV + (k + kk) * LD + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    // a later token's V may hold NaN: 0 * NaN must not reach this row
                    if (diag && k0 + k + kk > pos[i]) continue;
                    const float p = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        o[i][4 * c] = fmaf(p, vv[c].x, o[i][4 * c]);
                        o[i][4 * c + 1] = fmaf(p, vv[c].y, o[i][4 * c + 1]);
                        o[i][4 * c + 2] = fmaf(p, vv[c].z, o[i][4 * c + 2]);
                        o[i][4 * c + 3] = fmaf(p, vv[c].w, o[i][4 * c + 3]);
                    }
                }
            }
        }
    }
    if (bad) set_status(a.status, bad);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = ty + 16 * i;
        if (r >= rows) continue;
        const long orow = (long)(sq.r0 + tok0 + r / G) * a.Hq + g * G + r % G;
        const float inv = l[i] > 0.f ? 1.f / l[i] : l[i] == 0.f ? 0.f : l[i];  // a NaN sum stays NaN
        if (C > 1) {
            const long prow = (long)split * a.N * a.Hq + orow;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<float4*>(buf.o + prow * D + 4 * tx + 64 * c) =
                    make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
            if (tx == 0) buf.lse2[prow] = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
            continue;
        }
        E* dst = (E*)a.out + orow * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) dst[4 * tx + 64 * c + x] = Elt<E>::from_float(o[i][4 * c + x] * inv);
        if (a.lse && tx == 0)
            a.lse[orow] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
}

// Merge of the splits of each row, in split order; a warp per row, whose lanes
// read the splits' log2-sum-exps, two each, and then the columns.  A split with
// no visible key has the log2-sum-exp -inf and no weight.  Latency-bound: the
// launch starts under the splits', finds its rows and waits for them.
template <typename E, int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const PromptArgs a, const SplitBuf buf, int C) {
    static_assert(kMaxSplits <= 64, "two splits per lane");
    const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5), rows = (long)a.N * a.Hq;
    const int lane = threadIdx.x & 31;
    const int t = (int)(row / a.Hq);
    // rows of no sequence (behind the last one, past max_new) are left alone
    bool mine = row < rows && t >= a.row_start[0] && t < a.row_start[a.B];
    if (mine) {
        int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.row_start[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        const PromptSeq sq = prompt_seq(a, lo);
        mine = t >= sq.r0 && t < sq.r0 + sq.n;
    }
    // every block waits for the splits, so this launch never ends before them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!mine) return;
    auto lse2 = [&](int s) { return s < C ? buf.lse2[(long)s * rows + row] : -INFINITY; };
    const float x0 = lse2(lane), x1 = lse2(lane + 32);
    const bool nan = __any_sync(kFull, x0 != x0 || x1 != x1);
    float M = fmaxf(x0, x1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    const float w0 = exp2f(x0 - mu), w1 = exp2f(x1 - mu);
    constexpr int PL = D / 32;
    float acc[PL], wsum = 0.f;
#pragma unroll
    for (int e = 0; e < PL; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < C; ++s) {
        const float w = __shfl_sync(kFull, s < 32 ? w0 : w1, s & 31);
        const float* src = buf.o + ((long)s * rows + row) * D + lane * PL;
        wsum += w;
#pragma unroll
        for (int e = 0; e < PL; ++e)
            acc[e] = w == 0.f ? acc[e] : fmaf(w, src[e], acc[e]);  // (a NaN weight is not skipped)
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    E* dst = (E*)a.out + row * D + lane * PL;
#pragma unroll
    for (int e = 0; e < PL; ++e) dst[e] = Elt<E>::from_float(acc[e] * inv);
    if (a.lse && lane == 0)
        a.lse[row] = nan ? NAN : wsum == 0.f ? -INFINITY : (M + log2f(wsum)) * 0.69314718055994531f;
}

template <typename E, int D, int MI>
cudaError_t simt_launch(const PromptArgs& a, long tiles, int T, int splits, const SplitBuf& buf, cudaStream_t st) {
    constexpr int M = 16 * MI;
    const size_t smem = (size_t)(M + 2 * kSimtKeys) * (D + 4) * 4;
    static_assert(M * (kSimtKeys + 4) <= kSimtKeys * (D + 4), "P overlays K");
    auto kern = prompt_simt_kernel<E, D, MI>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    prefer_max_smem(kern);
    kern<<<dim3((unsigned)(tiles * a.Hkv), splits), kSimtThreads, smem, st>>>(a, buf, T, fast_div(T));
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t prompt_dispatch(const PromptArgs& a, cudaStream_t st) {
    const PromptPlan p = prompt_plan(num_sms(), prompt_tc_supported(a.page_size, a.dt), a.B, a.N, a.max_new,
                                     a.max_prefix, a.Hq, a.Hkv);
    const SplitBuf buf = split_buf(a.ws, (long)a.N * a.Hq, D, p.splits);
    cudaError_t e = p.tc ? prompt_tc_launch(a, p.tiles, p.splits, buf, p.table ? a.ws : nullptr, st)
                  : p.M == 16 ? simt_launch<E, D, 1>(a, p.tiles, p.T, p.splits, buf, st)
                              : simt_launch<E, D, 4>(a, p.tiles, p.T, p.splits, buf, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    return prompt_combine_launch(a, buf, p.splits, st);
}

}  // namespace

cudaError_t prompt_combine_launch(const PromptArgs& a, const SplitBuf& buf, int splits, cudaStream_t st) {
    const long rows = (long)a.N * a.Hq;
    void (*kern)(PromptArgs, SplitBuf, int);
    if (a.dt == MEDUSA_F32) kern = a.D == 128 ? prompt_combine_kernel<float, 128> : prompt_combine_kernel<float, 64>;
    else kern = a.D == 128 ? prompt_combine_kernel<__nv_bfloat16, 128> : prompt_combine_kernel<__nv_bfloat16, 64>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, buf, splits);
}

size_t prompt_workspace_size(int B, int N, int max_new, int max_prefix, int Hq, int Hkv, int D, int page_size,
                             medusa_dtype dt) {
    (void)max_new;
    (void)max_prefix;
    // A bound that grows with N (a call with fewer rows may split its keys more):
    // the plan takes no more splits than split_rows has room for.
    const size_t split = split_bytes(split_rows(num_sms(), N, Hq), D);
    const size_t few = decode_supported(B, 1, Hq, Hkv, page_size, dt) ? decode_workspace_size(D) : 0;
    // (a call whose keys are split has a small grid and no table)
    const bool tc = prompt_tc_supported(page_size, dt);
    const size_t table = tc ? prompt_table_bytes(N / prompt_tc_tokens(Hq / Hkv) + (B < N ? B : N)) : 0;
    const size_t most_of = few > split ? few : split;
    return most_of > table ? most_of : table;
}

cudaError_t prompt_launch(const PromptArgs& a, cudaStream_t st) {
    if (a.N == 0 || a.B == 0) return cudaSuccess;
    if (a.block_table && decode_supported(a.B, a.max_new, a.Hq, a.Hkv, a.page_size, a.dt)) return decode_launch(a, st);
    if (a.dt == MEDUSA_F32) return a.D == 128 ? prompt_dispatch<float, 128>(a, st) : prompt_dispatch<float, 64>(a, st);
    return a.D == 128 ? prompt_dispatch<__nv_bfloat16, 128>(a, st) : prompt_dispatch<__nv_bfloat16, 64>(a, st);
}

}  // namespace medusa
