// What the prompt and chunk attention kernels share: the packed batch's
// sequences, the order in which a grid takes its query tiles, and the merge
// of key splits.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "prompt_plan.h"

namespace medusa {

// Sequence b of a packed batch: n new rows from packed row r0 on, at
// positions p .. p + n - 1.
struct PromptSeq {
    int r0, n, p;
    int bad;  // status bits of lengths outside their ranges (clamped here)
};

__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs& a, int b) {
    PromptSeq s;
    s.r0 = a.row_start[b];
    const int r1 = a.row_start[b + 1];
    s.bad = 0;
    s.n = r1 - s.r0;
    if (s.r0 < 0 || r1 < s.r0 || r1 > a.N) {
        s.bad = MEDUSA_STATUS_BAD_LENGTH;
        s.n = 0;
    } else if (s.n > a.max_new) {
        s.bad = MEDUSA_STATUS_BAD_LENGTH;
        s.n = a.max_new;
    }
    s.p = a.prefix_len ? a.prefix_len[b] : 0;
    if (s.p < 0 || s.p > a.max_prefix) {
        s.bad |= MEDUSA_STATUS_BAD_PREFIX;
        s.p = s.p < 0 ? 0 : a.max_prefix;
    }
    if (a.block_table) {  // new rows past the table's last page
        const long room = (long)a.max_pages * a.page_size - s.p;
        if (s.n > room) {
            s.bad |= MEDUSA_STATUS_BAD_LENGTH;
            s.n = room < 0 ? 0 : (int)room;
        }
    }
    return s;
}

// Weight of a tile (tokens [t * T, (t + 1) * T) of its sequence): the number
// of runs of kWeightKeys keys that its last token sees.
constexpr int kWeightKeys = 128;

// Tiles of a sequence with at most w runs of kWeightKeys.
__device__ __forceinline__ int tiles_upto(int n, int p, int T, FastDiv d, int w) {
    const int room = w * kWeightKeys - p;  // (keys stay below 2^30 + 2^30)
    if (n == 0 || room <= 0) return 0;
    return room >= n ? div_by(n - 1, d) + 1 : div_by(room, d);
}

// The tile that comes idx-th when the tiles of all sequences are ordered by
// their number of key chunks, the longest first (so that a grid's last CTAs
// are its shortest), then by sequence.  One warp; every lane returns the
// result; b < 0: fewer tiles than idx + 1.  The weight is found by bisection
// on the count of heavier tiles, so nothing is stored.
struct PromptTile {
    int b, t;
    PromptSeq s;
};
__device__ inline PromptTile prompt_tile(const PromptArgs& a, int T, FastDiv d, int idx) {
    const int lane = threadIdx.x & 31;
    PromptTile r;
    r.b = -1;
    r.t = 0;
    PromptSeq mine;  // the lane's sequence when the batch fits a warp
    mine.r0 = mine.n = mine.p = 0;
    const bool one = a.B <= 32;
    if (one && lane < a.B) mine = prompt_seq(a, lane);
    auto from_lane = [&](const PromptSeq& s, int src) {
        r.s.r0 = __shfl_sync(kFull, s.r0, src);
        r.s.n = __shfl_sync(kFull, s.n, src);
        r.s.p = __shfl_sync(kFull, s.p, src);
    };
    if (a.B == 1) {  // its tiles from the last one back
        from_lane(mine, 0);
        const int nt = r.s.n > 0 ? div_by(r.s.n - 1, d) + 1 : 0;
        if (idx < nt) {
            r.b = 0;
            r.t = nt - 1 - idx;
        }
        return r;
    }
    auto seq = [&](int b) { return one ? mine : prompt_seq(a, b); };
    int total = 0, lo = 0, hi = 0;
    for (int b = lane; b < a.B; b += 32) {
        const PromptSeq s = seq(b);
        total += tiles_upto(s.n, s.p, T, d, INT_MAX / kWeightKeys);
        if (s.n > 0) hi = max(hi, (s.p + s.n + kWeightKeys - 1) / kWeightKeys);
    }
    total = __reduce_add_sync(kFull, total);
    hi = __reduce_max_sync(kFull, hi);
    if (idx >= total) return r;
    auto upto = [&](int w) {  // tiles of weight at most w
        int c = 0;
        for (int b = lane; b < a.B; b += 32) {
            const PromptSeq s = seq(b);
            c += tiles_upto(s.n, s.p, T, d, w);
        }
        return __reduce_add_sync(kFull, c);
    };
    while (lo < hi) {  // the smallest weight with at most idx heavier tiles
        const int mid = (lo + hi) >> 1;
        if (total - upto(mid) <= idx) hi = mid;
        else lo = mid + 1;
    }
    int rank = idx - (total - upto(lo));  // among the tiles of this weight
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int first = 0, cnt = 0;
        PromptSeq s = mine;
        if (b < a.B) {
            s = seq(b);
            first = tiles_upto(s.n, s.p, T, d, lo - 1);
            cnt = tiles_upto(s.n, s.p, T, d, lo) - first;
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(kFull, inc > rank);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.b = b0 + src;
            r.t = __shfl_sync(kFull, first + rank - (inc - cnt), src);
            from_lane(s, src);
            return r;
        }
        rank -= __shfl_sync(kFull, inc, 31);
    }
    return r;
}

// 2^x on the SFU (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float exp2_sfu(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// sign bits set where a half of w (two bf16) is infinite or NaN
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// bf16 pair `w` with its non-finite halves (bits of `bad`) cleared
__device__ __forceinline__ uint32_t clear2(uint32_t w, uint32_t bad) {
    return w & ~((bad >> 15) * 0xffffu);
}

// Partial results of key splits in the workspace.
struct SplitBuf {
    float* o;
    float* lse2;
};
inline SplitBuf split_buf(void* ws, long rows, int D, int splits) {
    SplitBuf s{nullptr, nullptr};
    if (splits > 1) {
        s.o = (float*)ws;
        s.lse2 = (float*)((char*)ws + split_lse_at(splits * rows, D));
    }
    return s;
}
// tensor-core kernel (bf16)
bool prompt_tc_supported(int page_size, medusa_dtype dt);
cudaError_t prompt_tc_launch(const PromptArgs& a, long tiles, int splits, const SplitBuf& buf, void* table,
                             cudaStream_t st);
size_t prompt_table_bytes(long tiles);
// few rows per (sequence, kv-head) over a paged cache (bf16)
bool decode_supported(int B, int max_new, int Hq, int Hkv, int page_size, medusa_dtype dt);
size_t decode_workspace_size(int D);
cudaError_t decode_launch(const PromptArgs& a, cudaStream_t st);
cudaError_t prompt_combine_launch(const PromptArgs& a, const SplitBuf& buf, int splits, cudaStream_t st);

}  // namespace medusa
