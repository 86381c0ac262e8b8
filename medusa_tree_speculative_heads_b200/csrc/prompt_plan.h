// Launch arithmetic of the prompt and chunk attention kernels: tiles, key
// splits and what they take of the workspace, and the division that finds a
// tile.  Builds without CUDA, so that it is checked on a CPU for any number of
// SMs.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MEDUSA_HD __host__ __device__ __forceinline__
#else
#define MEDUSA_HD inline
#endif

namespace medusa {

constexpr int kPromptTcRows = 128;  // rows of a query tile of the tensor-core kernel; a CTA takes two
constexpr int kPromptTcKeys = 128;  // keys per chunk
constexpr int kSimtKeys = 64;       // keys per chunk of the CUDA-core kernel
constexpr int kMaxSplits = 64;

// tokens per CTA of the tensor-core kernel
inline int prompt_tc_tokens(int G) { return 2 * (kPromptTcRows / G); }

// Exact x / T for 0 <= x < 2^31, 1 <= T <= 256, as x * m >> s: with 2^c the power
// of two at or above T, s = 31 + c and m = ceil(2^s / T) (below 2^32: T > 2^(c-1)),
// the excess of m * T over 2^s is below T <= 2^c, so it moves the quotient by less
// than x / 2^31 * 1 / T < 1 / T.
struct FastDiv {
    uint32_t m;
    int s;
};
inline FastDiv fast_div(int T) {
    int c = 0;
    while ((1 << c) < T) ++c;
    return FastDiv{(uint32_t)(((1ull << (31 + c)) + T - 1) / T), 31 + c};
}
MEDUSA_HD int div_by(int x, FastDiv d) { return (int)((uint64_t)(uint32_t)x * d.m >> d.s); }

// upper bound of the tiles of T tokens in a batch of at most N rows
inline long prompt_tiles(int B, int N, int max_new, int T) {
    const long per = ((long)max_new + T - 1) / T;
    const long packed = (long)N / T + (B < N ? B : N);
    return per * B < packed ? per * B : packed;
}

// Partial results of key splits: normalised fp32 rows [splits][N * Hq][D],
// then their log2-sum-exps [splits][N * Hq], each from a 256-byte boundary on.
inline size_t split_lse_at(long rows, int D) { return ((size_t)rows * D * 4 + 255) / 256 * 256; }
inline size_t split_bytes(long rows, int D) { return split_lse_at(rows, D) + ((size_t)rows * 4 + 255) / 256 * 256; }

// Partial rows (splits * N * Hq) that the workspace has room for: the rows of a
// full tile of the tensor-core kernel per SM, and at most kMaxSplits per row.
// Grows with N, so that a workspace serves every call of fewer rows.
inline long split_rows(int sms, int N, int Hq) {
    const long most = (long)sms * 2 * kPromptTcRows, rows = (long)N * Hq * kMaxSplits;
    return rows < most ? rows : most;
}

// The plan of a call: rows per tile, tokens per tile, key splits.
struct PromptPlan {
    bool tc;
    int M, T, splits;
    long tiles;
    bool table;  // the tiles are found by a launch of their own
};

inline PromptPlan prompt_plan(int sms, bool tc, int B, int N, int max_new, int max_prefix, int Hq, int Hkv) {
    PromptPlan p;
    const int G = Hq / Hkv;
    p.tc = tc;
    // CUDA cores: the small tile for up to 16 rows per (sequence, kv-head),
    // decoding, and where the large one leaves SMs idle (three sequences of up to
    // 149 tokens at 4 heads, 24 CTAs of 64 rows: 23.5 us; in tiles of 16: 14.8 us then)
    p.M = p.tc ? 2 * kPromptTcRows : 64;
    if (!p.tc && G <= 16 &&
        ((long)max_new * G <= 16 || prompt_tiles(B, N, max_new, 64 / G) * Hkv < sms))
        p.M = 16;
    p.T = p.tc ? prompt_tc_tokens(G) : p.M / G;
    p.tiles = prompt_tiles(B, N, max_new, p.T);
    const long items = p.tiles * Hkv;
    const int keys = p.tc ? kPromptTcKeys : kSimtKeys;
    const long chunks = ((long)max_prefix + max_new + keys - 1) / keys;
    // one CTA per SM (CUDA cores: two); a split keeps at least 8 of the tensor-core
    // kernel's chunks (the merge launch costs about as much as 4 of them), on CUDA
    // cores, where a chunk takes 6 to 19 us, one
    long s = items > 0 ? (p.tc ? 1L : 2L) * sms / items : 1;
    const long most = chunks / (p.tc ? 8 : 1);
    if (s > most) s = most;
    if (s > kMaxSplits) s = kMaxSplits;
    // The partials are laid out for all N rows.  Tiles that cover them never reach
    // this limit; tiles that do not (rows of no sequence, N > B * max_new) would.
    const long rows = (long)N * Hq, room = split_rows(sms, N, Hq);
    if (rows > 0 && s > room / rows) s = room / rows;
    p.splits = s < 1 ? 1 : (int)s;
    // A CTA of the tensor-core kernel takes up to 3000 cycles to find its tile among
    // several sequences, a launch that finds them all some 3 us.  Without and with it:
    // 64 prompts of 64 tokens (3.5 CTAs per SM) 44.4 and 45.8 us, 8 of 1024 (7) 121.5
    // and 121.6, 128 of 64 (7) 99 and 92, 16 of up to 4096 (10) 250 and 240, 40 of 512
    // (17) 255 and 228.
    p.table = p.tc && B > 1 && p.splits == 1 && p.tiles * Hkv > 4L * sms;
    return p;
}

}  // namespace medusa
